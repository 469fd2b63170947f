"""Rotary positions on the GPU: slots that are named twice, entries that are there twice."""
import pytest
import torch

pytestmark = pytest.mark.gpu
ps = pytest.importorskip("drift_aware_kv_spherical_gb300.polestar")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_slot_named_twice_holds_elements_of_either_row(dtype):
    """And an entry that is there twice writes the same twice."""
    g = torch.Generator().manual_seed(3)
    B, T, H, dh = 2, 300, 4, 64
    table = ps.RopeTable(dh, 32)
    K, V = (torch.randn(B, T, H, dh, generator=g).to(dtype).cuda() for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    pos = torch.arange(T, **i32).repeat(B, 1)
    each = torch.zeros(B, T, H, dh, dtype=dtype, device="cuda")
    ps.ps_rope(table, K=K, V=V, cache=(each, torch.zeros_like(each)), pos=pos)
    dst = (pos // 2).contiguous()
    Kc, Vc = (torch.zeros(B, T, H, dh, dtype=dtype, device="cuda") for _ in range(2))
    ps.ps_rope(table, K=K, V=V, cache=(Kc, Vc), pos=pos, dst=dst)
    for got, src in ((Kc, each), (Vc, V)):
        assert ((got[:, :T // 2] == src[:, ::2]) | (got[:, :T // 2] == src[:, 1::2])).all()
        assert not got[:, T // 2:].any()
    rows = torch.randint(0, T, (B, T), **i32)
    Kc.zero_()
    ps.ps_rope(table, K=K, V=V, cache=(Kc, Vc), pos=pos, rows=rows)
    for b in range(B):
        named = torch.zeros(T, dtype=torch.bool, device="cuda")
        named[rows[b].long()] = True
        assert torch.equal(Kc[b, named], each[b, named]) and not Kc[b, ~named].any()
