"""Rows that are computed again, because what they do not see is NaN: many of them, over
long caches, while the kernel's other warps wait."""
import numpy as np
import pytest
import torch

import test_gpu_attn as base

pytestmark = pytest.mark.gpu
ps = pytest.importorskip("drift_aware_kv_spherical_gb300.polestar")


@pytest.mark.parametrize("Tq,n,H,dh", [(1280, 100000, 32, 64), (700, 5001, 4, 128)])
def test_many_rows_over_long_caches(Tq, n, H, dh):
    """Every other row starts behind a slot that holds NaN in its tile."""
    g = torch.Generator(device="cuda").manual_seed(n)
    make = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    Q, K, V = make(Tq, H, dh), make(n, H, dh), make(n, H, dh)
    V[5] = float("nan")
    i32 = dict(dtype=torch.int32, device="cuda")
    span = torch.tensor([[6, n], [0, n]], **i32).repeat(Tq // 2, 1)
    O, lse = torch.zeros_like(Q), torch.zeros(Tq, H, device="cuda")
    ws = ps.workspace(ps.OP_ATTN, B=1, N=n, Hq=H, Hkv=H, dh=dh, P=Tq, k=Tq)
    ps.ps_attn(Q, K, V, O, lse, q_off=torch.tensor([0, Tq], **i32),
               k_off=torch.tensor([0, n], **i32), span=span, max_q=Tq, max_k=n, ws=ws)
    ps.ps_check()
    assert torch.isnan(O[1::2]).all() and torch.isfinite(lse).all()
    assert torch.isfinite(O[::2]).all()
    at = slice(0, None, 10)
    for h in (0, H - 1):
        q = Q[at, h].double()
        s = (q @ K[6:, h].double().T) * dh ** -0.5
        L = torch.logsumexp(s, 1)
        p = torch.exp(s - L[:, None])
        v = V[6:, h].double()
        want, size = p @ v, p @ v.abs()
        # scores: fp32 sums, 2^-20 of |q| |k| scale; weights and the result each half a step
        W = dh ** -0.5 * q.norm(dim=1) * K[:, h].double().norm(dim=1).max()
        err = 2.0 ** -20 * (3 + W)
        tol = size * (2.0 ** -8 + 2 * err[:, None])
        assert ((O[at, h].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()
        assert ((lse[at, h].double() - L).abs() <= err + 2.0 ** -22 * (1 + L.abs())).all()


@pytest.mark.parametrize("Hq,Hkv,dh", [(28, 4, 128), (8, 8, 64), (5, 1, 80)])
def test_rows_of_several_sequences(Hq, Hkv, dh):
    """More items than SMs for the first shape, sequences without rows among them."""
    r = np.random.RandomState(Hq)
    q = np.array([300, 0, 513, 40, 0, 2, 900, 9])
    k = q + r.randint(5, 200, len(q))
    q_off, k_off = (np.concatenate([[0], np.cumsum(x)]) for x in (q, k))
    Q, K, V = base._data(dh, int(q_off[-1]), int(k_off[-1]), Hq, Hkv, dh, torch.bfloat16)
    span = np.zeros((len(Q), 2), np.int64)
    span[:, 1] = 1 << 20
    span[r.rand(len(Q)) < 0.5, 0] = 4
    V[torch.from_numpy(k_off[:-1]).cuda() + 3] = float("nan")
    a = (q_off, k_off[:-1], k)
    for causal in (False, True):
        O, lse = base._run(Q, K, V, *a, span=span, causal=causal)
        base._near(O, lse, Q, K, V, *a, span=span, causal=causal)
    ps.ps_check()
