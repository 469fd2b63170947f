"""Rotary positions on the GPU: how exact an angle is."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ps = pytest.importorskip("drift_aware_kv_spherical_gb300.polestar")


@pytest.mark.parametrize("sign", [1, -1])
def test_angles_are_good_to_2_25_radians(sign):
    """Angles between an eighth and a sixteenth of a turn whose 30 bits end in 15.9 of 32
    units of 2^-32 turns: what fp32 holds of them is off by nearly half a step, 16 units or
    2.35e-8 radians, and always the same way.  sin and cos of 50 thousand such angles are
    each rounded, to 2 ulp at most and either way, so that the mean of what they say of the
    angle is good to 2^-22 / sqrt(50000) = 2^-29.8: 2^-25 holds, 2^-26 does not."""
    table = ps.RopeTable(16, 2, base=1.0)
    turns = np.uint64(table.turns.cpu().numpy().view(np.uint64)[0])
    found = []
    for at in range(0, 1 << 26, 1 << 22):
        p = (sign * np.arange(at, at + (1 << 22), dtype=np.int64))
        t = p.astype(np.uint64) * turns
        hi = t >> np.uint64(32)
        rest = (hi & np.uint64((1 << 30) - 1)).astype(np.int64)
        low = t & np.uint64(0xffffffff)
        at = (rest >= 1 << 28) & (rest < 1 << 29) & (rest % 32 == 15) & (low >= 0xe6000000)
        found.append((p[at], t[at]))
    pos, t = (np.concatenate(x) for x in zip(*found))
    assert len(pos) > 40000
    K = torch.zeros(1, len(pos), 1, 16, device="cuda")
    K[..., 0] = 1.0
    ps.ps_rope(table, K=K, pos=torch.from_numpy(pos.astype(np.int32)[None]).cuda())
    c, s = K[0, :, 0, 0].double().cpu().numpy(), K[0, :, 0, 1].double().cpu().numpy()
    quarter = (t >> np.uint64(62)).astype(np.float64)
    a = (t & np.uint64((1 << 62) - 1)).astype(np.float64) * 2.0 ** -64 * 2 * np.pi
    a += quarter * np.pi / 2      # (some 2^-52 radians)
    off = s * np.cos(a) - c * np.sin(a)
    assert abs(off.mean()) <= 2.0 ** -25
    assert np.abs(off).max() <= 2.0 ** -22
