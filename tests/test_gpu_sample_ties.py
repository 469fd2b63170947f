"""Draws among ties, every row decided: cuts in the middle of a value, and on a border."""
import numpy as np
import pytest
import torch

import oracle
import test_gpu_sample as base

pytestmark = pytest.mark.gpu


def _spread(kind, r, R, V):
    return dict(flat=lambda: np.full((R, V), 1.25), two=lambda: r.randint(0, 2, (R, V)) * 3.0,
                coarse=lambda: np.round(r.randn(R, V)), tiny=lambda: r.randn(R, V) * 1e-30,
                wide=lambda: r.randn(R, V) * 1e4,
                near_zero=lambda: np.abs(r.randn(R, V)) ** 9 * 1e-3,
                lowest=lambda: np.where(r.rand(R, V) < 0.7, float(np.finfo(np.float32).min),
                                        r.randn(R, V)))[kind]()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5, 3000, 40000])
@pytest.mark.parametrize("kind", ["flat", "two", "coarse", "tiny", "wide", "near_zero", "lowest"])
def test_ties_and_extreme_spreads_without_a_border(V, kind, dtype):
    """Shares of the mass that end inside an element, however many are alike."""
    r = np.random.RandomState(V)
    R = 12
    x = torch.from_numpy(_spread(kind, r, R, V)).to(dtype).cuda()
    u = r.rand(R)
    base._check(x, u)
    for k in (1, 2, V // 2, V - 1):
        base._check(x, u, top_k=[k] * R)
    for p in (0.00129, 0.370107, 0.99319):
        base._check(x, u, top_p=[p] * R)
        base._check(x, u, top_p=[p] * R, top_k=[max(V // 3, 1)] * R)
    base._check(x, u, temperature=[0.05, 20.0] * (R // 2), top_p=[0.7707] * R, min_p=[0.01] * R)


@pytest.mark.parametrize("shift", [0.0, -30.0, 40.0])
@pytest.mark.parametrize("std", [1e-5, 0.3, 3.0, 1e20])
def test_bf16_values_near_zero_and_far_apart_without_a_border(shift, std):
    r = np.random.RandomState(int(shift) % 97)
    R, V = 8, 5003
    x = torch.from_numpy(r.randn(R, V) * std + shift).bfloat16()
    x[:, ::7] = 0.0
    x[:, ::11] = -1e-30
    x = x.cuda()
    t = [1.0, 0.3, 5.0, 1e19] * 2
    for k in (1, 40, 700, V - 1):
        base._check(x, r.rand(R), top_k=[k] * R, temperature=t)
    for p in (0.01234, 0.5037, 0.9511):
        base._check(x, r.rand(R), top_p=[p] * R, temperature=t)
        base._check(x, r.rand(R), top_p=[p] * R, top_k=[500] * R, min_p=[0.02] * R, temperature=t)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [3000, 40000])
@pytest.mark.parametrize("kind", ["flat", "tiny"])
@pytest.mark.parametrize("p", [0.001, 0.37])
def test_a_share_of_equal_weights_that_ends_on_an_element(V, kind, dtype, p):
    """p V is a whole number but for fp32's rounding of p, so the element on the border is in
    or out: n is the whole number or one more, and all else follows from n.  Of equal w the
    token is the one of place floor(u n) by index, prob 1 / n."""
    r = np.random.RandomState(V)
    R = 12
    x = torch.from_numpy(_spread(kind, r, R, V)).to(dtype).cuda()
    u = (r.randint(0, V, R) + 0.5) / V        # (u n is no whole number)
    token, prob, n = base._draw(x, u, top_p=[p] * R)
    l = x.double().cpu().numpy()
    whole = round(p * V)
    for i in range(R):
        assert n[i] in (whole, whole + 1)
        left = np.sort(np.argsort(-l[i], kind="stable")[:n[i]])
        assert token[i] == left[int(np.floor(u[i] * n[i]))]
        assert abs(prob[i] * n[i] - 1) <= 2.0 ** -22
        want = oracle.sample(l[i], u[i], top_p=float(np.float32(p)))
        assert abs(want[2] - n[i]) <= 1
