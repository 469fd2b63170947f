"""Attention over packed sequences and cache rows: infinite keys that a row sees, few rows
beside long prompts on long caches."""
import numpy as np
import pytest
import torch

import test_gpu_attn as base

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dh", [64, 208])
@pytest.mark.parametrize("T,n", [(1, 200), (1, 9000), (20, 200), (20, 9000), (150, 300),
                                 (700, 1500)])
def test_keys_of_minus_infinity_have_no_weight(dtype, dh, T, n):
    """Queries of few bits, positive where some seen keys are -inf: a score of -inf, which
    leaves O and lse what the other slots make them."""
    Q, K, V = base._data(T + n, T, n, 4, 2, dh, dtype)
    Q = (torch.sign(Q) * 2.0 ** torch.randint(-2, 2, Q.shape, device="cuda")).to(dtype)
    Q[..., 0], Q[..., 3] = 1.0, 0.5
    K[5, :, 3], K[n - 1, :, 0], K[n // 2, 1, 3] = (-float("inf"),) * 3
    a = (np.array([0, T]), np.array([0]), np.array([n]))
    O, lse = base._run(Q, K, V, *a)
    base._near(O, lse, Q, K, V, *a)
    assert torch.isfinite(O).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("Hq,Hkv,dh", [(4, 4, 128), (28, 4, 64), (8, 8, 80), (4, 1, 128)])
@pytest.mark.parametrize("causal", [False, True])
def test_few_rows_beside_a_prompt_on_long_caches(Hq, Hkv, dh, causal):
    """Sequences of up to eight rows a KV head in more shares than a cluster holds, their
    partial sums by sequence."""
    q = [300, 1, 2, 0, 1, 1, 8, 40]
    k = [4000, 30000, 9, 100, 20000, 0, 12345, 7000]
    base._check(Hq + dh, q, k, Hq, Hkv, dh, BF, gap=2, pad=3, causal=causal)
    base._check(Hq, [2000, 1], [2000, 33000], Hq, Hkv, dh, BF, causal=causal)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1.0])
def test_rows_without_a_score_above_minus_infinity(dtype, T, bad):
    """All that they see has no weight: O is 0 whatever V holds, lse -inf."""
    Q, K, V = base._data(T, T, 3, 4, 2, 64, dtype)
    Q = torch.sign(Q)
    Q[..., 3] = 0.5
    K[1:, :, 3] = -float("inf")
    V[1:, :, ::5] = bad
    span = np.tile([[1, 3]], (T, 1))
    span[::3] = [[0, 1]]              # these see the one slot that is like others
    a = (np.array([0, T]), np.array([0]), np.array([3]))
    O, lse = base._run(Q, K, V, *a, span=span)
    rest = np.arange(T) % 3 != 0
    assert not O[rest].any() and torch.isneginf(lse[rest]).all()
    one = len(O[::3])
    base._near(O[::3], lse[::3], Q[::3], K[:1], V[:1], np.array([0, one]), np.array([0]),
               np.array([1]))         # (fp32: V's two tf32 terms leave 2^-22 of it)
