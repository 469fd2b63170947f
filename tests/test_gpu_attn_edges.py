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
