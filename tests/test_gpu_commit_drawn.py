"""The commit rule on confidences that are no probabilities."""
import numpy as np
import pytest
import torch

import test_gpu_sample as base

pytestmark = pytest.mark.gpu
ps = pytest.importorskip("drift_aware_kv_spherical_gb300.polestar")


@pytest.mark.parametrize("B,P", [(3, 40), (2, 7), (1, 1024)])
@pytest.mark.parametrize("kind", ["logs", "infinite", "nan"])
def test_progress_with_any_confidences(B, P, kind):
    """Logarithms of probabilities, all below -1; -inf; NaN, which counts as -inf: the
    largest is committed when nothing else is."""
    r = np.random.RandomState(P)
    c = (-1.5 - 3 * r.rand(B, P)).astype(np.float32)
    if kind == "infinite":
        c[:] = -np.inf
    elif kind == "nan":
        c[r.rand(B, P) < 0.5] = np.nan
        c[:, 0] = np.nan
        c[0] = np.nan
    role = r.choice([0, 0, 1, 2], P).astype(np.uint8)
    role[[0, P - 1]] = 0
    und = (r.rand(B, P) < 0.8).astype(np.uint8)
    und[:, 0] = 1
    D = r.rand(B, P).astype(np.float32)
    cuda = lambda x: torch.from_numpy(x.copy()).cuda()  # noqa: E731
    for mode in range(3):
        params = ps.CommitParams(-1.0, 1.0, 0.3, mode, 1)
        u, d_sum, d_cnt, d_prev = (cuda(und), cuda(D * 0), cuda(np.zeros((B, P), np.int32)),
                                   cuda(D * 0))
        commit = torch.zeros(B, P, dtype=torch.uint8, device="cuda")
        ps.ps_commit_drawn(cuda(c), cuda(role), u, cuda(D), P, d_sum, d_cnt, d_prev, None, P,
                           params, commit)
        for b in range(B):
            state = dict(undecided=und[b].copy(), d_sum=D[b] * 0, d_cnt=np.zeros(P, np.int32),
                         d_prev=D[b] * 0)
            x = np.where(np.isnan(c[b]), -np.inf, c[b]).astype(np.float64)
            want = base._rule(x, role, D[b], np.zeros(P, np.uint8), state, params)
            assert want.sum() == 1
            assert np.array_equal(commit[b].cpu().numpy(), want)
            assert np.array_equal(u[b].cpu().numpy(), state["undecided"])
            assert np.array_equal(d_cnt[b].cpu().numpy(), state["d_cnt"])
