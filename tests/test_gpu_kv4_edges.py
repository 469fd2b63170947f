"""The 4-bit KV cache at the edges of what its calls take: arrays that start at
any element, bounds and positions at the ends of their type, caps of any size,
more rows than 2^24, signed zeros and quotients out of range."""
import numpy as np
import pytest
import torch

import oracle
from drift_aware_kv_spherical_gb300 import polestar as ps
from tests._parity import Guarded, np_
from tests.test_gpu_kv4 import BF16, F32, _attn, _cache, _check_attn, _i32, _query, _tol

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    yield lib
    torch.cuda.synchronize()
    ps.ps_check()


def _weight(c, Q, lse, **opt):
    w = torch.zeros(c.B, c.Hkv, c.N, device="cuda")
    ps.ps_kv4_weight(c, Q, lse, None, w, **opt)
    return w


def _at_element_1(x):
    """x in memory that starts one element behind an aligned address."""
    buf = torch.zeros(x.numel() + 1, dtype=x.dtype, device=x.device)
    y = buf[1:].view(x.shape)
    y.copy_(x)
    return y


@pytest.mark.parametrize("T", [1, 10, 40, 150])
@pytest.mark.parametrize("with_pos", [False, True])
def test_arrays_that_start_at_any_element(T, with_pos):
    """len, span, kpos, qpos, slope, lse and the weights at an odd element give the
    bits that aligned ones give, in every kernel."""
    B, Hq, Hkv, dh, N = 2, 4, 2, 64, 300
    rng = np.random.default_rng(T)
    c, _, _ = _cache(B, Hkv, N, dh, T)
    Q, _ = _query(B, T, Hq, dh, BF16, T)
    lo = rng.integers(0, 200, (B, T))
    opt = dict(len=_i32([N, 280]), span=_i32(np.stack([lo, lo + 90], -1)),
               qpos=_i32(rng.integers(0, N, (B, T))),
               slope=torch.tensor([0.5, 0.25, 0.125, 0.0625], device="cuda"),
               kpos=_i32(np.stack([[rng.permutation(N) for _ in range(Hkv)] for _ in range(B)]))
               if with_pos else None)
    odd = {k: None if v is None else _at_element_1(v) for k, v in opt.items()}
    assert odd["span"].data_ptr() % 8 == 4
    O, lse = _attn(c, Q, scale=0.125, **opt)
    O2, lse2 = torch.zeros_like(Q), _at_element_1(torch.zeros_like(lse))
    ps.ps_kv4_attn(c, Q, O2, lse2, scale=0.125, ws=ps.workspace(
        ps.OP_KV4_ATTN, B=B, N=N, Hq=Hq, Hkv=Hkv, dh=dh, P=T), **odd)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    w0 = torch.rand(B, Hkv, N, device="cuda")
    w, w2 = torch.zeros_like(w0), _at_element_1(torch.zeros_like(w0))
    ps.ps_kv4_weight(c, Q, lse, w0, w, scale=0.125, **opt)
    ps.ps_kv4_weight(c, Q, lse2, _at_element_1(w0), w2, scale=0.125, **odd)
    assert torch.equal(w, w2)
