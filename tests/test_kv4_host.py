"""Host side of the 4-bit KV cache's calls, without a GPU: workspace sizes,
refusals before any CUDA call, the binding's layout checks."""
import ctypes
import os

import pytest
import torch


@pytest.fixture(scope="module")
def ps():
    from drift_aware_kv_spherical_gb300 import _build, polestar
    if not os.path.exists(polestar.LIB_PATH):
        _build.build()
    polestar.Library.load()
    return polestar


def test_workspace_sizes(ps):
    size = lambda **k: ps.ps_workspace_bytes(ps.OP_KV4_ATTN, **k)  # noqa: E731
    full = dict(B=8, N=65536, Hq=28, Hkv=4, dh=128, P=1)
    assert size(**full) % 256 == 0
    assert size(**full) >= 8 * 28 * 9 * (128 + 2) * 4    # more shares than a cluster holds
    assert size(B=1, N=64, Hq=4, Hkv=4, dh=64, P=1) == 0  # one share
    for bad in (dict(B=0), dict(N=0), dict(Hq=30), dict(Hkv=0), dict(dh=96), dict(P=0)):
        assert size(**{**full, **bad}) == 0, bad
    assert ps.ps_workspace_bytes(ps.OP_KV4_EVICT, B=2, N=100, Hkv=3, k=50) >= 2 * 3 * 50 * 4
    assert ps.ps_workspace_bytes(ps.OP_KV4_EVICT, B=2, N=100, Hkv=0, k=50) == 0


def test_null_arguments_are_refused_on_the_host(ps):
    cd = ps.Library.load().cdll
    err = ps.PS_ERR_ARG
    assert cd.ps_kv4_store(None, None, None, None, 0, 1, 64, 64, None, None, None, None) == err
    assert cd.ps_kv4_load(None, None, None, None, 0, 1, 64, 64, None, None, None, None) == err
    assert cd.ps_kv4_attn(None, None, None, None, None, None, 0, None) == err
    assert cd.ps_kv4_weight(None, None, None, None, None, None, None, 0, None) == err
    assert cd.ps_kv4_evict(None, None, None, None, None, None, 1, 0, 0, None, None, None, None, 0,
                           None) == err


def test_structs_match_the_header(ps):
    """The packed arguments have the layout of ps_kv4_cache and ps_kv4_query."""
    class Cache(ctypes.Structure):
        _fields_ = [(n, ctypes.c_void_p) for n in ("kcode", "kscale", "vcode", "vscale")] + \
                   [(n, ctypes.c_int) for n in ("B", "Hkv", "Ncache", "dh")] + \
                   [("kmul", ctypes.c_float), ("vmul", ctypes.c_float)]

    class Query(ctypes.Structure):
        _fields_ = [(n, ctypes.c_void_p) for n in ("Q", "len", "span", "kpos", "qpos", "slope")] + \
                   [(n, ctypes.c_int64) for n in ("q_bld", "q_ld")] + [(n, ctypes.c_int) for n in ("dtype", "T", "Hq")] + \
                   [("scale", ctypes.c_float), ("cap", ctypes.c_float)]

    c = Cache.from_buffer_copy(ps.Kv4Cache._pack.pack(1, 2, 3, 4, 5, 6, 7, 8, 0.5, 0.25))
    assert (c.kcode, c.vscale, c.B, c.dh, c.kmul, c.vmul) == (1, 4, 5, 8, 0.5, 0.25)
    raw = ps._Q_PACK.pack(1, 2, 3, 4, 5, 6, 1 << 41, 1 << 40, 1, 9, 10, 2.0, 30.0)
    q = Query.from_buffer_copy(raw.ljust(ctypes.sizeof(Query), b"\0"))
    assert (q.Q, q.slope, q.q_bld, q.q_ld, q.dtype, q.T, q.Hq, q.scale, q.cap) == \
        (1, 6, 1 << 41, 1 << 40, 1, 9, 10, 2.0, 30.0)


class _Dev:
    """A CPU tensor that says it is on the device: the binding's layout checks
    look at shapes and strides only."""

    def __init__(self, t):
        self.t, self.shape, self.is_cuda = t, t.shape, True

    def stride(self):
        return self.t.stride()

    def is_contiguous(self):
        return self.t.is_contiguous()

    def numel(self):
        return self.t.numel()


def test_row_strides(ps):
    x = torch.zeros(2, 5, 12, 8)
    assert ps._rows_ld(_Dev(x), 2, 12, 8) == (5, 480, 96)
    assert ps._rows_ld(_Dev(x[:, :, 4:8]), 2, 4, 8) == (5, 480, 96)
    assert ps._rows_ld(_Dev(x[:, 1:3]), 2, 12, 8) == (2, 480, 96)
    assert ps._rows_ld(_Dev(x[:, ::2]), 2, 12, 8) == (3, 480, 192)
    assert ps._rows_ld(_Dev(x[:, :1, :3]), 2, 3, 8) == (1, 480, 24)
    assert ps._rows_ld(_Dev(x[:1, 1:4, :5]), 1, 5, 8) == (3, 0, 96)
    for bad in (x.transpose(1, 2)[:, :, :5], x[:, :, ::2], x[..., ::2]):
        with pytest.raises(ValueError):
            ps._rows_ld(_Dev(bad), 2, bad.shape[2], bad.shape[3])
    with pytest.raises(ValueError):
        ps._rows_ld(_Dev(x), 2, 11, 8)
