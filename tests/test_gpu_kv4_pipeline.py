"""The 4-bit KV cache in use: kept by the pipeline behind its refresh, read by a
block's attention, grown token by token, cut and read again."""
import numpy as np
import pytest
import torch

import oracle
from drift_aware_kv_spherical_gb300 import polestar as ps
from drift_aware_kv_spherical_gb300 import workloads as wl
from drift_aware_kv_spherical_gb300.kv4 import Kv4Layer
from drift_aware_kv_spherical_gb300.pipeline import Pipeline
from tests._parity import np_

pytestmark = pytest.mark.gpu

W = wl.Workload("kv4_pipe", 91, B=2, N=160, d=256, Hq=4, Hkv=2, dh=64, C=8, iters=3, k=2, P=16,
                V=1024, dtype="bf16", planted=8, noise=1.0, drift_frac=0.1, drift_std=0.5,
                blk_start=64, logit_std=2.0, wq_std=0.05)


@pytest.fixture(autouse=True)
def _lib(lib):
    yield lib
    torch.cuda.synchronize()
    ps.ps_check()


def _inputs(t, H):
    H = H if t == 0 else wl.drift_rows(W, H, t)
    return H


def _bits(c):
    return [np_(x) for x in c.buffers]


def test_pipeline_stores_what_the_refresh_wrote():
    """After every step the 4-bit cache is the encoding of the bf16 cache, and the
    step's other results are those of a pipeline without it."""
    L = wl.make_layer(W, 0, "cuda")
    u, logits = wl.make_uniforms(W, 0, "cuda"), wl.make_logits(W, 0, "cuda")
    pipe, plain = Pipeline(W, layers=1, kv4=True, kmul=0.25, vmul=0.125), Pipeline(W, layers=1)
    H = L["H"]
    acts = [ps.SCHED_REFRESH | ps.SCHED_FULL | ps.SCHED_REINIT, ps.SCHED_REFRESH, ps.SCHED_REFRESH]
    for t, act in enumerate(acts):
        H = _inputs(t, H)
        Q = wl.make_queries(W, H, L["Wq"])
        for p in (pipe, plain):
            p.decode_step(act, [H], [Q], [L["Wk"]], [L["Wv"]], logits, [u])
        st = pipe.state[0]
        for X, i, S in ((st.Kc, 0, 0.25), (st.Vc, 2, 0.125)):
            code, sc = oracle.kv4_encode(np_(X).transpose(0, 2, 1, 3), S)
            assert np.array_equal(_bits(pipe.kv4[0].cache)[i], code), t
            assert np.array_equal(_bits(pipe.kv4[0].cache)[i + 1], sc), t
        for name in ("Kc", "Vc", "D", "mu", "pos", "npos"):
            assert torch.equal(getattr(st, name), getattr(plain.state[0], name)), name


def test_graph_steps_store_too():
    L = wl.make_layer(W, 0, "cuda")
    u, logits = wl.make_uniforms(W, 0, "cuda"), wl.make_logits(W, 0, "cuda")
    a, b = Pipeline(W, layers=1, kv4=True), Pipeline(W, layers=1, kv4=True)
    H = L["H"]
    first = ps.SCHED_REFRESH | ps.SCHED_FULL | ps.SCHED_REINIT
    for t in range(4):
        H = _inputs(t, H)
        Q = wl.make_queries(W, H, L["Wq"])
        args = ([H], [Q], [L["Wk"]], [L["Wv"]], logits, [u])
        a.decode_step(first if t == 0 else ps.SCHED_REFRESH, *args)
        (b.decode_step if t == 0 else b.graph_step)(first if t == 0 else ps.SCHED_REFRESH, *args)
    torch.cuda.synchronize()
    assert all(np.array_equal(x, y) for x, y in zip(_bits(a.kv4[0].cache), _bits(b.kv4[0].cache)))


def test_append_attend_weigh_evict():
    """Tokens appended one by one give the cache of one store; the attention, the
    weight and the cut cache's attention follow the oracle."""
    B, N, Hq, Hkv, dh = 2, 40, 4, 2, 64
    g = torch.Generator().manual_seed(3)
    K = torch.randn(B, N, Hkv, dh, generator=g).bfloat16().cuda()
    V = torch.randn(B, N, Hkv, dh, generator=g).bfloat16().cuda()
    kv = Kv4Layer(B, N, Hq, Hkv, dh, 0.25, 0.25)
    for t in range(30):
        kv.append(K[:, t:t + 1], V[:, t:t + 1])
    one = ps.Kv4Cache.empty(B, Hkv, N, dh, 0.25, 0.25)
    ps.ps_kv4_store(one, K[:, :30], V[:, :30])
    assert all(torch.equal(x, y) for x, y in zip(kv.cache.buffers, one.buffers))
    assert kv.len.tolist() == [30, 30]
    K64 = oracle.kv4_decode(*_bits(one)[:2], 0.25)
    V64 = oracle.kv4_decode(*_bits(one)[2:], 0.25)
    Q = torch.randn(B, 3, Hq, dh, generator=g).bfloat16().cuda()
    O, lse = torch.zeros_like(Q), torch.zeros(B, 3, Hq, device="cuda")
    qn = Q.double().cpu().numpy()
    s = oracle.kv4_scores(qn, K64, dh ** -0.5, length=[30, 30])
    Oref, lref = oracle.kv4_attention(s, V64)
    wref = 0
    for _ in range(2):
        kv.attend(Q, O, lse)
        kv.weigh(Q, lse)
        wref = wref + oracle.kv4_weight(s, lref, Hkv)
    # bf16's half step, P's 11 bits; weights to 2^-14 (scores and lse in fp32)
    assert np.all(np.abs(np_(O) - Oref) <= 2.0 ** -8 * np.abs(Oref) + 2.0 ** -10 * np.abs(V64).max())
    assert np.allclose(np_(lse), lref, rtol=0, atol=1e-4)
    assert np.allclose(np_(kv.w), wref, rtol=2.0 ** -14, atol=1e-7)
    w = np_(kv.w)
    old = kv.cache
    spare = kv.evict(12, sink=1, recent=3)
    assert spare["cache"] is old and kv.len.tolist() == [12, 12]
    at = np.stack([[oracle.kv4_keep(w[b, h], 30, 12, 1, 3) for h in range(Hkv)] for b in range(B)])
    assert np.array_equal(np_(kv.kpos)[:, :, :12], at)
    kv.attend(Q, O, lse, span=torch.tensor([0, 25], dtype=torch.int32,
                                           device="cuda").expand(B, 3, 2).contiguous())
    seen = np.zeros((B, Hkv, N), bool)
    np.put_along_axis(seen, at, True, 2)
    seen[:, :, 25:] = False
    s2 = np.where(np.repeat(seen, Hq // Hkv, 1)[:, None], s, -np.inf)
    Oref, lref = oracle.kv4_attention(s2, V64)
    assert np.all(np.abs(np_(O) - Oref) <= 2.0 ** -8 * np.abs(Oref) + 2.0 ** -10 * np.abs(V64).max())
    kv.evict(8)         # again, from positions to positions
    assert kv.len.tolist() == [8, 8]
    assert np.all(np.isin(np_(kv.kpos)[:, :, :8], at))


def test_example_runs():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "kv4_decode.py")
    spec = importlib.util.spec_from_file_location("kv4_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    cos, share = mod.main(steps=2)
    assert 0.5 <= share <= 1.0 and cos > 0.5
