"""The 4-bit KV cache on the GPU against the fp64 oracle: rows in and out and
eviction bit-exact; attention and its weight within bounds derived from the
operands' rounding (see _tol)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from drift_aware_kv_spherical_gb300 import polestar as ps
from tests._parity import Guarded, np_

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _lib(lib):
    yield lib
    torch.cuda.synchronize()
    ps.ps_check()


def _cache(B, Hkv, N, dh, seed, kmul=0.25, vmul=0.125, junk_from=None):
    """A cache of random rows (encoded by the oracle) and its K, V in fp64.
    Slots >= junk_from[b] hold 0xFF bytes (NaN scales), as unstored memory may."""
    rng = np.random.default_rng(seed)
    K = (rng.standard_normal((B, Hkv, N, dh)) * np.exp(0.4 * rng.standard_normal(dh)))
    V = rng.standard_normal((B, Hkv, N, dh)) * 0.7
    kc, ks = oracle.kv4_encode(K.astype(np.float32), kmul)
    vc, vs = oracle.kv4_encode(V.astype(np.float32), vmul)
    K, V = oracle.kv4_decode(kc, ks, kmul), oracle.kv4_decode(vc, vs, vmul)
    if junk_from is not None:
        for b, n in enumerate(junk_from):
            for x in (kc, ks, vc, vs):
                x[b, :, n:] = 0xFF
    c = ps.Kv4Cache(*(torch.from_numpy(x).cuda() for x in (kc, ks, vc, vs)), kmul=kmul, vmul=vmul)
    return c, K, V


def _i32(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def _query(B, T, Hq, dh, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    Q = (torch.randn(B, T, Hq, dh, generator=g) * std).to(dtype)
    return Q.cuda(), Q.double().numpy()


def _tol(Q, K, V, scale, cap, dtype):
    """(score error, output error) bounds.

    Scores: products of f16 operands are exact (fp32 queries: two f16 terms,
    2^-22 relative); dh / 16 accumulations of 16 products, each to 2^-22 of the
    largest partial sum, at most scale * sum |q k|; the cap's tanh to 2^-22 of
    the cap; fp32 steps to log2 units and ex2 to 2^-21 of |s| + 1.
    Output: weights to e^(2 ds) - 1, P to 2^-11 (bf16 queries) or 2^-21 of
    each, sums to 2^-19; then bf16's half step of 2^-8."""
    sabs = scale * np.einsum("bthd,bhd->bth", np.abs(Q),
                             np.repeat(np.abs(K).max(2), Q.shape[2] // K.shape[1], 1)).max()
    top = min(sabs, cap) if cap > 0 else sabs
    ds = 2.0 ** -22 * (sabs * (Q.shape[3] / 16 + 2) + 2 * cap) + 2.0 ** -21 * (top + 1)
    dp = np.expm1(2 * ds) + (2.0 ** -11 if dtype == BF16 else 2.0 ** -21) + 2.0 ** -19
    return ds, dp * np.abs(V).max()


def _check_attn(O, lse, Oref, lref, ds, do, dtype, what=""):
    O, lse = O.double().cpu().numpy(), lse.double().cpu().numpy()
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -23
    err = np.abs(O - Oref) - half * np.abs(Oref)
    assert err.max() <= do, (what, err.max(), do)
    dead = np.isneginf(lref)
    assert np.all(np.isneginf(lse[dead])) and np.all(O[dead] == 0), what
    e = np.abs(lse[~dead] - lref[~dead])
    lim = 2 * ds + 2.0 ** -20 * (1 + np.abs(lref[~dead]))
    assert np.all(e <= lim), (what, e.max(), ds)


def _masks(kind, B, T, N, Hkv, seed):
    """(len, span, qpos, kpos) of a mask kind."""
    rng = np.random.default_rng(seed)
    length = rng.integers(0, N + 1, B)
    length[0] = N
    qpos = rng.integers(0, N, (B, T))
    span = np.zeros((B, T, 2), np.int64)
    kpos = None
    if kind == "none":
        return None, None, qpos, None
    if kind == "len":
        return length, None, qpos, None
    if kind == "causal":
        span[..., 1] = qpos + 1
    elif kind == "documents":        # short spans, some empty, some reversed, some past the end
        span[..., 0] = rng.integers(-5, N, (B, T))
        span[..., 1] = span[..., 0] + rng.integers(-3, max(2, N // 3), (B, T))
        span[0, 0] = [N, N + 100]
    elif kind == "kpos":
        span[..., 1] = qpos + 1
        kpos = np.stack([[rng.permutation(N) * 3 for _ in range(Hkv)] for _ in range(B)])
        qpos = qpos * 3
        span = span * 3
    return length, span, qpos, kpos


CASES = [  # B, T, Hq, Hkv, dh, N, dtype, mask, cap, bias
    (1, 1, 4, 4, 64, 1, BF16, "none", 0, False),
    (1, 1, 4, 4, 128, 17, BF16, "len", 0, False),
    (2, 1, 28, 4, 128, 1000, BF16, "len", 0, False),
    (2, 1, 28, 4, 128, 777, F32, "len", 0, True),
    (1, 1, 8, 1, 256, 333, BF16, "none", 30.0, False),
    (3, 2, 32, 2, 64, 130, BF16, "documents", 0, False),
    (2, 16, 4, 4, 64, 128, F32, "causal", 0, False),
    (2, 32, 4, 4, 128, 768, BF16, "len", 0, False),
    (2, 33, 14, 2, 128, 517, BF16, "documents", 50.0, True),
    (1, 5, 6, 2, 256, 259, F32, "documents", 20.0, True),
    (1, 130, 4, 2, 128, 300, BF16, "causal", 0, False),
    (2, 130, 2, 2, 64, 257, F32, "documents", 0, True),
    (1, 100, 8, 2, 64, 201, BF16, "kpos", 0, True),
    (2, 70, 6, 2, 128, 385, BF16, "kpos", 25.0, False),
    (1, 300, 2, 1, 128, 1023, BF16, "documents", 0, True),
    (1, 257, 4, 4, 128, 640, BF16, "none", 0, False),
    (1, 129, 7, 1, 256, 200, BF16, "causal", 0, False),
    (1, 1, 2, 2, 128, 4111, BF16, "kpos", 0, True),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,dh,N,dtype,mask,cap,bias", CASES)
def test_attention_and_weight(B, T, Hq, Hkv, dh, N, dtype, mask, cap, bias):
    seed = B + 3 * T + 7 * Hq + N
    length, span, qpos, kpos = _masks(mask, B, T, N, Hkv, seed)
    c, K, V = _cache(B, Hkv, N, dh, seed, junk_from=length)
    Q, Qn = _query(B, T, Hq, dh, dtype, seed, 1.5)
    scale = dh ** -0.5
    slope = (0.5 ** np.arange(1, Hq + 1)).astype(np.float32) if bias else None
    opt = dict(scale=scale, len=_i32(length), span=_i32(span), kpos=_i32(kpos),
               qpos=_i32(qpos) if bias else None,
               slope=torch.from_numpy(slope).cuda() if bias else None, cap=float(cap))
    sizes = dict(B=B, N=N, Hq=Hq, Hkv=Hkv, dh=dh, P=T)
    O, lse = Guarded((B, T, Hq, dh), dtype, fill=7), Guarded((B, T, Hq), F32, fill=7)
    ps.ps_kv4_attn(c, Q, O.t, lse.t, ws=ps.workspace(ps.OP_KV4_ATTN, **sizes), **opt)
    s = oracle.kv4_scores(Qn, K, scale, length, span, kpos, qpos if bias else None, slope, cap)
    Oref, lref = oracle.kv4_attention(s, V)
    dist = 0.0 if not bias else float(np.abs(qpos).max() + (N if kpos is None else kpos.max()))
    ds, do = _tol(Qn, K, V, scale, cap, dtype)
    ds += 2.0 ** -22 * dist                   # the bias term's own fp32 rounding
    do += np.expm1(2.0 ** -21 * dist) * np.abs(V).max()
    _check_attn(O.t, lse.t, Oref, lref, ds, do, dtype)
    assert O.intact() and lse.intact()
    # the weight, from the oracle's lse, added to what is there; in place too
    lse32 = torch.from_numpy(lref).float().cuda()
    w0 = torch.rand(B, Hkv, N, device="cuda")
    w = Guarded((B, Hkv, N), F32, fill=7)
    ws = ps.workspace(ps.OP_KV4_WEIGHT, **sizes)
    ps.ps_kv4_weight(c, Q, lse32, None, w.t, ws=ws, **opt)
    ref = oracle.kv4_weight(s, lse32.double().cpu().numpy(), Hkv)
    got = w.t.double().cpu().numpy()
    # each term to the score's and lse's error, sums to 2^-20 (plus terms ex2 flushes to 0)
    lim = ref * (np.expm1(2 * ds + 2.0 ** -21 * np.abs(lref[np.isfinite(lref)]).max(initial=0))
                 + 2.0 ** -18) + 1e-30
    assert np.all(np.abs(got - ref) <= lim), np.max(np.abs(got - ref) / lim)
    assert w.intact()
    w1 = w0.clone()
    ps.ps_kv4_weight(c, Q, lse32, w1, w1, ws=ws, **opt)
    assert torch.equal(w1, w0 + w.t)
    # identical calls give identical bits
    O2, lse2 = torch.zeros_like(O.t), torch.zeros_like(lse.t)
    ps.ps_kv4_attn(c, Q, O2, lse2, ws=ps.workspace(ps.OP_KV4_ATTN, **sizes), **opt)
    assert torch.equal(O2, O.t) and torch.equal(lse2, lse.t)


def _attn(c, Q, **opt):
    B, T, Hq, dh = Q.shape
    O, lse = torch.empty_like(Q, memory_format=torch.contiguous_format), torch.empty(
        B, T, Hq, device="cuda")
    ps.ps_kv4_attn(c, Q, O, lse, ws=ps.workspace(ps.OP_KV4_ATTN, B=B, N=c.N, Hq=Hq, Hkv=c.Hkv,
                                                 dh=dh, P=T), **opt)
    return O, lse


@pytest.mark.parametrize("T", [1, 40, 200])
def test_peaked_and_huge_scores(T):
    """Scores of several hundred, growing along the cache (the running maximum
    moves at every step) and falling along it."""
    B, H, N, dh = 1, 2, 500, 64
    K = np.zeros((B, H, N, dh), np.float32)
    K[..., 0] = np.linspace(-6, 6, N)
    K[0, 1] = K[0, 1, ::-1]
    V = np.random.default_rng(0).standard_normal((B, H, N, dh)).astype(np.float32)
    enc = [*oracle.kv4_encode(K, 1.0), *oracle.kv4_encode(V, 0.5)]
    c = ps.Kv4Cache(*(torch.from_numpy(x).cuda() for x in enc), kmul=1.0, vmul=0.5)
    K, V = oracle.kv4_decode(enc[0], enc[1], 1.0), oracle.kv4_decode(enc[2], enc[3], 0.5)
    Q = torch.zeros(B, T, H, dh)
    Q[..., 0] = torch.linspace(-80, 80, T)[None, :, None] if T > 1 else 80.0
    O, lse = _attn(c, Q.to(BF16).cuda(), scale=1.0)
    s = oracle.kv4_scores(Q.to(BF16).double().numpy(), K, 1.0)
    ds, do = _tol(Q.numpy(), K, V, 1.0, 0, BF16)
    _check_attn(O, lse, *oracle.kv4_attention(s, V), ds, do, BF16)


@pytest.mark.parametrize("T,dtype", [(3, BF16), (3, F32), (140, BF16)])
def test_query_magnitudes(T, dtype):
    """Rows of very different sizes in one tile, down to all zero."""
    c, K, V = _cache(1, 1, 200, 128, 4)
    Q, _ = _query(1, T, 2, 128, F32, 4)
    Q = (Q * torch.logspace(-12, 1, 2 * T, device="cuda").reshape(1, T, 2, 1)).to(dtype)
    Q[0, 1] = 0
    O, lse = _attn(c, Q, scale=0.1)
    Qn = Q.double().cpu().numpy()
    ds, do = _tol(Qn, K, V, 0.1, 0, dtype)
    _check_attn(O, lse, *oracle.kv4_attention(oracle.kv4_scores(Qn, K, 0.1), V), ds, do, dtype)


@pytest.mark.parametrize("T", [4, 150])
def test_nan_query_row_stays_its_own(T):
    c, K, V = _cache(1, 1, 333, 128, 5)
    Q, _ = _query(1, T, 2, 128, BF16, 5)
    bad = Q.clone()
    bad[0, 1, 0, 3] = float("nan")
    bad[0, 2, 1, 5] = float("inf")
    O, lse = _attn(c, Q, scale=0.1)
    Ob, lb = _attn(c, bad, scale=0.1)
    same = torch.ones(T, 2, dtype=torch.bool)
    same[1, 0] = same[2, 1] = False
    assert torch.equal(Ob[0][same], O[0][same]) and torch.equal(lb[0][same], lse[0][same])
    assert torch.isnan(Ob[0, 1, 0]).all() and torch.isnan(lb[0, 1, 0])
    assert torch.isnan(Ob[0, 2, 1]).all()


def test_strided_queries_and_rows():
    """Q, K and V as parts of one projection's output."""
    B, T, Hq, Hkv, dh, N = 2, 37, 4, 2, 128, 64
    g = torch.Generator().manual_seed(6)
    qkv = torch.randn(B, T, (Hq + 2 * Hkv), dh, generator=g).to(BF16).cuda()
    Q, K, V = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    a, b = ps.Kv4Cache.empty(B, Hkv, N, dh), ps.Kv4Cache.empty(B, Hkv, N, dh)
    ps.ps_kv4_store(a, K, V)
    ps.ps_kv4_store(b, K.contiguous(), V.contiguous())
    assert all(torch.equal(x, y) for x, y in zip(a.buffers, b.buffers))
    n = torch.full((B,), T, dtype=torch.int32, device="cuda")
    O, lse = _attn(a, Q, scale=0.1, len=n)
    O2, lse2 = _attn(a, Q.contiguous(), scale=0.1, len=n)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("B,R,Hkv,dh,N,dtype", [(1, 1, 1, 64, 1, BF16), (2, 37, 3, 128, 50, BF16),
                                                (3, 130, 2, 64, 131, F32), (1, 9, 5, 256, 40, BF16),
                                                (2, 64, 4, 128, 64, F32)])
def test_store_and_load_bit_exact(B, R, Hkv, dh, N, dtype):
    rng = np.random.default_rng(R)
    K = torch.from_numpy(rng.standard_normal((B, R, Hkv, dh)).astype(np.float32) * 3).to(dtype)
    V = torch.from_numpy(rng.standard_normal((B, R, Hkv, dh)).astype(np.float32)).to(dtype)
    K[0, 0, 0, :16] = 0
    K[0, 0, 0, 16], K[0, 0, 0, 17], K[0, 0, 0, 18] = float("inf"), float("-inf"), float("nan")
    V[0, 0, 0, :16] = -1e-30                     # scale rounds to 0
    V[0, -1, -1, :16] = torch.arange(16) * 0.25 * 0.3     # ties of E2M1 with S = 0.3
    off = rng.integers(0, N - R + 1, B)
    kmul, vmul = 0.7, 0.3
    bufs = [Guarded((B, Hkv, N, dh // q), torch.uint8, fill=0x3C) for q in (2, 16, 2, 16)]
    c = ps.Kv4Cache(*(g.t for g in bufs), kmul=kmul, vmul=vmul)
    ps.ps_kv4_store(c, K.cuda(), V.cuda(), off=_i32(off))
    want = [np.full(g.t.shape, 0x3C, np.uint8) for g in bufs]
    for i, (X, S) in enumerate(((K, kmul), (V, vmul))):
        code, sc = oracle.kv4_encode(X.float().numpy(), S)
        for b in range(B):
            want[2 * i][b, :, off[b]:off[b] + R] = code[b].transpose(1, 0, 2)
            want[2 * i + 1][b, :, off[b]:off[b] + R] = sc[b].transpose(1, 0, 2)
    for g, x in zip(bufs, want):
        assert np.array_equal(np_(g.t), x) and g.intact()
    for out in (BF16, F32):
        Kb, Vb = (Guarded((B, R, Hkv, dh), out, fill=3) for _ in range(2))
        ps.ps_kv4_load(c, Kb.t, Vb.t, off=_i32(off))
        for got, i, S in ((Kb, 0, kmul), (Vb, 2, vmul)):
            v = oracle.kv4_decode(want[i], want[i + 1], S).astype(np.float32)  # one rounding
            ref = np.stack([v[b, :, off[b]:off[b] + R].transpose(1, 0, 2) for b in range(B)])
            assert torch.equal(got.t.cpu(), torch.from_numpy(ref).to(out)) and got.intact()


def test_store_lists_and_skipped_entries():
    """Listed rows only; entries out of range and past cnt are skipped, offsets
    that leave the cache too."""
    B, R, Hkv, dh, N = 3, 50, 2, 128, 60
    rng = np.random.default_rng(8)
    X = torch.from_numpy(rng.standard_normal((B, R, Hkv, dh)).astype(np.float32)).to(BF16).cuda()
    rows = np.full((B, R), -1)
    rows[0, :6] = [4, 0, 49, 7, -3, 50]
    rows[1, :4] = [1, 2, 3, 4]
    rows[2, :3] = [0, 20, 49]
    cnt, off = np.array([6, 2, 3]), np.array([0, 5, -20])
    c = ps.Kv4Cache.empty(B, Hkv, N, dh)
    full = ps.Kv4Cache.empty(B, Hkv, N, dh)
    ps.ps_kv4_store(c, X, -X, off=_i32(off), rows=_i32(rows), cnt=_i32(cnt))
    ps.ps_kv4_store(full, X, -X)
    hit = {(0, 4): 4, (0, 0): 0, (0, 49): 49, (0, 7): 7, (1, 6): 1, (1, 7): 2, (2, 0): 20, (2, 29): 49}
    for x, y in zip(c.buffers, full.buffers):
        x, y = np_(x), np_(y)
        for b in range(B):
            for n in range(N):
                want = y[b, :, hit[b, n]] if (b, n) in hit else np.zeros_like(x[b, :, n])
                assert np.array_equal(x[b, :, n], want), (b, n)
    K, V = torch.full_like(X, 9), torch.full_like(X, 9)
    ps.ps_kv4_load(c, K, V, off=_i32(off), rows=_i32(rows), cnt=_i32(cnt))
    touched = {(b, r) for (b, _), r in hit.items()}
    for b in range(B):
        for r in range(R):
            assert bool((K[b, r] == 9).all()) != ((b, r) in touched), (b, r)


EVICT = [(1, 1, 64, 5, 3, 0, 0, "rand"), (2, 3, 128, 1500, 700, 4, 32, "rand"),
         (2, 2, 128, 2048, 1024, 0, 0, "ties"), (1, 2, 256, 300, 299, 1, 298, "rand"),
         (3, 1, 128, 700, 650, 10, 20, "nan"), (1, 4, 64, 5000, 17, 17, 0, "rand"),
         (2, 2, 128, 1025, 400, 3, 5, "zero"), (1, 1, 128, 9000, 4096, 4, 64, "neg"),
         (1, 2, 64, 20000, 7000, 4, 100, "ties"), (2, 1, 64, 16384, 16000, 0, 9, "rand")]


@pytest.mark.parametrize("B,Hkv,dh,N,keep,sink,recent,kind", EVICT)
@pytest.mark.parametrize("with_pos", [False, True])
def test_evict(B, Hkv, dh, N, keep, sink, recent, kind, with_pos):
    rng = np.random.default_rng(N + keep)
    w = np.exp(rng.standard_normal((B, Hkv, N)) * 3).astype(np.float32)
    if kind == "ties":
        w = np.round(w)
    elif kind == "nan":
        w[rng.random(w.shape) < 0.3] = np.nan
        w[rng.random(w.shape) < 0.1] = np.inf
        w[rng.random(w.shape) < 0.1] = -np.inf
    elif kind == "zero":
        w[:] = 0
    elif kind == "neg":
        w = rng.standard_normal(w.shape).astype(np.float32)
        w[..., ::7] = -0.0
        w[..., 1::7] = 0.0
    length = rng.integers(0, N + 1, B)
    length[0] = N
    kpos = rng.integers(0, 10 * N, (B, Hkv, N)) if with_pos else None
    src = ps.Kv4Cache(*(torch.from_numpy(rng.integers(0, 256, (B, Hkv, N, dh // q), dtype=np.uint8))
                        .cuda() for q in (2, 16, 2, 16)))
    M = keep + 3
    bufs = [Guarded((B, Hkv, M, dh // q), torch.uint8, fill=0x3C) for q in (2, 16, 2, 16)]
    dst = ps.Kv4Cache(*(g.t for g in bufs))
    wd, kd, ld = Guarded((B, Hkv, M), F32, fill=5), Guarded((B, Hkv, M), torch.int32, fill=-9), \
        Guarded((B,), torch.int32)
    ps.ps_kv4_evict(src, dst, torch.from_numpy(w).cuda(), wd.t, ld.t, keep, sink=sink,
                    recent=recent, len=_i32(length), kpos=_i32(kpos), kpos_dst=kd.t,
                    ws=ps.workspace(ps.OP_KV4_EVICT, B=B, N=N, Hkv=Hkv, k=keep))
    assert list(np_(ld.t)) == [min(int(n), keep) for n in length]
    for b in range(B):
        for h in range(Hkv):
            at = oracle.kv4_keep(w[b, h], int(length[b]), keep, sink, recent)
            k = len(at)
            for x, g in zip(src.buffers, bufs):
                assert np.array_equal(np_(g.t)[b, h, :k], np_(x)[b, h, at])
                assert np.all(np_(g.t)[b, h, k:] == 0x3C)
            assert np.array_equal(np_(wd.t)[b, h, :k], w[b, h, at], equal_nan=True)
            assert np.all(np_(wd.t)[b, h, k:] == 5)
            assert np.array_equal(np_(kd.t)[b, h, :k], kpos[b, h, at] if with_pos else at)
            assert np.all(np_(kd.t)[b, h, k:] == -9)
    assert all(g.intact() for g in (*bufs, wd, kd, ld))


def test_offsets_past_32_bits():
    """The last slots of a cache whose code arrays pass 2^31 bytes."""
    B, Hkv, dh = 1, 2, 64
    N = (1 << 31) // (Hkv * dh // 2) + 1000
    c = ps.Kv4Cache.empty(B, Hkv, N, dh)
    K = torch.randn(1, 100, Hkv, dh, device="cuda").to(BF16)
    ps.ps_kv4_store(c, K, -K, off=_i32([N - 100]))
    Kb, Vb = torch.zeros_like(K), torch.zeros_like(K)
    ps.ps_kv4_load(c, Kb, Vb, off=_i32([N - 100]))
    assert torch.equal(Kb, -Vb) and float((Kb.float() - K.float()).abs().max()) < 1.0
    K64 = Kb.double().cpu().numpy().transpose(0, 2, 1, 3)
    for T in (1, 80):
        Q, Qn = _query(1, T, 4, dh, BF16, 9)
        O, lse = _attn(c, Q, scale=0.125, span=_i32(np.tile([N - 100, N + 5], (1, T, 1))))
        ds, do = _tol(Qn, K64, K64, 0.125, 0, BF16)
        _check_attn(O, lse, *oracle.kv4_attention(oracle.kv4_scores(Qn, K64, 0.125), -K64), ds, do,
                    BF16)


def test_runs_on_the_given_stream():
    c, _, _ = _cache(1, 2, 300, 128, 10)
    Q, _ = _query(1, 3, 4, 128, BF16, 10)
    want, lw = _attn(c, Q, scale=0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    O, lse = _attn(c, Q, scale=0.1, stream=s)
    s.synchronize()
    assert torch.equal(O, want) and torch.equal(lse, lw)


def test_empty_calls():
    c, _, _ = _cache(1, 2, 30, 128, 11)
    z = torch.zeros(1, 0, 4, 128, dtype=BF16, device="cuda")
    ps.ps_kv4_attn(c, z, z, scale=1.0)
    zk = torch.zeros(1, 0, 2, 128, dtype=BF16, device="cuda")
    ps.ps_kv4_store(c, zk, zk)
    e = ps.Kv4Cache.empty(0, 2, 30, 128)
    z = torch.zeros(0, 3, 4, 128, dtype=BF16, device="cuda")
    ps.ps_kv4_attn(e, z, z, scale=1.0)


def test_refusals():
    c, _, _ = _cache(1, 2, 30, 128, 12)
    Q, _ = _query(1, 3, 4, 128, BF16, 12)
    O, lse = torch.zeros_like(Q), torch.zeros(1, 3, 4, device="cuda")

    def arg(fn):
        with pytest.raises(ps.PolestarError) as e:
            fn()
        assert e.value.status == ps.PS_ERR_ARG

    ws = ps.workspace(ps.OP_KV4_ATTN, B=1, N=30, Hq=4, Hkv=2, dh=128, P=3)
    arg(lambda: ps.ps_kv4_attn(c, Q, O, lse, scale=float("nan"), ws=ws))
    arg(lambda: ps.ps_kv4_attn(c, Q, O, lse, scale=1.0, cap=-1.0, ws=ws))
    arg(lambda: ps.ps_kv4_attn(c, Q[:, :, :3], O[:, :, :3].contiguous(), scale=1.0, ws=ws))  # 3 of 2
    arg(lambda: ps.ps_kv4_attn(c, Q, O, lse, scale=1.0, slope=torch.ones(4, device="cuda"), ws=ws))
    big = ps.Kv4Cache.empty(1, 2, 8192, 128)
    with pytest.raises(ps.PolestarError) as e:
        ps.ps_kv4_attn(big, Q, O, lse, scale=1.0)
    assert e.value.status == ps.PS_ERR_WORKSPACE
    bad = ps.Kv4Cache(*c.buffers, kmul=0.0)
    arg(lambda: ps.ps_kv4_attn(bad, Q, O, lse, scale=1.0, ws=ws))
    odd = ps.Kv4Cache.empty(1, 2, 30, 96)
    q96 = torch.zeros(1, 3, 4, 96, dtype=BF16, device="cuda")
    arg(lambda: ps.ps_kv4_attn(odd, q96, q96.clone(), scale=1.0))
    d = ps.Kv4Cache.empty(1, 2, 10, 128)
    w, wd = torch.zeros(1, 2, 30, device="cuda"), torch.zeros(1, 2, 10, device="cuda")
    ld = torch.zeros(1, dtype=torch.int32, device="cuda")
    ews = ps.workspace(ps.OP_KV4_EVICT, B=1, N=30, Hkv=2, k=30)
    arg(lambda: ps.ps_kv4_evict(c, d, w, wd, ld, 11, ws=ews))                 # dst too short
    arg(lambda: ps.ps_kv4_evict(c, d, w, wd, ld, 5, sink=3, recent=3, ws=ews))
    arg(lambda: ps.ps_kv4_evict(c, d, w, wd, ld, 0, ws=ews))                  # other tensor scales too
    same = ps.Kv4Cache(*d.buffers, kmul=c.kmul, vmul=c.vmul)
    with pytest.raises(ps.PolestarError) as e:
        ps.ps_kv4_evict(c, same, w, wd, ld, 5)
    assert e.value.status == ps.PS_ERR_WORKSPACE
    for bad_call in (lambda: ps.ps_kv4_attn(c, Q.transpose(1, 2), O, scale=1.0, ws=ws),
                     lambda: ps.ps_kv4_attn(c, Q, O.float(), scale=1.0, ws=ws),
                     lambda: ps.ps_kv4_attn(c, Q, O, lse, scale=1.0, ws=ws,
                                            len=torch.ones(1, dtype=torch.int64, device="cuda")),
                     lambda: ps.ps_kv4_store(c, Q[:, :, :2], O[:, :, 2:].contiguous()),
                     lambda: ps.Kv4Cache(*c.buffers[:3], c.buffers[3][..., :4])):
        with pytest.raises(ValueError):
            bad_call()
    lib = ps.Library.load()
    assert lib.cdll.ps_kv4_attn(None, c._c, None, None, None, None, 0, None) == ps.PS_ERR_ARG
    assert lib.cdll.ps_kv4_store(lib.handle(), None, None, None, 0, 1, 256, 256, None, None, None,
                                 None) == ps.PS_ERR_ARG
    q = ps._kv4_query(c, Q, None, None, None, None, None, 1.0, 0.0)[2]
    off4 = ctypes.c_void_p(O.data_ptr() + 4)
    assert lib.cdll.ps_kv4_attn(lib.handle(), c._c, q, off4, None, ws.data_ptr() if ws is not None
                                else None, 1 << 20, None) == ps.PS_ERR_ARG
    assert torch.all(O == 0)


def test_graph_capture():
    """The calls capture into a CUDA graph and replay with the same bits."""
    c, _, _ = _cache(2, 2, 900, 128, 13)
    Q, _ = _query(2, 3, 8, 128, BF16, 13)
    O, lse = torch.zeros_like(Q), torch.zeros(2, 3, 8, device="cuda")
    w = torch.zeros(2, 2, 900, device="cuda")
    sizes = dict(B=2, N=900, Hq=8, Hkv=2, dh=128, P=3)
    ws, ww = ps.workspace(ps.OP_KV4_ATTN, **sizes), ps.workspace(ps.OP_KV4_WEIGHT, **sizes)

    def step():
        ps.ps_kv4_attn(c, Q, O, lse, scale=0.1, ws=ws)
        ps.ps_kv4_weight(c, Q, lse, None, w, scale=0.1, ws=ww)

    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (O, lse, w)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in (O, lse, w):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((O, lse, w), want))


@pytest.mark.parametrize("B,T,Hq,Hkv,dh,N,mask,cap,bias", [
    (1, 65, 1, 1, 128, 1, "none", 0, False),
    (1, 128, 3, 3, 64, 256, "none", 0, False),
    (2, 129, 2, 1, 128, 257, "len", 0, False),
    (1, 1500, 2, 2, 64, 700, "causal", 0, False),
    (1, 2049, 1, 1, 128, 300, "none", 0, False),
    (3, 401, 7, 1, 128, 1025, "documents", 0, False),
    (1, 333, 4, 2, 64, 5000, "documents", 0.75, True),
    (2, 200, 4, 4, 128, 511, "causal", 40.0, False),
    (1, 500, 4, 2, 128, 600, "kpos", 10.0, True),
])
def test_weight_of_many_rows(B, T, Hq, Hkv, dh, N, mask, cap, bias):
    """Rows and slots that end inside tiles, rows split over CTAs, steps that see
    nothing; the sum over all rows of a head is as good as its terms."""
    seed = T + N
    length, span, qpos, kpos = _masks(mask, B, T, N, Hkv, seed)
    c, K, V = _cache(B, Hkv, N, dh, seed, junk_from=length)
    Q, Qn = _query(B, T, Hq, dh, BF16, seed, 1.0)
    scale = dh ** -0.5
    slope = (0.5 ** np.arange(1, Hq + 1)).astype(np.float32) if bias else None
    s = oracle.kv4_scores(Qn, K, scale, length, span, kpos, qpos if bias else None, slope, cap)
    _, lref = oracle.kv4_attention(s, V)
    lse = torch.from_numpy(lref).float().cuda()
    opt = dict(scale=scale, len=_i32(length), span=_i32(span), kpos=_i32(kpos),
               qpos=_i32(qpos) if bias else None,
               slope=torch.from_numpy(slope).cuda() if bias else None, cap=float(cap))
    w = Guarded((B, Hkv, N), F32, fill=7)
    w0 = torch.rand(B, Hkv, N, device="cuda")
    ps.ps_kv4_weight(c, Q, lse, None, w.t, **opt)
    ref = oracle.kv4_weight(s, lse.double().cpu().numpy(), Hkv)
    dist = 0.0 if not bias else float(np.abs(qpos).max() + (N if kpos is None else kpos.max()))
    ds, _ = _tol(Qn, K, V, scale, cap, BF16)
    ds += 2.0 ** -22 * dist
    lim = ref * (np.expm1(2 * ds + 2.0 ** -21 * np.abs(lref[np.isfinite(lref)]).max(initial=0))
                 + 2.0 ** -18) + 1e-30
    got = w.t.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= lim), np.max(np.abs(got - ref) / lim)
    assert w.intact()
    w1 = w0.clone()
    ps.ps_kv4_weight(c, Q, lse, w1, w1, **opt)
    assert torch.equal(w1, w0 + w.t)


@pytest.mark.parametrize("T,dh,N,mask,cap", [(150, 128, 700, "none", 30.0), (40, 64, 1100, "len", 0.5),
                                             (300, 128, 513, "causal", 3.0),
                                             (77, 64, 640, "documents", 50.0)])
def test_capped_scores_of_many_rows(T, dh, N, mask, cap):
    """Capped scores without a bias: small ones, and ones at the cap."""
    test_attention_and_weight(2, T, 6, 2, dh, N, BF16, mask, cap, False)


@pytest.mark.parametrize("T", [1, 20, 90])
def test_queries_of_part_of_a_sequence(T):
    """Q as some tokens of a longer [B][T'][Hq][dh]: a stride between sequences."""
    B, Hq, Hkv, dh, N = 3, 4, 2, 64, 300
    c, _, _ = _cache(B, Hkv, N, dh, 8)
    Q, _ = _query(B, T + 9, Hq, dh, BF16, 8)
    part = Q[:, 5:5 + T]
    O, lse = _attn(c, part, scale=0.125)
    O2, lse2 = _attn(c, part.contiguous(), scale=0.125)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    w, w2 = torch.zeros(B, Hkv, N, device="cuda"), torch.zeros(B, Hkv, N, device="cuda")
    ps.ps_kv4_weight(c, part, lse, None, w, scale=0.125)
    ps.ps_kv4_weight(c, part.contiguous(), lse, None, w2, scale=0.125)
    assert torch.equal(w, w2)
