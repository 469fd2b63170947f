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


CAPS = [1e-30, 1e-3, 0.5, 50.0, 64.0, 65.0, 1e4, 1e6, 1e9, 1e20, 3e38]


@pytest.mark.parametrize("T", [1, 12, 40, 150])
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("bias", [False, True])
def test_caps_of_any_size(T, cap, bias):
    """Scores within a dozen under caps from far below to far above them, rows near
    a cap of 1e4 among them: every row's lse is as good as its own scores, its
    weights sum to 1, and attention and weight agree.

    A row's scores: products as _tol; score / cap, its tanh and the product with
    the cap to 2^-20 of the score, or up to a cap of 64 to 2^-21.5 of that, which is
    less where the score is past a third of it."""
    B, Hq, Hkv, dh, N = 1, 4, 2, 64, 333
    scale = dh ** -0.5
    c, K, V = _cache(B, Hkv, N, dh, 17)
    Q, _ = _query(B, T, Hq, dh, BF16, T, 1.5)
    if T > 1:
        Q[0, 1] *= 2000.0            # products up to some 1e4 beside rows of a dozen
    Qn = Q.double().cpu().numpy()
    opt = dict(cap=float(cap))
    qpos = slope = None
    if bias:
        qpos, slope = np.full((B, T), N // 2), np.full(Hq, 2.0 ** -6, np.float32)
        opt.update(qpos=_i32(qpos), slope=torch.from_numpy(slope).cuda())
    s = oracle.kv4_scores(Qn, K, scale, cap=float(np.float32(cap)), qpos=qpos, slope=slope)
    Oref, lref = oracle.kv4_attention(s, V)
    O, lse = _attn(c, Q, scale=scale, **opt)
    Kg = np.repeat(np.abs(K), Hq // Hkv, 1)
    sabs = scale * np.einsum("bthd,bhnd->bthn", np.abs(Qn), Kg).max(-1)
    top = np.minimum(sabs, cap)
    capped = 2.0 ** -20 * top + (2.0 ** -21.5 * cap if cap <= 64 else 0.0)
    # the cap's slope is at most 1: products' errors do not grow, and nothing passes it
    ds = np.minimum(2.0 ** -22 * sabs * (dh / 16 + 2), 2 * top) + capped + 2.0 ** -21 * (top + 1)
    if bias:
        ds = ds + 2.0 ** -21 * (N / 2 * 2.0 ** -6 + top)
    lim = 2 * ds + 2.0 ** -20 * (1 + np.abs(lref))
    err = np.abs(np_(lse).astype(np.float64) - lref)
    assert np.all(err <= lim), (err / lim).max()
    # P to 2^-11, then bf16's half step
    do = (np.expm1(2 * ds) + 2.0 ** -11 + 2.0 ** -19)[..., None] * np.abs(V).max()
    assert np.all(np.abs(np_(O).astype(np.float64) - Oref) <= do + 2.0 ** -8 * np.abs(Oref))
    # the weight from the attention's own lse: every row's sums to 1
    row = np.expm1(3 * ds + lim + 2.0 ** -21 * np.abs(lref)) + 2.0 ** -18
    w = np_(_weight(c, Q, lse, scale=scale, **opt)).astype(np.float64)
    per = row.reshape(B, T, Hkv, Hq // Hkv).sum((1, 3))
    assert np.all(np.abs(w.sum(-1) - T * Hq // Hkv) <= per), (w.sum(-1), per)


@pytest.mark.parametrize("T", [1, 150])
@pytest.mark.parametrize("cap", [0.0, 30.0, 1e6])
def test_a_nan_query_stays_nan_under_a_cap(T, cap):
    c, _, _ = _cache(1, 1, 256, 128, 5)
    Q, _ = _query(1, T, 2, 128, BF16, 5, 4000.0 if cap == 1e6 else 30.0)
    want, lw = _attn(c, Q, scale=1.0, cap=cap)
    Q[0, 0, 1, 3] = float("nan")
    O, lse = _attn(c, Q, scale=1.0, cap=cap)
    assert torch.isnan(O[0, 0, 1]).all() and torch.isnan(lse[0, 0, 1])
    assert torch.equal(O[0, 0, 0], want[0, 0, 0]) and torch.equal(O[0, 1:], want[0, 1:])
    assert torch.isfinite(want.float()).all() and torch.isfinite(lw).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_rows_than_2_to_the_24(dtype):
    """The first and the last tokens of a call with more than 2^24 rows a KV head get
    what a call of their own gets, output, lse and weight."""
    T, tail, N, dh = (1 << 24) + 300, 400, 16, 64
    c, _, _ = _cache(1, 1, N, dh, 21)
    g = torch.Generator(device="cuda").manual_seed(1)
    Q = torch.randn(1, T, 1, dh, generator=g, device="cuda", dtype=dtype)
    O, lse = _attn(c, Q, scale=0.125)
    Ot, lt = _attn(c, Q[:, -tail:].contiguous(), scale=0.125)
    assert torch.equal(O[:, -tail:], Ot) and torch.equal(lse[:, -tail:], lt)
    Oh, lh = _attn(c, Q[:, :tail].contiguous(), scale=0.125)
    assert torch.equal(O[:, :tail], Oh) and torch.equal(lse[:, :tail], lh)
    if dtype == BF16:   # every row's weights sum to 1, each to 2^-18, added with compensation
        w = _weight(c, Q, lse, scale=0.125)
        assert abs(float(w.double().sum()) - T) <= T * 2.0 ** -18
    # a span that the last rows alone have: what they weigh is theirs
    span = torch.zeros(1, T, 2, dtype=torch.int32, device="cuda")
    span[:, -tail:, 1] = N
    wt = _weight(c, Q[:, -tail:].contiguous(), lt, scale=0.125)
    ws = _weight(c, Q, lse, scale=0.125, span=span)
    assert torch.allclose(ws, wt, rtol=2.0 ** -18, atol=0)


@pytest.mark.parametrize("dh", [128, 256])
def test_lists_of_more_entries_than_2_to_the_24(dh):
    """Entries at both ends of a list of more than 2^24 warps' entries; all others
    name no row."""
    R, n = (1 << 24) * (512 // dh) + 40, 30
    X = torch.randn(n, dh, device="cuda").to(BF16)
    rows = torch.full((1, R), -1, dtype=torch.int32, device="cuda")
    rows[0, :n // 2] = torch.arange(n // 2)
    rows[0, -(n - n // 2):] = torch.arange(n // 2, n)
    c, want = ps.Kv4Cache.empty(1, 1, n, dh), ps.Kv4Cache.empty(1, 1, n, dh)
    ps.ps_kv4_store(want, X.view(1, n, 1, dh), -X.view(1, n, 1, dh))
    lib = ps.Library.load()
    Y = -X
    st = lib.cdll.ps_kv4_store(lib.handle(0), c._c, X.data_ptr(), Y.data_ptr(), ps.PS_BF16, R, 0,
                               dh, None, rows.data_ptr(), None,
                               torch.cuda.current_stream().cuda_stream)
    assert st == ps.PS_OK
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(c.buffers, want.buffers))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mul", [1.0, 0.7, 2.0 ** -60, 1e-37, 2.0 ** -126])
def test_store_keeps_signs(dtype, mul):
    """Zeros of both signs in live blocks, values whose code is a zero, quotients far
    past 6 and past fp32 (a block scale that saturates under a small tensor scale),
    NaN of both signs: bits as the oracle's divisions give them."""
    R, dh = 64, 64
    rng = np.random.default_rng(7)
    X = (rng.standard_normal((1, R, 1, dh)) * np.float64(mul) * 100).astype(np.float32)
    X[0, 0, 0, ::3], X[0, 0, 0, 1::3] = -0.0, 0.0
    X[0, 1, 0, :] = -0.0                                  # a block of nothing else: scale 0
    X[0, 2, 0, ::2] *= 1e-4                               # small ones, to zeros of their sign
    X[0, 3, 0, ::2] = -0.0
    for r, big in ((4, 1e30), (5, 3e38), (6, 1e38)):      # saturated scales
        X[0, r, 0, :] = np.where(rng.random(dh) < 0.5, -1, 1) * big
        X[0, r, 0, ::5] = -0.0
        X[0, r, 0, 1::5] = -np.float32(mul)
    X[0, 7, 0, ::4], X[0, 7, 0, 1::4] = np.float32("nan"), -np.float32("nan")
    X[0, 8, 0, ::4], X[0, 8, 0, 1::4] = -np.inf, np.inf
    X[0, 9, 0, :] = np.where(rng.random(dh) < 0.5, -1, 1) * np.float32(1e-45)
    X[0, 9, 0, 0] = np.float32(mul) * 448 * 6
    K = torch.from_numpy(X).to(dtype)
    c = ps.Kv4Cache.empty(1, 1, R, dh, mul, mul)
    ps.ps_kv4_store(c, K.cuda(), -K.cuda())
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        for x, at in ((K, 0), (-K, 2)):
            code, scale = oracle.kv4_encode(x.float().numpy().transpose(0, 2, 1, 3), mul)
            assert np.array_equal(np_(c.buffers[at + 1]), scale)
            bad = np.argwhere(np_(c.buffers[at]) != code)
            assert bad.size == 0, (bad[:8], dtype, mul)


def _against_oracle(c, K, V, Q, dtype, scale, dist=0.0, **opt):
    """Attention, and the weight from the oracle's lse, against the oracle; `dist`:
    the largest distance bias."""
    Qn = Q.double().cpu().numpy()
    s = oracle.kv4_scores(Qn, K, scale, opt.get("len"), opt.get("span"), opt.get("kpos"),
                          opt.get("qpos"), opt.get("slope"))
    Oref, lref = oracle.kv4_attention(s, V)
    dev = {k: torch.from_numpy(v).cuda() if k == "slope" else _i32(v) for k, v in opt.items()}
    O, lse = _attn(c, Q, scale=scale, **dev)
    ds, do = _tol(Qn, K, V, scale, 0, dtype)
    ds, do = ds + 2.0 ** -22 * dist, do + np.expm1(2.0 ** -21 * dist) * np.abs(V).max()
    _check_attn(O, lse, Oref, lref, ds, do, dtype)
    lse32 = torch.from_numpy(lref).float().cuda()
    w = np_(_weight(c, Q, lse32, scale=scale, **dev)).astype(np.float64)
    ref = oracle.kv4_weight(s, lse32.double().cpu().numpy(), c.Hkv)
    big = np.abs(lref[np.isfinite(lref)]).max(initial=0)
    lim = ref * (np.expm1(2 * ds + 2.0 ** -21 * big) + 2.0 ** -18) + 1e-30
    assert np.all(np.abs(w - ref) <= lim), np.max(np.abs(w - ref) / lim)


@pytest.mark.parametrize("T", [1, 12, 40, 150])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bias", [False, True])
def test_any_position_is_seen_without_a_span(T, dtype, bias):
    """Positions below 0 and at the end of their type, as an offset or a mark may
    leave them: without a span a row sees every filled slot."""
    B, Hq, Hkv, dh, N = 2, 4, 2, 64, 203
    rng = np.random.default_rng(T)
    c, K, V = _cache(B, Hkv, N, dh, T)
    Q, _ = _query(B, T, Hq, dh, dtype, T)
    opt = dict(len=np.array([N, 150]))
    if bias:
        opt.update(kpos=rng.integers(-300, 300, (B, Hkv, N)), qpos=rng.integers(-9, 9, (B, T)),
                   slope=np.array([0.25, 0.125, 0.0625, 0.03125], np.float32))
    else:
        opt["kpos"] = rng.choice([-(1 << 31), -1, 0, 7, (1 << 31) - 1], (B, Hkv, N))
    _against_oracle(c, K, V, Q, dtype, 0.125, 310 * 0.25 if bias else 0.0, **opt)


LOWEST, HIGHEST = -(1 << 31), (1 << 31) - 1


@pytest.mark.parametrize("T", [1, 12, 40, 150, 290])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["open", "mixed", "below"])
@pytest.mark.parametrize("with_pos", [False, True])
def test_spans_that_are_open_at_their_ends(T, dtype, kind, with_pos):
    """Bounds at the ends of their type: no lower bound, no upper one, neither, spans
    that end before the first slot, in one tile with ordinary ones."""
    B, Hq, Hkv, dh, N = 2, 2, 1, 64, 330
    rng = np.random.default_rng(T)
    c, K, V = _cache(B, Hkv, N, dh, T)
    Q, _ = _query(B, T, Hq, dh, dtype, T)
    span = np.empty((B, T, 2), np.int64)
    if kind == "open":
        span[..., 0], span[..., 1] = LOWEST, HIGHEST
    elif kind == "mixed":
        span[..., 0] = rng.choice([LOWEST, LOWEST + 1, -3, 0, 100], (B, T))
        span[..., 1] = rng.choice([HIGHEST, 64, 200, N, LOWEST + 5], (B, T))
    else:
        span[..., 0], span[..., 1] = LOWEST, rng.choice([LOWEST + 5, -64, -1, 0], (B, T))
        span[:, ::3] = [50, 250]
    opt = dict(len=np.array([N, 300]), span=span)
    if with_pos:
        opt["kpos"] = rng.integers(-100, 400, (B, Hkv, N))
    _against_oracle(c, K, V, Q, dtype, 0.125, **opt)


def test_sizes_that_leave_their_type_are_refused():
    """Counts whose products leave an int, and slots up to the largest one: an
    error, and nothing launched."""
    lib = ps.Library.load()
    c, _, _ = _cache(1, 1, 30, 64, 3)
    Q, _ = _query(1, 3, 1, 64, BF16, 3)
    O, lse = torch.full_like(Q, 7), torch.full((1, 3, 1), 7.0, device="cuda")
    w = torch.full((1, 1, 30), 7.0, device="cuda")
    ptr = [t.data_ptr() for t in c.buffers]

    def calls(B, N, T, Hq):
        cc = ps.Kv4Cache._pack.pack(*ptr, B, 1, N, 64, 1.0, 1.0)
        q = ps._Q_PACK.pack(Q.data_ptr(), 0, 0, 0, 0, 0, 64 * Hq, 64 * Hq, ps.PS_BF16, T, Hq,
                            1.0, 0.0)
        return (lib.cdll.ps_kv4_attn(lib.handle(0), cc, q, O.data_ptr(), lse.data_ptr(), None, 0,
                                     None),
                lib.cdll.ps_kv4_weight(lib.handle(0), cc, q, lse.data_ptr(), None, w.data_ptr(),
                                       None, 0, None))

    most = (1 << 31) - 1
    for sizes in ((1, most, 3, 1), (1, 30, most, 1), (1, 30, 1 << 30, 4), (1, 30, most, 4096),
                  (1, 30, most, most)):
        assert calls(*sizes) == (ps.PS_ERR_ARG, ps.PS_ERR_ARG), sizes
    torch.cuda.synchronize()
    assert bool((O == 7).all()) and bool((w == 7).all())


def test_reading_back_into_rows_shared_by_sequences_is_refused():
    c, _, _ = _cache(2, 1, 30, 64, 4)
    one = [torch.full((1, 30, 1, 64), 7.0, device="cuda") for _ in range(2)]
    shared = [x.expand(2, -1, -1, -1) for x in one]
    with pytest.raises(ps.PolestarError) as e:
        ps.ps_kv4_load(c, *shared)
    assert e.value.status == ps.PS_ERR_ARG and all(bool((x == 7).all()) for x in one)
    ps.ps_kv4_store(c, *shared)      # as inputs they may
    out = [torch.zeros(2, 30, 1, 64, device="cuda") for _ in range(2)]
    ps.ps_kv4_load(c, *out)
    assert all(torch.equal(x[0], x[1]) for x in out)


@pytest.mark.parametrize("T", [1, 20, 40, 150])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("how", ["", "bias", "cap", "negative"])
def test_scores_of_any_magnitude(T, dtype, how):
    """Finite queries give finite rows however large the scores, up to where fp32
    scores lie 2^70 apart: each row a mean of the values it sees, the value itself
    where one score is clear of the others by more than the products' rounding."""
    B, H, N, dh, scale = 1, 2, 700, 64, 0.125
    c, K, V = _cache(B, H, N, dh, 31)
    for mag in (1e5, 1e6, 1e7, 1e8, 1e9, 1e12, 1e30):
        Q, _ = _query(B, T, H, dh, dtype, 31)
        Q = Q * mag
        opt = {}
        if how == "bias":
            opt = dict(qpos=_i32(np.full((B, T), N // 2)), slope=torch.full((H,), 2.0 ** -7,
                                                                          device="cuda"))
        elif how == "cap":
            opt = dict(cap=mag)
        O, lse = _attn(c, Q, scale=-scale if how == "negative" else scale, **opt)
        Qn = Q.double().cpu().numpy()
        s = oracle.kv4_scores(Qn, K, -scale if how == "negative" else scale,
                              cap=float(np.float32(mag)) if how == "cap" else 0.0)
        sabs = scale * np.einsum("bthd,bhnd->bthn", np.abs(Qn), np.abs(K)).max(-1)
        top = np.sort(s, -1)[..., -2:]
        assert torch.isfinite(O.float()).all() and torch.isfinite(lse).all(), mag
        # a score to 2^-19 of the sum of its terms' sizes, twice; 60: e^-60 and a bias
        clear = top[..., 1] - top[..., 0] > 2.0 ** -17 * sabs + 60
        On = np_(O).astype(np.float64)
        assert np.abs(On).max() <= np.abs(V).max() * (1 + 2.0 ** -7)
        at = s.argmax(-1)                                    # [B][T][H]
        want = np.stack([[V[b, np.arange(H), at[b, t]] for t in range(T)] for b in range(B)])
        assert np.all(np.abs(On - want)[clear] <= 2.0 ** -8 * np.abs(want)[clear] + 1e-6), mag
        err = np.abs(np_(lse).astype(np.float64) - top[..., 1])
        assert np.all(err <= 2.0 ** -18 * sabs + 8 + N * 2.0 ** -8), (mag, err.max())
