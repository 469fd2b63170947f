"""Kv4Layer and the pipeline around an eviction, on the GPU: what a refresh, a
captured step and further tokens do to a cut cache, and layers on streams of their
own."""
import numpy as np
import pytest
import torch

import oracle
from drift_aware_kv_spherical_gb300 import polestar as ps
from drift_aware_kv_spherical_gb300 import workloads as wl
from drift_aware_kv_spherical_gb300.kv4 import Kv4Layer
from drift_aware_kv_spherical_gb300.pipeline import Pipeline
from tests._parity import Guarded, np_

pytestmark = pytest.mark.gpu

W = wl.Workload("kv4_cut", 92, B=2, N=160, d=256, Hq=4, Hkv=2, dh=64, C=8, iters=3, k=2, P=16,
                V=1024, dtype="bf16", planted=8, noise=1.0, drift_frac=0.1, drift_std=0.5,
                blk_start=64, logit_std=2.0, wq_std=0.05)
FIRST = ps.SCHED_REFRESH | ps.SCHED_FULL | ps.SCHED_REINIT


@pytest.fixture(autouse=True)
def _lib(lib):
    yield lib
    torch.cuda.synchronize()
    ps.ps_check()


def _holds_its_positions(layer, st, kmul, vmul):
    """Every filled slot is the encoding of the bf16 cache's row at its position."""
    n, kpos = layer.len.tolist(), np_(layer.kpos)
    for i, (X, S) in enumerate(((st.Kc, kmul), (st.Vc, vmul))):
        enc = oracle.kv4_encode(np_(X).transpose(0, 2, 1, 3), S)
        for got, want in zip(layer.cache.buffers[2 * i:2 * i + 2], enc):
            for b in range(W.B):
                for h in range(W.Hkv):
                    at = kpos[b, h, :n[b]]
                    assert np.array_equal(np_(got)[b, h, :n[b]], want[b, h, at])


def _cut(pipe, keep, seed):
    layer = pipe.kv4[0]
    layer.w.copy_(torch.rand(layer.w.shape, generator=torch.Generator().manual_seed(seed)))
    layer.evict(keep, sink=2, recent=5)


@pytest.mark.parametrize("graphs", [False, True])
def test_refreshes_after_an_eviction(graphs):
    """The kept slots follow the refreshed rows of their own positions, through
    captured steps too, whose graphs from before an eviction are not replayed."""
    L = wl.make_layer(W, 0, "cuda")
    u, logits = wl.make_uniforms(W, 0, "cuda"), wl.make_logits(W, 0, "cuda")
    pipe = Pipeline(W, layers=1, kv4=True, kmul=0.25, vmul=0.125)
    H = L["H"]
    for t in range(8):
        H = H if t == 0 else wl.drift_rows(W, H, t)
        Q = wl.make_queries(W, H, L["Wq"])
        act = FIRST if t == 0 else ps.SCHED_REFRESH | (ps.SCHED_FULL if t == 5 else 0)
        step = pipe.graph_step if graphs and t > 0 else pipe.decode_step
        idle = None if pipe.kv4[0]._spare is None else \
            [x.clone() for x in pipe.kv4[0]._spare["cache"].buffers]
        step(act, [H], [Q], [L["Wk"]], [L["Wv"]], logits, [u])
        if idle is not None:
            now = pipe.kv4[0]._spare["cache"].buffers
            assert all(torch.equal(x, y) for x, y in zip(idle, now)), t
            _holds_its_positions(pipe.kv4[0], pipe.state[0], 0.25, 0.125)
        if t in (2, 3, 6):
            _cut(pipe, {2: 100, 3: 90, 6: 40}[t], t)


def test_tokens_appended_to_a_cut_cache_are_attended():
    """Append, evict, append: attention and weight over the cut cache with its
    positions follow the oracle on the rows that are left."""
    B, N, Hq, Hkv, dh = 2, 64, 4, 2, 64
    g = torch.Generator().manual_seed(5)
    K, V = (torch.randn(B, 80, Hkv, dh, generator=g).bfloat16().cuda() for _ in range(2))
    kv = Kv4Layer(B, N, Hq, Hkv, dh, 0.25, 0.25)
    kv.append(K[:, :50], V[:, :50])
    Q = torch.randn(B, 3, Hq, dh, generator=g).bfloat16().cuda()
    O, lse = torch.zeros_like(Q), torch.zeros(B, 3, Hq, device="cuda")
    kv.attend(Q, O, lse)
    kv.weigh(Q, lse)
    kv.evict(30, sink=2, recent=4)
    kv.append(K[:, 50:70], V[:, 50:70])
    assert kv.len.tolist() == [50, 50]
    kpos = np_(kv.kpos)[:, :, :50]
    assert np.array_equal(kpos[:, :, 30:], np.broadcast_to(np.arange(50, 70), (B, Hkv, 20)))
    full = [oracle.kv4_decode(*oracle.kv4_encode(np_(X).transpose(0, 2, 1, 3), 0.25), 0.25)
            for X in (K, V)]
    K64, V64 = (np.take_along_axis(X, kpos[..., None], 2) for X in full)
    qpos = np.array([[69, 60, 55]] * B)
    span = np.stack([np.zeros_like(qpos), qpos + 1], -1)
    slope = np.array([0.5, 0.25, 0.125, 0.0625], np.float32)
    see = dict(span=torch.from_numpy(span.astype(np.int32)).cuda(),
               qpos=torch.from_numpy(qpos.astype(np.int32)).cuda(),
               slope=torch.from_numpy(slope).cuda())
    s = oracle.kv4_scores(Q.double().cpu().numpy(), K64, dh ** -0.5, span=span, kpos=kpos,
                          qpos=qpos, slope=slope)
    Oref, lref = oracle.kv4_attention(s, V64)
    w0 = np_(kv.w)
    kv.attend(Q, O, lse, **see)
    kv.weigh(Q, lse, **see)
    # bf16's half step, P's 11 bits; weights to 2^-14 (scores and lse in fp32)
    assert np.all(np.abs(np_(O) - Oref) <=
                  2.0 ** -8 * np.abs(Oref) + 2.0 ** -10 * np.abs(V64).max())
    assert np.allclose(np_(lse), lref, rtol=0, atol=1e-4)
    drawn = np_(kv.w)[:, :, :50] - w0[:, :, :50]
    assert np.all(w0[:, :, 30:] == 0) and np.all(np_(kv.w)[:, :, 50:] == 0)
    assert np.allclose(drawn, oracle.kv4_weight(s, lref, Hkv), rtol=2.0 ** -14, atol=2.0 ** -20)


def _filled(B, N, Hq, Hkv, dh, T, seed):
    g = torch.Generator().manual_seed(seed)
    kv = Kv4Layer(B, N, Hq, Hkv, dh, 0.25, 0.25)
    kv.append(*(torch.randn(B, T, Hkv, dh, generator=g).bfloat16().cuda() for _ in range(2)))
    kv.w.copy_(torch.rand(B, Hkv, N, generator=g))
    return kv


def _state(kv):
    return (*kv.cache.buffers, kv.w, kv.kpos, kv.len)


def test_evictions_on_another_stream():
    """With the current stream held up: everything an eviction does, the new
    buffers' first values included, is on the stream that was given, and the next
    owner of a spare waits for the last one."""
    want = [_filled(2, 300, 4, 2, 64, 200, i) for i in range(2)]
    got = [_filled(2, 300, 4, 2, 64, 200, i) for i in range(2)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for keep in (120, 50):
        for kv in want:
            kv.evict(keep, sink=1, recent=3)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)           # about 0.1 s, on the current stream
    got[0].evict(120, sink=1, recent=3, stream=s[0])
    with torch.cuda.stream(s[0]):
        torch.cuda._sleep(100_000_000)       # layer 0's old rows are not given up before this
        spare = got[0].evict(50, sink=1, recent=3, stream=s[0].cuda_stream)
    got[1].evict(120, sink=1, recent=3, spare=spare, stream=s[1])
    got[1].evict(50, sink=1, recent=3, stream=s[1])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert a.len.tolist() == b.len.tolist() == [50, 50]
        assert all(torch.equal(x[:, :, :50], y[:, :, :50])
                   for x, y in zip(_state(a)[:6], _state(b)[:6]))
        assert torch.equal(a.w, b.w) and torch.equal(a.kpos, b.kpos)


def test_attention_on_two_streams_at_once(monkeypatch):
    """A call's partial sums are its own: the same shape on two streams gives
    what each gives alone."""
    B, N, Hq, Hkv, dh = 1, 20000, 8, 2, 128
    kv = _filled(B, N, Hq, Hkv, dh, N, 3)
    g = torch.Generator().manual_seed(4)
    Qs = [torch.randn(B, 1, Hq, dh, generator=g).bfloat16().cuda() for _ in range(2)]
    want, outs = [], []
    for Q in Qs:
        O, lse = torch.zeros_like(Q), torch.zeros(B, 1, Hq, device="cuda")
        kv.attend(Q, O, lse)
        want.append((O, lse))
    assert ps.ps_workspace_bytes(ps.OP_KV4_ATTN, B=B, N=N, Hq=Hq, Hkv=Hkv, dh=dh, P=1) > 0
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    used, call = {}, ps.ps_kv4_attn
    monkeypatch.setattr(ps, "ps_kv4_attn", lambda *a, ws, stream, **k: (
        used.setdefault(stream, ws.data_ptr()), call(*a, ws=ws, stream=stream, **k)))
    for i in range(40):
        for Q, s in zip(Qs, streams):
            O, lse = torch.zeros_like(Q), torch.zeros(B, 1, Hq, device="cuda")
            s.wait_stream(torch.cuda.current_stream())
            kv.attend(Q, O, lse, stream=s)
            outs.append((O, lse))
    torch.cuda.synchronize()
    for i, (O, lse) in enumerate(outs):
        assert torch.equal(O, want[i % 2][0]) and torch.equal(lse, want[i % 2][1]), i
    assert used[streams[0]] != used[streams[1]]


@pytest.mark.parametrize("B,R,Hkv,dh,N,dtype", [
    (2, 60, 3, 64, 50, torch.bfloat16), (1, 9, 2, 256, 1, torch.float32),
    (3, 200, 1, 128, 130, torch.float32), (1, 1, 5, 128, 700, torch.bfloat16)])
@pytest.mark.parametrize("listed", [False, True])
def test_store_by_positions(B, R, Hkv, dh, N, dtype, listed):
    """Rows to the slots that hold their positions, which differ from head to head;
    everything else untouched: bits as the oracle's."""
    rng = np.random.default_rng(R + N)
    K, V = (torch.from_numpy(rng.standard_normal((B, R, Hkv, dh)).astype(np.float32)).to(dtype)
            for _ in range(2))
    span = max(N, R) + 40
    kpos = np.sort(np.stack([[rng.choice(span, N, False) for _ in range(Hkv)]
                             for _ in range(B)]), -1) - 20
    off = rng.integers(-10, 10, B)
    rows = rng.integers(-2, R + 2, (B, R))
    cnt = rng.integers(0, R + 1, B)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    bufs = [Guarded((B, Hkv, N, dh // q), torch.uint8, fill=0x3C) for q in (2, 16, 2, 16)]
    c = ps.Kv4Cache(*(g.t for g in bufs), kmul=0.7, vmul=0.3)
    opt = dict(rows=i32(rows), cnt=i32(cnt)) if listed else {}
    ps.ps_kv4_store(c, K.cuda(), V.cuda(), off=i32(off), kpos=i32(kpos), **opt)
    enc = [oracle.kv4_encode(X.float().numpy().transpose(0, 2, 1, 3), S)
           for X, S in ((K, 0.7), (V, 0.3))]
    for b in range(B):
        entries = rows[b, :cnt[b]] if listed else np.arange(R)
        named = {int(r) + int(off[b]): int(r) for r in entries if 0 <= r < R}
        for h in range(Hkv):
            for n in range(N):
                r = named.get(int(kpos[b, h, n]))
                for i, g in enumerate(bufs):
                    want = 0x3C if r is None else enc[i // 2][i % 2][b, h, r]
                    assert np.all(np_(g.t[b, h, n]) == want), (b, h, n, r)
    assert all(g.intact() for g in bufs)


@pytest.mark.parametrize("B,Hkv,dh,N,M,keep", [
    (2, 3, 64, 100, 100, 40), (1, 2, 128, 3000, 2000, 700), (3, 1, 64, 9000, 9100, 8000),
    (1, 1, 256, 5, 5, 5)])
@pytest.mark.parametrize("again", [False, True])
def test_an_eviction_that_goes_on(B, Hkv, dh, N, M, keep, again):
    """ps_kv4_evict_on: what ps_kv4_evict gives, and behind it the positions that come
    next, without weight; from slots and from positions that were shifted before."""
    rng = np.random.default_rng(N)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    src = ps.Kv4Cache(*(torch.from_numpy(rng.integers(0, 256, (B, Hkv, N, dh // q), dtype=np.uint8))
                        .cuda() for q in (2, 16, 2, 16)))
    w = torch.rand(B, Hkv, N, device="cuda")
    length = rng.integers(0, N + 1, B)
    length[0] = N
    shift = rng.integers(1, 1000, B) if again else np.zeros(B, int)
    kpos = np.arange(N) + shift[:, None, None] + np.zeros((B, Hkv, 1), int)
    opt = dict(len=i32(length), kpos=i32(kpos) if again else None,
               ws=ps.workspace(ps.OP_KV4_EVICT, B=B, N=N, Hkv=Hkv, k=keep))
    sink = min(2, keep)
    got, want = [], []
    for out in (got, want):
        d = ps.Kv4Cache(*(torch.full((B, Hkv, M, dh // q), 0x3C, dtype=torch.uint8, device="cuda")
                          for q in (2, 16, 2, 16)))
        wd = Guarded((B, Hkv, M), torch.float32, fill=5)
        kd = Guarded((B, Hkv, M), torch.int32, fill=-9)
        ld, sd = Guarded((B,), torch.int32, fill=-9), Guarded((B,), torch.int32, fill=-9)
        on = dict(shift=i32(shift) if again else None, shift_dst=sd.t) if out is got else {}
        ps.ps_kv4_evict(src, d, w, wd.t, ld.t, keep, sink=sink, kpos_dst=kd.t, **opt, **on)
        assert all(g.intact() for g in (wd, kd, ld, sd))
        out.extend([*d.buffers, wd.t, kd.t, ld.t, sd.t])
    kept = np.minimum(length, keep)
    assert got[6].tolist() == list(kept) == want[6].tolist()
    assert got[7].tolist() == list(shift + length - kept) and want[7].tolist() == [-9] * B
    for b in range(B):
        k = int(kept[b])
        for x, y in zip(got[:6], want[:6]):
            assert torch.equal(x[b, :, :k], y[b, :, :k])
        assert all(bool((x[b, :, k:] == 0x3C).all()) for x in got[:4])
        assert bool((got[4][b, :, k:] == 0).all())
        after = torch.arange(k, M, dtype=torch.int32) + int(shift[b] + length[b] - k)
        assert torch.equal(got[5][b, :, k:].cpu(), after.expand(Hkv, -1))
        assert bool((want[5][b, :, k:] == -9).all()) and bool((want[4][b, :, k:] == 5).all())


def test_what_an_eviction_that_goes_on_needs():
    c, d = ps.Kv4Cache.empty(1, 1, 30, 64), ps.Kv4Cache.empty(1, 1, 30, 64)
    w, wd = torch.zeros(1, 1, 30, device="cuda"), torch.zeros(1, 1, 30, device="cuda")
    ld, sd = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    kd = torch.zeros(1, 1, 30, dtype=torch.int32, device="cuda")
    ws = ps.workspace(ps.OP_KV4_EVICT, B=1, N=30, Hkv=1, k=5)
    for bad in (dict(shift_dst=sd), dict(shift=sd, shift_dst=sd, kpos_dst=kd)):
        with pytest.raises(ps.PolestarError) as e:
            ps.ps_kv4_evict(c, d, w, wd, ld, 5, ws=ws, **bad)
        assert e.value.status == ps.PS_ERR_ARG
    for bad in (dict(shift_dst=sd.long(), kpos_dst=kd),
                dict(shift_dst=sd, kpos_dst=kd, shift=wd[0])):
        with pytest.raises(ValueError):
            ps.ps_kv4_evict(c, d, w, wd, ld, 5, ws=ws, **bad)
    K = torch.zeros(1, 4, 1, 64, device="cuda")
    with pytest.raises(ValueError):
        ps.ps_kv4_store(c, K, K, kpos=kd[:, :, :20])
