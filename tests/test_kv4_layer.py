"""Kv4Layer's own bookkeeping on the CPU: which buffers a layer owns, what its
slots hold, how far it is filled.  The native calls are stood in for by the
oracle on CPU tensors."""
import numpy as np
import pytest
import torch

import oracle
from drift_aware_kv_spherical_gb300 import kv4
from drift_aware_kv_spherical_gb300 import polestar as ps

B, N, HQ, HKV, DH = 2, 24, 4, 2, 64
KMUL, VMUL = 0.25, 0.125


class _Cache:
    """A Kv4Cache over CPU tensors."""

    def __init__(self, kcode, kscale, vcode, vscale, kmul=1.0, vmul=1.0):
        self.buffers = (kcode, kscale, vcode, vscale)
        self.B, self.Hkv, self.N, half = kcode.shape
        self.dh, self.kmul, self.vmul, self.device = 2 * half, kmul, vmul, kcode.device

    @classmethod
    def empty(cls, B, Hkv, N, dh, kmul=1.0, vmul=1.0, device="cpu"):
        mk = [torch.zeros(B, Hkv, N, dh // q, dtype=torch.uint8) for q in (2, 16, 2, 16)]
        return cls(*mk, kmul=kmul, vmul=vmul)


def _store(c, K, V, off=None, rows=None, cnt=None, stream=None, kpos=None):
    R = K.shape[1]
    for b in range(c.B):
        n = R if cnt is None else min(int(cnt[b]), R)
        for j in range(n):
            r = j if rows is None else int(rows[b, j])
            at = r + (0 if off is None else int(off[b]))
            if not 0 <= r < R:
                continue
            for X, S, code, scale in ((K, c.kmul, *c.buffers[:2]), (V, c.vmul, *c.buffers[2:])):
                a, s = oracle.kv4_encode(X[b, r].float().numpy(), S)
                for h in range(c.Hkv):
                    held = torch.arange(c.N) if kpos is None else kpos[b, h]
                    for n in (held == at).nonzero().flatten():
                        code[b, h, n] = torch.from_numpy(a[h])
                        scale[b, h, n] = torch.from_numpy(s[h])


def _evict(src, dst, w, w_dst, len_dst, keep, sink=0, recent=0, len=None, kpos=None,
           kpos_dst=None, ws=None, stream=None, shift=None, shift_dst=None):
    if sink + recent > keep or keep > dst.N:
        raise ps.PolestarError(ps.PS_ERR_ARG, "ps_kv4_evict")
    assert not set(t.data_ptr() for t in src.buffers) & set(t.data_ptr() for t in dst.buffers)
    for b in range(src.B):
        n = int(len[b])
        len_dst[b] = min(n, keep)
        if shift_dst is not None:
            shift_dst[b] = (0 if shift is None else int(shift[b])) + n - min(n, keep)
        for h in range(src.Hkv):
            at = torch.from_numpy(oracle.kv4_keep(w[b, h].numpy(), n, keep, sink, recent))
            k = at.numel()
            for x, y in zip(src.buffers, dst.buffers):
                y[b, h, :k] = x[b, h, at]
            w_dst[b, h, :k] = w[b, h, at]
            kpos_dst[b, h, :k] = (at if kpos is None else kpos[b, h, at]).int()
            if shift_dst is not None:
                w_dst[b, h, k:] = 0
                kpos_dst[b, h, k:] = torch.arange(k, dst.N) + int(shift_dst[b])


@pytest.fixture(autouse=True)
def _native(monkeypatch):
    monkeypatch.setattr(ps, "Kv4Cache", _Cache)
    monkeypatch.setattr(ps, "ps_kv4_store", _store)
    monkeypatch.setattr(ps, "ps_kv4_evict", _evict)
    monkeypatch.setattr(ps, "ps_workspace_bytes", lambda op, **k: 0)


def _layer():
    return kv4.Kv4Layer(B, N, HQ, HKV, DH, KMUL, VMUL, device="cpu")


def _rows(T, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, T, HKV, DH, generator=g).bfloat16(),
            torch.randn(B, T, HKV, DH, generator=g).bfloat16())


def _weights(layer, seed):
    layer.w.copy_(torch.rand(layer.w.shape, generator=torch.Generator().manual_seed(seed)))


def _snap(layer):
    return [t.clone() for t in (*layer.cache.buffers, layer.w, layer.kpos, layer.len)]


def _owned(layer):
    ts = (*layer.cache.buffers, layer.w, layer.kpos, layer.len)
    return {t.data_ptr() for t in ts}


# ---- whose buffers they are
@pytest.mark.parametrize("carry", [False, True])
def test_layers_that_pass_one_spare_on_keep_their_own_rows(carry):
    """Two rounds of evictions over three layers with one spare, given up between
    the rounds or carried over: no layer's live buffers are another's, and every
    layer ends as a layer that was evicted by itself."""
    layers, alone = [_layer() for _ in range(3)], [_layer() for _ in range(3)]
    for i, (a, b) in enumerate(zip(layers, alone)):
        for x in (a, b):
            x.append(*_rows(20, i))
            _weights(x, i)
    spare = None
    for keep in (12, 7):
        if not carry:
            spare = None
        for layer in layers:
            others = [_snap(x) for x in layers if x is not layer and x.kpos is not None]
            spare = layer.evict(keep, sink=1, recent=2, spare=spare)
            after = [_snap(x) for x in layers if x is not layer and x.kpos is not None]
            assert all(torch.equal(p, q) for x, y in zip(others, after) for p, q in zip(x, y))
        for layer in alone:
            layer.evict(keep, sink=1, recent=2)
        live = [_owned(x) for x in layers]
        assert all(not (live[i] & live[j]) for i in range(3) for j in range(i))
        for a, b in zip(layers, alone):
            assert a.len.tolist() == [keep] * B == b.len.tolist()
            for x, y in zip(_snap(a)[:6], _snap(b)[:6]):
                assert torch.equal(x[:, :, :keep], y[:, :, :keep])


def test_a_spare_serves_one_eviction():
    a, b = _layer(), _layer()
    for x in (a, b):
        x.append(*_rows(10, 1))
        _weights(x, 1)
    spare = a.evict(6)
    b.evict(6, spare=spare)
    with pytest.raises(ValueError):
        a.evict(4, spare=spare)
    own = a.evict(4)                 # makes buffers of its own again
    with pytest.raises(ps.PolestarError):
        a.evict(2, sink=3)           # a refused call changes nothing
    assert own["cache"] is not a.cache and a.len.tolist() == [4, 4]
    assert a.evict(2)["len"].tolist() == [4, 4]
    assert not own                   # was a's own spare, and is its live cache now


# ---- what the slots hold
def test_slots_behind_the_kept_ones_hold_nothing_of_an_older_cache():
    """After every eviction they are the next positions' and have no weight."""
    a = _layer()
    a.append(*_rows(N, 2))
    a.len.copy_(torch.tensor([N, N - 5]))
    for keep in (15, 9, 4):
        _weights(a, keep)
        a.evict(keep, recent=1)
        for b, total in enumerate((N, N - 5)):
            assert torch.all(a.w[b, :, keep:] == 0)
            want = torch.arange(total, total + N - keep, dtype=torch.int32).expand(HKV, -1)
            assert torch.equal(a.kpos[b, :, keep:], want)
            assert torch.all(a.kpos[b, :, keep - 1] == total - 1)   # the last one is kept
    short = _layer()                 # fewer slots than are kept
    short.append(*_rows(6, 3))
    _weights(short, 3)
    short.evict(10)
    assert torch.equal(short.kpos, torch.arange(N, dtype=torch.int32).expand(B, HKV, N))
    assert torch.all(short.w[:, :, 6:] == 0)


@pytest.mark.parametrize("cuts", [[(20, 8)], [(20, 8), (3, 9), (7, 5)]])
def test_appending_goes_on_after_an_eviction(cuts):
    """Append, evict, append, ...: every slot holds the row of the position that
    kpos names, sequences of unequal length too, and new tokens compete for their
    place in the next eviction by the weight they drew themselves."""
    a = _layer()
    K, V = _rows(48, 4)
    code, scale = oracle.kv4_encode(K.float().numpy().transpose(0, 2, 1, 3), KMUL)
    a.append(K[:, :2], V[:, :2])
    a.len[1] = 0                     # the second sequence starts two tokens later
    at, total = 2, np.array([2, 0])
    for T, keep in cuts:
        for _ in range(T):           # row `at` of sequence b is its position total[b]
            a.append(K[:, at:at + 1], V[:, at:at + 1])
            at += 1
            total += 1
        filled = a.len.clone()
        _weights(a, keep)
        for b in range(B):
            a.w[b, :, int(filled[b]):] = 0
        a.evict(keep, sink=1, recent=2)
        assert a.len.tolist() == [min(int(n), keep) for n in filled]
        for b in range(B):
            n = int(a.len[b])
            first = at - total[b]    # the row of its position 0
            for h in range(HKV):
                pos = a.kpos[b, h, :n].numpy()
                assert np.all(np.diff(pos) > 0) and pos[-1] == total[b] - 1
                assert np.array_equal(a.cache.buffers[0][b, h, :n], code[b, h, pos + first])
                assert np.array_equal(a.cache.buffers[1][b, h, :n], scale[b, h, pos + first])
    a.append(K[:, at:at + 4], V[:, at:at + 4])
    for b in range(B):
        n = int(a.len[b])
        assert a.kpos[b, 0, n - 4:n].tolist() == list(range(total[b], total[b] + 4))
        assert torch.all(a.w[b, :, n - 4:] == 0)


@pytest.mark.parametrize("how", ["all", "cnt", "rows", "rows+cnt", "off"])
def test_a_store_after_an_eviction_goes_to_the_slots_of_its_positions(how):
    """Every head's slot takes the row of the position it holds; evicted positions,
    unlisted rows and entries out of range leave everything as it was."""
    a = _layer()
    a.append(*_rows(20, 6))
    _weights(a, 6)                   # other slots are kept for every head
    a.evict(11, sink=1, recent=3)
    before = [t.clone() for t in (*a.cache.buffers, a.kpos, a.w, a.len)]
    R = 20
    K, V = _rows(R, 7)
    g = np.random.default_rng(8)
    rows = np.full((B, R), -1)
    rows[0, :9] = [3, 0, 19, 7, 12, -4, 20, 99, 5]
    rows[1] = g.permutation(R)
    cnt, off = np.array([8, 5]), np.array([2, -3])
    opt = {}
    if "rows" in how:
        opt["rows"] = torch.from_numpy(rows.astype(np.int32))
    if "cnt" in how:
        opt["cnt"] = torch.from_numpy(cnt.astype(np.int32))
    if how == "off":
        opt["off"] = torch.from_numpy(off.astype(np.int32))
    a.store(K, V, **opt)
    enc = [oracle.kv4_encode(X.float().numpy().transpose(0, 2, 1, 3), S)
           for X, S in ((K, KMUL), (V, VMUL))]
    for b in range(B):
        entries = range(R) if "rows" not in how else rows[b]
        entries = list(entries)[:cnt[b]] if "cnt" in how else list(entries)
        named = {int(r) + (int(off[b]) if how == "off" else 0): int(r)
                 for r in entries if 0 <= r < R}
        for h in range(HKV):
            for n in range(N):
                r = named.get(int(a.kpos[b, h, n]))
                for i, x in enumerate(a.cache.buffers):
                    want = before[i][b, h, n] if r is None else \
                        torch.from_numpy(enc[i // 2][i % 2][b, h, r])
                    assert torch.equal(x[b, h, n], want), (b, h, n, r)
    assert all(torch.equal(x, y) for x, y in zip((a.kpos, a.w, a.len), before[4:]))


def test_an_eviction_changes_what_a_captured_store_holds():
    a = _layer()
    a.append(*_rows(20, 9))
    seen = {a.addresses()}
    for keep in (12, 11):            # twice: the first buffers again, now with kpos
        a.evict(keep)
        assert a.addresses() not in seen
        seen.add(a.addresses())


# ---- how much it keeps
def test_workspaces_of_many_lengths_share_a_few_buffers(monkeypatch):
    """Prompts of every length up to 300 and evictions to many sizes keep no more
    than four times the largest call's bytes (powers of two up to the next one);
    every call has enough."""
    need = lambda op, B, N, Hq, Hkv, dh, P=0, k=0: 1000 * (P + k)  # noqa: E731
    kv4._ws_bytes.cache_clear()
    monkeypatch.setattr(ps, "ps_workspace_bytes", need)
    seen = []
    for name in ("ps_kv4_attn", "ps_kv4_weight"):
        monkeypatch.setattr(ps, name, lambda *a, ws, **k: seen.append(ws))
    a = _layer()
    for T in range(1, 301):
        a.attend(torch.zeros(B, T, HQ, DH), None)
        a.weigh(torch.zeros(B, T, HQ, DH), None)
        assert all(ws.nbytes >= 1000 * T for ws in seen[-2:])
    kept = {ws.data_ptr(): ws.nbytes for ws in seen}
    assert sum(kept.values()) <= 4 * 300 * 1000
    kv4._ws_bytes.cache_clear()


# ---- how far it is filled
def test_appending_past_the_capacity_is_refused():
    """A call that some sequence has no room for raises and changes nothing, however
    `len` came to be what it is; one that fits exactly does not."""
    def full(layer, T, why):
        before = [t.clone() for t in (*layer.cache.buffers, layer.len)]
        with pytest.raises(ValueError, match="no room"):
            layer.append(*_rows(T, 1))
        after = (*layer.cache.buffers, layer.len)
        assert all(torch.equal(x, y) for x, y in zip(before, after)), why

    a = _layer()
    full(a, N + 1, "empty")
    a.append(*_rows(N - 1, 2))
    full(a, 2, "one slot left")
    a.append(*_rows(1, 3))
    full(a, 1, "filled by appends")
    _weights(a, 1)
    a.evict(10)
    a.append(*_rows(N - 10, 4))
    full(a, 1, "filled again after an eviction")
    a.len[0] = 3                      # the other sequence is full still
    full(a, 1, "changed in place")
    a.len = torch.tensor([3, N - 2], dtype=torch.int32)
    full(a, 3, "replaced")
    a.append(*_rows(2, 5))
    assert a.len.tolist() == [5, N]
    a.evict(4)                        # of a len that was set by the caller
    assert a.len.tolist() == [4, 4]
    full(a, N - 3, "known from the eviction")
    a.append(*_rows(N - 4, 6))
    b = _layer()
    b.len.fill_(N)
    full(b, 1, "filled by the caller")


def test_appending_reads_nothing_back(monkeypatch):
    """A loop of appends and evictions never waits for the device to learn `len`."""
    a = _layer()
    monkeypatch.setattr(torch.Tensor, "tolist", None)
    for _ in range(3):
        a.append(*_rows(12, 1))
        a.evict(12)
