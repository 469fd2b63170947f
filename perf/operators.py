"""The workloads of the 4-bit KV cache operators (store, load, attention,
accumulated weight, eviction), each with a plain form in elementary torch
operations.

A cache holds K and V rows of every (sequence, KV head, slot) as E2M1 codes
[B][Hkv][N][dh/2] (element 2j in the low nibble of byte j) with one E4M3 scale
per 16 elements [B][Hkv][N][dh/16] and a tensor scale; an element is
value(code) * scale * tensor scale.

`own` False: the plain form, 32-bit arithmetic on the same packed buffers.
`own` True: the calls a user makes of drift_aware_kv_spherical_gb300.polestar.
"""

import math

import numpy as np
import torch

own = False

KMUL, VMUL = 0.25, 0.0625   # tensor scales of K and V, as a calibration leaves them


# ------------------------------------------------------------------- the cases
def _attn(name, B, T, Hq, Hkv, dh, N, dtype="bf16", ragged=False, span="", cap=0.0, bias=False):
    return dict(name=name, op="attn", B=B, T=T, Hq=Hq, Hkv=Hkv, dh=dh, N=N, dtype=dtype,
                ragged=ragged, span=span, cap=cap, bias=bias)


def listed():
    return [
        # one token of a Dream-7B-shaped layer (28 query, 4 KV heads) against a
        # 1024-slot cache: the call whose latency a single user waits for
        _attn("attn_token_dream", 1, 1, 28, 4, 128, 1024),
        # one token for each of eight users with long, unequal histories; capped scores
        _attn("attn_token_long", 8, 1, 28, 4, 128, 65536, ragged=True, cap=30.0),
        # a 32-token block of four LLaDA-8B-shaped sequences against their 768-row
        # windows: a step of block decoding
        _attn("attn_block_llada", 4, 32, 32, 32, 128, 768),
        # packed documents with a shared prompt: every query sees its own document or
        # the rows of the prompt before it, some (padding) see nothing; distance bias
        # and capped scores; lengths that fill no tile
        _attn("attn_window_documents", 4, 1001, 28, 4, 128, 2047, ragged=True,
              span="documents", cap=50.0, bias=True),
        # every position of a 4096-row window against the whole window: the pass that
        # rebuilds a window
        _attn("attn_window_dense", 2, 4096, 32, 32, 128, 4096),
        # the tiny fp32 layer (4 heads of 64), causal
        _attn("attn_tiny_f32", 1, 16, 4, 4, 64, 128, dtype="f32", span="causal"),
        # the weight one token a user puts on a long cache, added to what earlier
        # tokens left there
        dict(name="weight_token_long", op="weight", B=8, T=1, Hq=28, Hkv=4, dh=128, N=32768,
             dtype="bf16", ragged=True, span="", cap=0.0, bias=False),
        # the weight a 32-token block puts on a 4096-row cache
        dict(name="weight_block_llada", op="weight", B=4, T=32, Hq=32, Hkv=32, dh=128, N=4096,
             dtype="bf16", ragged=False, span="", cap=0.0, bias=False),
        # one user's cache cut from 2048 rows to 1024, then read back
        dict(name="evict_dream", op="evict", B=1, Hkv=4, dh=128, N=2048, keep=1024, sink=4,
             recent=32, ragged=False),
        # eight sequences of 32 heads cut from up to 8192 rows to 4096, then read back
        dict(name="evict_batch", op="evict", B=8, Hkv=32, dh=128, N=8192, keep=4096, sink=4,
             recent=64, ragged=True),
        # the positions that one sparse refresh touched (a list, unequal counts) of a
        # four-sequence 768-row window, stored and read back
        dict(name="store_refresh", op="store", B=4, R=768, Hkv=32, dh=128, N=768, dtype="bf16",
             listed=True),
        # a whole batch of 4096-row windows stored and read back
        dict(name="store_window", op="store", B=8, R=4096, Hkv=32, dh=128, N=4096,
             dtype="bf16", listed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# a drawn case does no more than these (the largest listed case's, and room for
# the plain form's score matrices)
_MOST_FLOPS = 5.0e11
_MOST_BYTES = 1.3e9


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "weight", "evict", "store"])
    while True:
        Hq, Hkv = rng.choice([(4, 4), (28, 4), (32, 32), (32, 8), (8, 1), (16, 16)])
        dh = rng.choice([64, 128, 128])
        B = _log(rng, 1, 16)
        if op in ("attn", "weight"):
            T = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 64, 2048)])
            c = dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, dh=dh, N=_log(rng, 64, 65536),
                     dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]),
                     ragged=rng.random() < 0.5,
                     span=rng.choice(["", "", "causal", "prefix", "documents"]),
                     cap=rng.choice([0.0, 0.0, 30.0, 50.0]), bias=rng.random() < 0.25)
        elif op == "evict":
            N = _log(rng, 128, 16384)
            keep = max(8, int(N * rng.uniform(0.2, 0.9)))
            c = dict(op=op, B=B, Hkv=Hkv, dh=dh, N=N, keep=keep, sink=rng.choice([0, 1, 4]),
                     recent=rng.randint(0, keep // 2 - 2), ragged=rng.random() < 0.5)
        else:
            R = _log(rng, 1, 8192)
            c = dict(op=op, B=B, R=R, Hkv=Hkv, dh=dh, N=R + rng.randint(0, 64),
                     dtype=rng.choice(["bf16", "bf16", "f32"]), listed=rng.random() < 0.5)
        w = work(c)
        scores = B * c.get("T", 0) * Hq * c["N"]
        if w["flops"] <= _MOST_FLOPS and w["bytes"] <= _MOST_BYTES and scores <= 1.0e9:
            return c


# ------------------------------------------------------------------- inputs
def _dt(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _encode(x, mul):
    """E2M1 codes and E4M3 scales of x [..., dh] (f32), 16 elements a block."""
    shape = x.shape
    x = x.reshape(*shape[:-1], shape[-1] // 16, 16)
    m = torch.tensor(mul, dtype=torch.float32, device=x.device)
    s8 = (x.abs().amax(-1) / (6.0 * m)).clamp(max=448.0).to(torch.float8_e4m3fn)
    g = (s8.float() * m)[..., None]
    y = torch.where(g > 0, x / g, torch.zeros_like(x))
    a = y.abs()
    idx = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
           + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8)
           + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    c = (idx + 8 * torch.signbit(y).to(torch.uint8)).reshape(*shape[:-1], shape[-1] // 2, 2)
    return c[..., 0] + 16 * c[..., 1], s8.view(torch.uint8)


def _decode(code, scale, mul):
    """f32 values [..., dh] of codes [..., dh/2] and scales [..., dh/16]."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0,
                        -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=code.device)
    v = lut[torch.stack((code & 15, code >> 4), -1).int()]
    v = v.reshape(*scale.shape, 16) * scale.view(torch.float8_e4m3fn).float()[..., None]
    return v.reshape(*code.shape[:-1], 2 * code.shape[-1]) * mul


def _spans(case, seed, lens):
    """[lo, hi) of the positions that each query row sees, and the rows' positions."""
    B, T, N = case["B"], case["T"], case["N"]
    r = np.random.RandomState(seed % (1 << 31))
    # the queries are the last T positions of their sequence (or all of them)
    qpos = np.maximum(lens[:, None] - T, 0) + np.arange(T)[None, :]
    span = np.zeros((B, T, 2), np.int32)
    if case["span"] == "causal":
        span[..., 1] = qpos + 1
    elif case["span"] == "prefix":      # a prompt that everyone sees, then causal
        span[..., 1] = np.maximum(qpos + 1, (lens // 2)[:, None])
    else:
        for b in range(B):
            cuts = np.unique(np.concatenate([[0], r.randint(0, N + 1, max(1, N // 256)), [N]]))
            d = np.minimum(np.searchsorted(cuts, qpos[b], side="right") - 1, len(cuts) - 2)
            span[b, :, 0], span[b, :, 1] = cuts[d], cuts[d + 1]
            span[b, r.rand(T) < 0.05] = 0     # padding rows see nothing
    return span, qpos.astype(np.int32)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    r = np.random.RandomState((int(seed) + 77) % (1 << 31))
    B, Hkv, dh, N, op = case["B"], case["Hkv"], case["dh"], case["N"], case["op"]
    i32 = dict(dtype=torch.int32, device=dev)
    st = dict(case=dict(case))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def cache(n):
        # hidden channels of a trained model have unequal spreads, K's most
        ks = torch.exp(0.5 * normal(Hkv, 1, dh))
        kc, ks8 = _encode((normal(B, Hkv, n, dh) * ks).bfloat16().float(), KMUL)
        vc, vs8 = _encode((normal(B, Hkv, n, dh) * 0.5).bfloat16().float(), VMUL)
        return kc, ks8, vc, vs8

    if op == "store":
        R = case["R"]
        st["K"] = (normal(B, R, Hkv, dh) * 1.3).to(_dt(case))
        st["V"] = (normal(B, R, Hkv, dh) * 0.5).to(_dt(case))
        st["cache"] = tuple(torch.zeros(B, Hkv, N, dh // q, dtype=torch.uint8, device=dev)
                            for q in (2, 16, 2, 16))
        st["off"] = torch.from_numpy(r.randint(0, N - R + 1, B).astype(np.int32)).to(dev)
        st["rows"] = st["cnt"] = None
        if case["listed"]:               # ascending positions, -1 behind them
            rows = np.full((B, R), -1, np.int32)
            cnt = np.zeros(B, np.int32)
            for b in range(B):
                p = np.flatnonzero(r.rand(R) < r.uniform(0.05, 0.3))
                rows[b, :p.size], cnt[b] = p, p.size
            st["rows"], st["cnt"] = torch.from_numpy(rows).to(dev), torch.from_numpy(cnt).to(dev)
        st["K_back"], st["V_back"] = torch.zeros_like(st["K"]), torch.zeros_like(st["V"])
        return st

    st["cache"] = cache(N)
    lens = r.randint(max(1, N // 2), N + 1, B) if case["ragged"] else np.full(B, N)
    st["len"] = torch.from_numpy(lens.astype(np.int32)).to(dev)
    if op == "evict":
        keep = case["keep"]
        st["w"] = torch.exp(2.0 * normal(B, Hkv, N)) * 0.01     # a few rows draw most weight
        st["kpos"] = torch.arange(N, **i32).expand(B, Hkv, N).contiguous()
        st["dst"] = tuple(torch.zeros(B, Hkv, keep, dh // q, dtype=torch.uint8, device=dev)
                          for q in (2, 16, 2, 16))
        st["w_dst"] = torch.zeros(B, Hkv, keep, device=dev)
        st["kpos_dst"] = torch.zeros(B, Hkv, keep, **i32)
        st["len_dst"] = torch.zeros(B, **i32)
        st["K_back"] = torch.zeros(B, keep, Hkv, dh, dtype=torch.bfloat16, device=dev)
        st["V_back"] = torch.zeros_like(st["K_back"])
        return st

    T, Hq = case["T"], case["Hq"]
    st["Q"] = (normal(B, T, Hq, dh) * 1.2).to(_dt(case))
    st["scale"] = 1.0 / math.sqrt(dh)
    st["span"] = st["qpos"] = st["slope"] = None
    span, qpos = _spans(case, int(seed) + 5, lens)
    if case["span"]:
        st["span"] = torch.from_numpy(span).to(dev)
    if case["bias"]:
        st["qpos"] = torch.from_numpy(qpos).to(dev)
        st["slope"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev).float() / Hq)
    if op == "attn":
        st["O"] = torch.zeros_like(st["Q"])
        st["lse"] = torch.zeros(B, T, Hq, device=dev)
    else:
        st["lse"] = torch.logsumexp(_scores(st), -1).reshape(B, Hkv, T, Hq // Hkv).permute(
            0, 2, 1, 3).reshape(B, T, Hq).contiguous()
        # earlier tokens left about as much as these will
        st["w"] = torch.rand(B, Hkv, N, generator=g, device=dev) * (2.0 * T * (Hq // Hkv) / N)
        st["w_out"] = torch.zeros_like(st["w"])
    return st


# ------------------------------------------------------------------- plain forms
def _scores(st):
    """Scores [B][Hkv][T * G][N] (row t * G + j: token t, head j of the group),
    -inf where a row does not see a slot."""
    c = st["case"]
    B, T, Hq, Hkv, dh, N = c["B"], c["T"], c["Hq"], c["Hkv"], c["dh"], c["N"]
    G = Hq // Hkv
    q = st["Q"].float().reshape(B, T, Hkv, G, dh).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, dh)
    k = _decode(st["cache"][0], st["cache"][1], KMUL)
    s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    if c["cap"] > 0:
        s = c["cap"] * torch.tanh(s / c["cap"])
    pos = torch.arange(N, device=s.device)
    s = s.reshape(B, Hkv, T, G, N)
    if c["bias"]:
        dist = (st["qpos"][:, :, None] - pos).abs().float()
        s = s - st["slope"].reshape(Hkv, 1, G, 1) * dist[:, None, :, None, :]
    see = (pos < st["len"][:, None])[:, None, :]
    if st["span"] is not None:
        see = see & (pos >= st["span"][..., :1]) & (pos < st["span"][..., 1:])
    s = s.masked_fill(~see[:, None, :, None, :], -math.inf)
    return s.reshape(B, Hkv, T * G, N)


def _rows_back(x, c):
    """[B][Hkv][T * G][...] to [B][T][Hq][...]."""
    B, T, Hq, Hkv = c["B"], c["T"], c["Hq"], c["Hkv"]
    x = x.reshape(B, Hkv, T, Hq // Hkv, *x.shape[3:])
    return x.transpose(1, 2).reshape(B, T, Hq, *x.shape[4:])


def _plain_attn(st):
    c = st["case"]
    s = _scores(st)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _decode(st["cache"][2], st["cache"][3], VMUL)) / l.clamp(min=1e-38)
    lse = (torch.log(l) + m).squeeze(-1)
    return _rows_back(o, c).to(st["Q"].dtype), _rows_back(lse, c)


def _plain_weight(st):
    c = st["case"]
    B, T, Hq, Hkv = c["B"], c["T"], c["Hq"], c["Hkv"]
    lse = st["lse"].reshape(B, T, Hkv, Hq // Hkv).permute(0, 2, 1, 3).reshape(B, Hkv, -1, 1)
    p = torch.exp(_scores(st) - lse)
    p = torch.where(torch.isinf(lse), torch.zeros_like(p), p)
    return st["w"] + p.sum(2)


def _plain_evict(st):
    c = st["case"]
    B, Hkv, N, keep = c["B"], c["Hkv"], c["N"], c["keep"]
    n = st["len"].long()[:, None, None]
    slot = torch.arange(N, device=n.device).expand(B, Hkv, N)
    w = torch.where((slot < c["sink"]) | (slot >= n - c["recent"]),
                    torch.full_like(st["w"], math.inf), st["w"])
    w = torch.where(slot < n, w, torch.full_like(w, -math.inf))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    order = torch.sort(order, dim=-1).values          # kept slots, ascending
    live = order < n                                  # rows behind a short sequence stay zero

    def take(x):
        at = order.reshape(*order.shape, *[1] * (x.dim() - 3))
        got = torch.gather(x, 2, at.expand(*order.shape, *x.shape[3:]))
        return torch.where(live.reshape(at.shape), got, torch.zeros_like(got))

    got = [take(x) for x in st["cache"]]
    k = _decode(got[0], got[1], KMUL).transpose(1, 2).bfloat16()
    v = _decode(got[2], got[3], VMUL).transpose(1, 2).bfloat16()
    return dict(K=k, V=v, w=take(st["w"]), kpos=take(st["kpos"]),
                len=torch.clamp(st["len"], max=keep))


def _plain_store(st):
    c = st["case"]
    out = []
    r = torch.arange(c["R"], device=st["K"].device)
    hit = torch.ones(c["B"], c["R"], dtype=torch.bool, device=r.device)
    if st["rows"] is not None:
        hit = ((st["rows"][:, :, None] == r) & (r[:, None] < st["cnt"][:, None, None])).any(1)
    at = (st["off"][:, None] + r).long()
    b = torch.arange(c["B"], device=r.device)[:, None].expand_as(at)
    for x, code, scale, mul in ((st["K"], *st["cache"][:2], KMUL), (st["V"], *st["cache"][2:], VMUL)):
        c4, s8 = _encode(x.float(), mul)
        code.transpose(1, 2)[b[hit], at[hit]] = c4[hit]
        scale.transpose(1, 2)[b[hit], at[hit]] = s8[hit]
        back = _decode(code.transpose(1, 2)[b, at], scale.transpose(1, 2)[b, at], mul)
        out.append(torch.where(hit[..., None, None], back, torch.zeros_like(back)).to(x.dtype))
    return out[0], out[1]


# ------------------------------------------------------------------- one pass
def _own(st):
    from drift_aware_kv_spherical_gb300 import polestar as ps
    c = st["case"]
    if "handle" not in st:       # what a user's program keeps beside its buffers
        st["handle"] = ps.Kv4Cache(*st["cache"], kmul=KMUL, vmul=VMUL)
        if c["op"] == "evict":
            st["dst_handle"] = ps.Kv4Cache(*st["dst"], kmul=KMUL, vmul=VMUL)
            st["ws"] = ps.workspace(ps.OP_KV4_EVICT, B=c["B"], N=c["N"], Hkv=c["Hkv"], k=c["keep"])
        elif c["op"] in ("attn", "weight"):
            op = ps.OP_KV4_ATTN if c["op"] == "attn" else ps.OP_KV4_WEIGHT
            st["ws"] = ps.workspace(op, B=c["B"], N=c["N"], Hq=c["Hq"], Hkv=c["Hkv"],
                                    dh=c["dh"], P=c["T"])
    h = st["handle"]
    if c["op"] == "store":
        ps.ps_kv4_store(h, st["K"], st["V"], off=st["off"], rows=st["rows"], cnt=st["cnt"])
        ps.ps_kv4_load(h, st["K_back"], st["V_back"], off=st["off"], rows=st["rows"],
                       cnt=st["cnt"])
        return st["K_back"], st["V_back"]
    if c["op"] == "evict":
        d = st["dst_handle"]
        ps.ps_kv4_evict(h, d, st["w"], st["w_dst"], st["len_dst"], c["keep"], sink=c["sink"],
                        recent=c["recent"], len=st["len"], kpos=st["kpos"],
                        kpos_dst=st["kpos_dst"], ws=st["ws"])
        ps.ps_kv4_load(d, st["K_back"], st["V_back"])
        return dict(K=st["K_back"], V=st["V_back"], w=st["w_dst"], kpos=st["kpos_dst"],
                    len=st["len_dst"])
    opt = dict(len=st["len"], span=st["span"], qpos=st["qpos"], slope=st["slope"],
               scale=st["scale"], cap=c["cap"], ws=st["ws"])
    if c["op"] == "attn":
        ps.ps_kv4_attn(h, st["Q"], st["O"], st["lse"], **opt)
        return st["O"], st["lse"]
    ps.ps_kv4_weight(h, st["Q"], st["lse"], st["w"], st["w_out"], **opt)
    return st["w_out"]


def run(state):
    if own:
        return _own(state)
    return dict(attn=_plain_attn, weight=_plain_weight, evict=_plain_evict,
                store=_plain_store)[state["case"]["op"]](state)


# ------------------------------------------------------------------- needed work
def work(case):
    """Bytes and operations of one pass.  Ragged lengths count 3/4 of the slots
    (their mean), spans the share of the score matrix that they leave on average."""
    B, Hkv, dh, N, op = case["B"], case["Hkv"], case["dh"], case["N"], case["op"]
    row = 2 * (dh // 2 + dh // 16)                     # K and V of one slot and head
    esz = 4 if case.get("dtype") == "f32" else 2
    live = N * (0.75 if case.get("ragged") else 1.0)
    if op == "store":
        rows = B * case["R"] * Hkv * (0.175 if case["listed"] else 1.0)
        # rows read, cache written, cache read, rows written
        return dict(bytes=rows * (2 * 2 * dh * esz + 2 * row), flops=0)
    if op == "evict":
        kept = B * Hkv * min(case["keep"], live)
        return dict(bytes=B * Hkv * live * 4 + kept * (2 * row + 3 * 4 + row + 2 * dh * 2), flops=0)
    T, Hq = case["T"], case["Hq"]
    q = B * T * Hq * (dh * esz + 4)
    share = 1.0
    if case["span"] == "documents":
        share = min(1.0, 2.0 / max(1, N // 256))
    elif case["span"] in ("causal", "prefix"):
        share = max(0.5, 1.0 - T / (2.0 * live))
    seen = min(live, share * live + T) if case["span"] == "documents" else live
    if op == "attn":
        return dict(bytes=B * Hkv * seen * row + q + B * T * Hq * dh * esz,
                    flops=4.0 * B * T * Hq * dh * live * share)
    return dict(bytes=B * Hkv * (seen * row / 2 + 8.0 * N) + q,
                flops=2.0 * B * T * Hq * dh * live * share)


# ------------------------------------------------------------------- 64 bits
def _pow2(e):
    """2 ** e, exactly, of whole e in [-32, 32]."""
    t = torch.tensor([2.0 ** k for k in range(-32, 33)], dtype=torch.float64, device=e.device)
    return t[e.long() + 32]


def _values64(code, scale, mul):
    """f64 values of a packed cache part, from the bit fields."""
    lo, hi = (code & 15).long(), (code >> 4).long()
    n = torch.stack((lo, hi), -1).flatten(-2)
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e == 0, 0.5 * m, _pow2(e - 1) * (1.0 + 0.5 * m))
    v = torch.where(n >= 8, -mag, mag)
    s = scale.long()
    se, sm = (s >> 3) & 15, (s & 7).double()
    sv = torch.where(se == 0, sm / 512.0, _pow2(se - 7) * (1.0 + sm / 8.0))
    return v * sv.repeat_interleave(16, -1) * mul


def _quantised64(x, mul):
    """The values that rows x (f64) have once stored: each block's scale and
    element rounded to the nearest E4M3 / E2M1 value, ties to even."""
    x = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    a = x.abs().amax(-1, keepdim=True) / (6.0 * mul)
    ulp = _pow2(torch.frexp(a.clamp(min=2.0 ** -6, max=2.0 ** 20)).exponent - 4)
    s = torch.round(a / ulp).mul(ulp).clamp(max=448.0)
    g = s * mul
    y = torch.where(g > 0, x / torch.where(g > 0, g, torch.ones_like(g)), torch.zeros_like(x))
    ay = y.abs()
    step = torch.where(ay < 2.0, 0.5, torch.where(ay < 4.0, 1.0, 2.0))
    q = torch.minimum(torch.round(ay / step) * step, torch.full_like(ay, 6.0))
    return (torch.sign(y) * q * g).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    B, Hkv, dh, N, op = case["B"], case["Hkv"], case["dh"], case["N"], case["op"]
    if op == "store":
        out = []
        for x, mul in ((st["K"], KMUL), (st["V"], VMUL)):
            y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
            for b in range(B):
                if st["rows"] is None:
                    y[b] = _quantised64(x[b].double(), mul)
                else:
                    r = st["rows"][b, :int(st["cnt"][b])].long()
                    y[b, r] = _quantised64(x[b, r].double(), mul)
            out.append(y)
        return tuple(out)
    if op == "evict":
        keep, sink, recent = case["keep"], case["sink"], case["recent"]
        dev = st["w"].device
        k = torch.zeros(B, keep, Hkv, dh, dtype=torch.float64, device=dev)
        v, w = torch.zeros_like(k), torch.zeros(B, Hkv, keep, dtype=torch.float64, device=dev)
        pos = torch.zeros(B, Hkv, keep, dtype=torch.int32, device=dev)
        wn = st["w"].cpu().numpy().astype(np.float64)
        lens = st["len"].cpu().numpy()
        for b in range(B):
            n = int(lens[b])
            mid = np.arange(sink, max(sink, n - recent))
            for h in range(Hkv):
                best = mid[np.lexsort((mid, -wn[b, h, mid]))][:keep - sink - recent]
                at = np.sort(np.concatenate([np.arange(sink), best, np.arange(n - recent, n)]))
                t = torch.from_numpy(at if n > keep else np.arange(n)).to(dev)
                part = [x[b, h, t] for x in st["cache"]]
                k[b, :len(t), h] = _values64(part[0], part[1], KMUL)
                v[b, :len(t), h] = _values64(part[2], part[3], VMUL)
                w[b, h, :len(t)], pos[b, h, :len(t)] = st["w"][b, h, t].double(), st["kpos"][b, h, t]
        return dict(K=k, V=v, w=w, kpos=pos, len=torch.from_numpy(np.minimum(lens, keep)))
    T, Hq = case["T"], case["Hq"]
    G = Hq // Hkv
    if 4.0 * B * T * Hq * N * dh > 6e11:
        return None
    dev = st["Q"].device
    pos = torch.arange(N, device=dev)
    O = torch.zeros(B, T, Hq, dh, dtype=torch.float64, device=dev)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=dev)
    wout = st["w"].double() if op == "weight" else None
    for b in range(B):
        n = int(st["len"][b])
        see = (pos < n).expand(T, N)
        if st["span"] is not None:
            see = see & (pos >= st["span"][b, :, :1]) & (pos < st["span"][b, :, 1:])
        any_ = see.any(1)
        for h in range(Hq):
            kv = h // G
            k64 = _values64(st["cache"][0][b, kv], st["cache"][1][b, kv], KMUL)
            s = (st["Q"][b, :, h].double() @ k64.T) * st["scale"]
            if case["cap"] > 0:
                s = case["cap"] * torch.tanh(s / case["cap"])
            if case["bias"]:
                s = s - st["slope"][h].double() * (st["qpos"][b][:, None] - pos).abs().double()
            s = torch.where(see, s, torch.full_like(s, -math.inf))
            if op == "weight":
                p = torch.exp(s - st["lse"][b, :, h, None].double())
                wout[b, kv] += torch.where(any_[:, None], p, torch.zeros_like(p)).sum(0)
                continue
            l = torch.logsumexp(s, 1)
            p = torch.where(any_[:, None], torch.exp(s - l[:, None]), torch.zeros_like(s))
            lse[b, :, h] = l
            O[b, :, h] = p @ _values64(st["cache"][2][b, kv], st["cache"][3][b, kv], VMUL)
    return wout if op == "weight" else (O, lse)
