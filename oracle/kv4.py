"""The 4-bit KV cache (oracle): rows in and out, attention over it, the weight
that attention puts on its slots, eviction by that weight.

[Polestar §2.A, sparse updates] keeps a KV cache; holding it in NVFP4 and
evicting from it are additions of this library with no counterpart on the page.
The definitions are include/polestar.h's.  Storing is defined in fp32 (one IEEE
rounding a step), as in ``nvfp4``; everything else is fp64 on the stored values.
"""

import numpy as np

from .nvfp4 import e2m1_decode, e2m1_encode, e4m3_decode, e4m3_encode

_F32 = np.float32


def kv4_encode(X, S):
    """Rows X [..., dh] (fp32) with the tensor scale S: codes [..., dh/2] and
    scales [..., dh/16] (uint8)."""
    X = np.asarray(X, _F32)
    blk = X.reshape(*X.shape[:-1], X.shape[-1] // 16, 16)
    S = _F32(S)
    amax = np.max(np.where(np.isnan(blk), _F32(0), np.abs(blk)), axis=-1)
    with np.errstate(over="ignore"):
        sc = e4m3_encode((amax / _F32(_F32(6.0) * S)).astype(_F32))
    den = (e4m3_decode(sc).astype(_F32) * S).astype(_F32)[..., None]
    live = den > 0
    ratio = (blk / np.where(live, den, _F32(1))).astype(_F32)
    q = np.where(live, e2m1_encode(np.where(np.isnan(ratio), _F32(6), ratio)), 0)
    q = q.reshape(X.shape)
    return (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8), sc.astype(np.uint8)


def kv4_decode(codes, scales, S):
    """Values code * scale * S (fp64; S as fp32) [..., dh]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    s = np.repeat(e4m3_decode(scales), 16, axis=-1)
    return e2m1_decode(c) * s * float(_F32(S))


def kv4_scores(Q, K, scale, length=None, span=None, kpos=None, qpos=None, slope=None, cap=0.0):
    """Scores [B][T][Hq][N] (fp64, -inf where the row does not see the slot) of
    Q [B][T][Hq][dh] against K [B][Hkv][N][dh]."""
    B, T, Hq, _ = Q.shape
    Hkv, N = K.shape[1], K.shape[2]
    G = Hq // Hkv
    pos = np.broadcast_to(np.arange(N), (B, Hkv, N)) if kpos is None else np.asarray(kpos)
    s = np.empty((B, T, Hq, N))
    for b in range(B):
        n = N if length is None else int(length[b])
        for h in range(Hq):
            g = h // G
            x = scale * (Q[b, :, h].astype(np.float64) @ K[b, g].T)
            if cap > 0:
                x = cap * np.tanh(x / cap)
            if slope is not None:
                x = x - float(slope[h]) * np.abs(qpos[b][:, None] - pos[b, g][None, :])
            see = np.broadcast_to(np.arange(N) < n, (T, N))
            if span is not None:
                see = see & (pos[b, g] >= span[b, :, :1]) & (pos[b, g] < span[b, :, 1:])
            s[b, :, h] = np.where(see, x, -np.inf)
    return s


def kv4_attention(s, V):
    """(O [B][T][Hq][dh], lse [B][T][Hq]) of scores s and V [B][Hkv][N][dh]; a
    row that sees nothing gives 0 and -inf."""
    B, T, Hq, N = s.shape
    G = Hq // V.shape[1]
    m = s.max(-1, keepdims=True)
    base = np.where(np.isfinite(m), m, 0.0)
    p = np.exp(s - base)
    l = p.sum(-1, keepdims=True)
    O = np.einsum("bthn,bhnd->bthd", p, np.repeat(V, G, axis=1)) / np.where(l > 0, l, 1.0)
    with np.errstate(divide="ignore"):
        return O, (np.log(l) + base)[..., 0]


def kv4_weight(s, lse, Hkv):
    """Weight [B][Hkv][N] that the rows put on each slot: the sum over tokens
    and the KV head's query heads of exp(s - lse)."""
    B, T, Hq, N = s.shape
    lse = np.asarray(lse, np.float64)[..., None]
    p = np.where(np.isfinite(s) & np.isfinite(lse), np.exp(s - np.where(np.isfinite(lse), lse, 0)),
                 0.0)
    return p.reshape(B, T, Hkv, Hq // Hkv, N).sum(axis=(1, 3))


def kv4_keep(w, n, keep, sink, recent):
    """Ascending slots kept of one head's n live ones, by weights w."""
    if n <= keep:
        return np.arange(n)
    key = np.where(np.isnan(w[:n]), -np.inf, w[:n].astype(np.float64))
    rank = np.where(np.isnan(w[:n]), 1, 0)      # NaN below -inf
    mid = np.arange(sink, n - recent)
    order = mid[np.lexsort((mid, rank[mid], -key[mid]))]
    return np.sort(np.concatenate([np.arange(sink), order[:keep - sink - recent],
                                   np.arange(n - recent, n)]))
