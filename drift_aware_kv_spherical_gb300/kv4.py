"""A layer's 4-bit KV cache as a decoder keeps it: the packed buffers, how far
each sequence has filled them, what position each slot holds, and the attention
weight its slots have drawn.

All arithmetic is in the ps_kv4_* calls (include/polestar.h); this class owns
their buffers and passes them on.  Until the first eviction slot n holds position
n; afterwards `kpos` says which, for every KV head.  The slots behind the kept
ones are those of the positions that come next, and have drawn no weight.
"""

import contextlib
import functools

import torch

from . import polestar as ps


def _on(stream, device):
    """Torch's work on `stream` (a torch stream, a raw one, None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(stream, device)
    return torch.cuda.stream(stream)


@functools.lru_cache(maxsize=256)
def _ws_bytes(op, **sizes):
    return ps.ps_workspace_bytes(op, **sizes)


class Kv4Layer:
    """B sequences, Hkv KV heads of dh, up to N slots each; Hq query heads."""

    def __init__(self, B, N, Hq, Hkv, dh, kmul=1.0, vmul=1.0, device="cuda"):
        self.Hq = Hq
        self.cache = ps.Kv4Cache.empty(B, Hkv, N, dh, kmul, vmul, device)
        self.len = torch.zeros(B, dtype=torch.int32, device=device)
        self.w = torch.zeros(B, Hkv, N, dtype=torch.float32, device=device)
        self.kpos = None
        self._note_len(0)
        self._shift = None      # [B]: position of a slot behind the kept ones, less the slot
        self._spare = None
        self._ws = {}

    def _workspace(self, op, stream, **sizes):
        """The scratch of a call on `stream`: its own, allocated there, at the next
        power of two of bytes.  So calls of many lengths share a few buffers (at most
        four times the largest call's bytes in all), and none that a captured graph
        uses is ever given back."""
        c = self.cache
        n = _ws_bytes(op, B=c.B, N=c.N, Hq=self.Hq, Hkv=c.Hkv, dh=c.dh, **sizes)
        if n == 0:
            return None
        key = (ps.raw_stream(stream, c.device), n.bit_length())
        if key not in self._ws:
            with _on(stream, c.device):
                self._ws[key] = torch.empty(1 << n.bit_length(), dtype=torch.uint8,
                                            device=c.device)
        return self._ws[key]

    def store(self, K, V, off=None, rows=None, cnt=None, stream=None):
        """Rows of K and V [B][R][Hkv][dh] as positions off[b] + r (see
        ps.ps_kv4_store); `len` is the caller's to set.  Before the first eviction
        a position is its slot.  After it every KV head takes the row into the slot
        that holds the position, and skips a position that it has evicted."""
        ps.ps_kv4_store(self.cache, K, V, off=off, rows=rows, cnt=cnt, kpos=self.kpos,
                        stream=stream)

    def addresses(self):
        """Where a captured store reads and writes: a graph of it holds while these
        stay as they are."""
        return tuple(t.data_ptr() for t in (*self.cache.buffers, self.kpos) if t is not None)

    def append(self, K, V):
        """K and V of the next T tokens of every sequence, behind what is there:
        slots len[b], len[b] + 1, ..., which hold the positions that come next
        after an eviction too.  Refused where some sequence has no room for them
        (a captured call cannot know at its replays: past the capacity they store
        nothing, and `len` must not be let grow that far)."""
        T = K.shape[1]
        if self._capturing():
            self._len_seen = False      # from now on `len` changes at replays too
        elif (top := self._filled()) + T > self.cache.N:
            raise ValueError(f"no room for {T} more tokens: {top} of {self.cache.N} slots "
                             "are filled")
        ps.ps_kv4_store(self.cache, K, V, off=self.len)
        known = self._known()
        self.len += T
        if known:
            self._note_len(self._top + T)

    def _capturing(self):
        return self.len.is_cuda and torch.cuda.is_current_stream_capturing()

    # Slots of the fullest sequence (`_top`): known on the host from one append or
    # eviction to the next, read back only after the caller has changed `len`.
    def _note_len(self, top):
        self._top, self._len_seen = top, (self.len, self.len._version)

    def _known(self):
        seen = self._len_seen
        return bool(seen) and seen[0] is self.len and seen[1] == self.len._version

    def _filled(self):
        if not self._known():
            top = max(self.len.tolist(), default=0)
            if self._len_seen is False:
                return top
            self._note_len(top)
        return self._top

    def attend(self, Q, O, lse=None, *, scale=None, stream=None, **see):
        """Attention of Q [B][T][Hq][dh] over the cache into O; `see`: span,
        qpos, slope, cap as in ps.ps_kv4_attn."""
        scale = self.cache.dh ** -0.5 if scale is None else scale
        ps.ps_kv4_attn(self.cache, Q, O, lse, scale=scale, len=self.len, kpos=self.kpos,
                       ws=self._workspace(ps.OP_KV4_ATTN, stream, P=Q.shape[1]),
                       stream=stream, **see)

    def weigh(self, Q, lse, *, scale=None, stream=None, **see):
        """Adds the weight that Q's rows put on every slot to `w`; lse as attend
        wrote it for the same arguments."""
        scale = self.cache.dh ** -0.5 if scale is None else scale
        ps.ps_kv4_weight(self.cache, Q, lse, self.w, self.w, scale=scale, len=self.len,
                         kpos=self.kpos, ws=self._workspace(ps.OP_KV4_WEIGHT, stream, P=Q.shape[1]),
                         stream=stream, **see)

    def evict(self, keep, sink=0, recent=0, spare=None, stream=None):
        """Cuts every sequence to `keep` slots: the first `sink`, the last
        `recent`, the heaviest of the others.  The kept slots move to `spare`,
        the buffers that an earlier eviction of a layer of this shape left
        behind (not given: this layer's own ones, made on the first call), and
        the old ones are returned as the next call's spare.  Layers of one shape
        can pass one spare on, round after round:

            for layer in layers:
                spare = layer.evict(keep, spare=spare)

        A spare serves one eviction, which empties it.  Everything runs on
        `stream`, behind what the spare's last owner enqueued on its own."""
        with _on(stream, self.cache.device):
            return self._evict(keep, sink, recent, spare, stream)

    def _evict(self, keep, sink, recent, spare, stream):
        c = self.cache
        i32 = dict(dtype=torch.int32, device=c.device)
        if spare is None:
            spare = self._spare     # empty once another layer has taken it
            if not spare:
                spare = dict(
                    cache=ps.Kv4Cache.empty(c.B, c.Hkv, c.N, c.dh, c.kmul, c.vmul, c.device),
                    w=torch.empty_like(self.w), kpos=torch.empty(c.B, c.Hkv, c.N, **i32),
                    len=torch.empty(c.B, **i32), shift=torch.empty(c.B, **i32))
        elif not spare:
            raise ValueError("an eviction has taken this spare already")
        here = torch.cuda.current_stream(c.device) if c.device.type == "cuda" else None
        if spare.get("stream", here) != here and not torch.cuda.is_current_stream_capturing():
            here.wait_stream(spare["stream"])   # (a capture begins behind everything)
        ps.ps_kv4_evict(c, spare["cache"], self.w, spare["w"], spare["len"], keep, sink=sink,
                        recent=recent, len=self.len, kpos=self.kpos, kpos_dst=spare["kpos"],
                        shift=self._shift, shift_dst=spare["shift"],
                        ws=self._workspace(ps.OP_KV4_EVICT, stream, k=keep), stream=stream)
        kpos, shift = self.kpos, self._shift
        if kpos is None:
            kpos, shift = torch.empty(c.B, c.Hkv, c.N, **i32), torch.empty(c.B, **i32)
        if self._capturing():
            self._len_seen = False
        known = self._known()
        # the one reference to the old buffers that a later eviction, this
        # layer's or another's, may write through: whoever takes them empties it
        self._spare = dict(cache=c, w=self.w, kpos=kpos, len=self.len, shift=shift, stream=here)
        if here is not None:    # they may have been allocated on another stream, and may be freed
            for t in (*c.buffers, self.w, kpos, self.len, shift):
                t.record_stream(here)
        self.cache, self.w, self.kpos, self.len, self._shift = (
            spare[k] for k in ("cache", "w", "kpos", "len", "shift"))
        if known:
            self._note_len(min(self._top, keep))
        spare.clear()
        return self._spare
