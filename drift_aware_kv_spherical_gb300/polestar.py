"""Thin Python binding of libpolestar's C ABI (include/polestar.h).

Argument marshalling only: every function below forwards torch device
tensors as raw pointers to the function of the same name in libpolestar.so,
and every step of the computation runs in its CUDA kernels.  There is no CPU
path: if the library is missing or a call fails, a PolestarError is raised.
"""

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpolestar.so")

PS_OK, PS_ERR_ARG, PS_ERR_UNSUPPORTED, PS_ERR_WORKSPACE, PS_ERR_CUDA, PS_ERR_TIMEOUT = range(6)
PS_F32, PS_BF16 = 0, 1
(OP_KMEANS, OP_NVFP4, OP_PROXY_KL, OP_TOPK, OP_REFRESH, OP_COMMIT, OP_KV4_ATTN,
 OP_KV4_WEIGHT, OP_KV4_EVICT, OP_ATTN) = range(10)
EXPORTED = ["ps_create", "ps_destroy", "ps_check", "ps_status_string", "ps_last_cuda_error",
            "ps_trace_enable", "ps_trace_count", "ps_trace_get",
            "ps_workspace_bytes", "ps_kmeans_spherical", "ps_nvfp4_residual",
            "ps_proxy_attn_kl", "ps_topk_drift", "ps_refresh_kv", "ps_commit",
            "ps_store_record_bytes", "ps_host_alloc", "ps_host_free",
            "ps_nvfp4_pack_clusters", "ps_nvfp4_fetch_dequant", "ps_schedule_step", "ps_drift_score",
            "ps_block_progress", "ps_kv4_store", "ps_kv4_load", "ps_kv4_attn",
            "ps_kv4_weight", "ps_kv4_evict", "ps_kv4_store_pos", "ps_kv4_evict_on",
            "ps_rope_turns", "ps_rope", "ps_attn", "ps_sample", "ps_commit_drawn"]

_p = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t
_i64 = ctypes.c_int64


class PolestarError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        lib = Library.load()
        msg = f"{where}: {lib.status_string(status)} ({status})"
        if status == PS_ERR_CUDA:
            msg += f" [{lib.cdll.ps_last_cuda_error().decode()}]"
        super().__init__(msg)


class CommitParams(ctypes.Structure):
    _fields_ = [("tau_s", ctypes.c_float), ("alpha", ctypes.c_float),
                ("ratio", ctypes.c_float), ("mode", ctypes.c_int),
                ("ensure_progress", ctypes.c_int)]


class ScheduleParams(ctypes.Structure):
    _fields_ = [("tau_upd", ctypes.c_int), ("full_period", ctypes.c_int),
                ("block_len", ctypes.c_int)]


class ScheduleState(ctypes.Structure):
    _fields_ = [("since", ctypes.c_int), ("refreshes", ctypes.c_int),
                ("block_start", ctypes.c_int)]


class RopeParams(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int), ("scaling", ctypes.c_int)] + \
               [(n, ctypes.c_double) for n in ("base", "factor", "low", "high", "orig_len")]


ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}

SCHED_REFRESH, SCHED_FULL, SCHED_SLIDE, SCHED_REINIT = 1, 2, 4, 8
SCORER_KL, SCORER_COSINE, SCORER_ENTROPY = 0, 1, 2

_SIGS = {
    "ps_create": (_i, [_i, ctypes.POINTER(_p)]),
    "ps_destroy": (_i, [_p]),
    "ps_check": (_i, [_p, _p, _i]),
    "ps_status_string": (ctypes.c_char_p, [_i]),
    "ps_last_cuda_error": (ctypes.c_char_p, []),
    "ps_trace_enable": (_i, [_p, _i]),
    "ps_trace_count": (_i, [_p]),
    "ps_trace_get": (_i, [_p, _i, ctypes.POINTER(ctypes.c_char_p),
                          ctypes.POINTER(ctypes.c_float)]),
    "ps_workspace_bytes": (_sz, [_i] * 11),
    "ps_store_record_bytes": (_sz, [_i]),
    "ps_host_alloc": (_i, [_sz, ctypes.POINTER(_p)]),
    "ps_host_free": (_i, [_p]),
    "ps_drift_score": (_i, [_p, _p, _p, _i, _i, _i, _i, _p, _p]),
    "ps_block_progress": (_i, [_p, _p, _p, _p, _i, _i, _p, _p]),
    "ps_schedule_step": (_i, [ctypes.POINTER(ScheduleParams), ctypes.POINTER(ScheduleState),
                              _i, _i]),
    "ps_nvfp4_pack_clusters": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _p, _p, _p, _p]),
    "ps_nvfp4_fetch_dequant": (_i, [_p, _p, _p, _p, _p, _i, _p, _p, _p, _i, _i, _i, _i, _p,
                                    _p]),
    "ps_kmeans_spherical": (_i, [_p, _p, _i, _i, _i, _i, _i, _i, _i, _p, _p, _p,
                                 _p, _p, _p, _p, _p, _sz, _p]),
    "ps_nvfp4_residual": (_i, [_p, _p, _i, _p, _p, _p, _i, _i, _i, _i, _p, _p, _p,
                               _p, _sz, _p]),
    "ps_proxy_attn_kl": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _p,
                              _p, _p, _p, _sz, _p]),
    "ps_topk_drift": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _p, _p, _p, _p, _p, _p,
                           _sz, _p]),
    "ps_refresh_kv": (_i, [_p, _p, _i, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p, _p,
                           _i, _i, _p, _sz, _p]),
    "ps_commit": (_i, [_p, _p, _i, _i, _i, _i, _p, _p, _p, _i, _p, _p, _p, _p, _i,
                       CommitParams, _p, _p, _p, _p, _sz, _p]),
    "ps_kv4_store": (_i, [_p, _p, _p, _p, _i, _i, _i64, _i64, _p, _p, _p, _p]),
    "ps_kv4_store_pos": (_i, [_p, _p, _p, _p, _i, _i, _i64, _i64, _p, _p, _p, _p, _p]),
    "ps_kv4_load": (_i, [_p, _p, _p, _p, _i, _i, _i64, _i64, _p, _p, _p, _p]),
    "ps_kv4_attn": (_i, [_p, _p, _p, _p, _p, _p, _sz, _p]),
    "ps_kv4_weight": (_i, [_p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "ps_kv4_evict": (_i, [_p, _p, _p, _p, _p, _p, _i, _i, _i, _p, _p, _p, _p, _sz, _p]),
    "ps_rope_turns": (_i, [ctypes.POINTER(RopeParams), _p]),
    "ps_rope": (_i, [_p, _p, _p, _i, _p]),
    "ps_attn": (_i, [_p, _p, _p, _p, _p, _sz, _p]),
    "ps_sample": (_i, [_p, _p, _p, _p, _p, _p]),
    "ps_commit_drawn": (_i, [_p, _p, _i, _i, _p, _p, _p, _i, _p, _p, _p, _p, _i, CommitParams,
                             _p, _p]),
    "ps_kv4_evict_on": (_i, [_p, _p, _p, _p, _p, _p, _i, _i, _i, _p, _p, _p, _p, _p, _p, _sz, _p]),
}


class Library:
    """The loaded libpolestar.so (one per process)."""

    _inst = None

    def __init__(self, path):
        self.cdll = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(self.cdll, name)
            fn.restype = res
            fn.argtypes = args
        self.path = path
        self._handles = {}

    @classmethod
    def load(cls, path=None):
        if cls._inst is None:
            path = path or LIB_PATH
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is not built; run `python -c 'import __graft_entry__ as g; "
                    "g.build()'` (libpolestar has no CPU fallback)")
            cls._inst = cls(path)
        return cls._inst

    def status_string(self, s):
        return self.cdll.ps_status_string(s).decode()

    def handle(self, device=None):
        """A process-wide handle for `device` (created on first use)."""
        dev = torch.cuda.current_device() if device is None else device
        if dev not in self._handles:
            dev = int(dev)
            h = _p()
            st = self.cdll.ps_create(dev, ctypes.byref(h))
            if st != PS_OK:
                raise PolestarError(st, "ps_create")
            self._handles[dev] = h
        return self._handles[dev]


def _lib():
    return Library.load()


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libpolestar takes device tensors only")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _dtype(t):
    if t.dtype == torch.float32:
        return PS_F32
    if t.dtype == torch.bfloat16:
        return PS_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


def _check(st, where):
    if st != PS_OK:
        raise PolestarError(st, where)


def _ws(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)


def ps_workspace_bytes(op, B=0, N=0, d=0, C=0, Hq=0, Hkv=0, dh=0, k=0, P=0, V=0):
    return int(_lib().cdll.ps_workspace_bytes(op, B, N, d, C, Hq, Hkv, dh, k, P, V))


def workspace(op, device=None, **sizes):
    """A caller-owned workspace tensor large enough for `op` at `sizes`."""
    n = ps_workspace_bytes(op, **sizes)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def ps_check(synchronize=True, stream=None):
    lib = _lib()
    _check(lib.cdll.ps_check(lib.handle(), _stream(stream), int(synchronize)), "ps_check")


def ps_kmeans_spherical(H, mu, assign, rho, chat, counts, iters, init_mode=0,
                        init_u=None, objective=None, ws=None, stream=None):
    lib = _lib()
    B, N, d = H.shape
    C = mu.shape[1]
    w, wn = _ws(ws)
    st = lib.cdll.ps_kmeans_spherical(
        lib.handle(), _ptr(H), _dtype(H), B, N, d, C, iters, init_mode,
        _ptr(init_u), _ptr(mu), _ptr(assign), _ptr(rho), _ptr(chat), _ptr(counts),
        _ptr(objective), w, wn, _stream(stream))
    _check(st, "ps_kmeans_spherical")


def ps_nvfp4_residual(H, mu, assign, rho, codes, scales, tensor_scale, ws=None,
                      stream=None):
    lib = _lib()
    B, N, d = H.shape
    C = mu.shape[1] if mu is not None else 1
    w, wn = _ws(ws)
    st = lib.cdll.ps_nvfp4_residual(
        lib.handle(), _ptr(H), _dtype(H), _ptr(mu), _ptr(assign), _ptr(rho), B, N,
        d, C, _ptr(codes), _ptr(scales), _ptr(tensor_scale), w, wn, _stream(stream))
    _check(st, "ps_nvfp4_residual")


def ps_proxy_attn_kl(Q, chat, Wk, A_prev, A_cur, D, Hkv, ws=None, stream=None):
    lib = _lib()
    B, N, Hq, dh = Q.shape
    C, d = chat.shape[1], chat.shape[2]
    w, wn = _ws(ws)
    st = lib.cdll.ps_proxy_attn_kl(
        lib.handle(), _ptr(Q), _ptr(chat), _ptr(Wk), _dtype(Q), B, N, d, C, Hq, Hkv,
        dh, _ptr(A_prev), _ptr(A_cur), _ptr(D), w, wn, _stream(stream))
    _check(st, "ps_proxy_attn_kl")


def ps_topk_drift(D, assign, counts, k, sel, sel_score, pos, npos, posmask=None,
                  ws=None, stream=None):
    lib = _lib()
    B, N = D.shape
    C = counts.shape[1]
    w, wn = _ws(ws)
    st = lib.cdll.ps_topk_drift(
        lib.handle(), _ptr(D), _ptr(assign), _ptr(counts), B, N, C, k, _ptr(sel),
        _ptr(sel_score), _ptr(pos), _ptr(npos), _ptr(posmask), w, wn, _stream(stream))
    _check(st, "ps_topk_drift")


def ps_refresh_kv(H, pos, npos, Wk, Wv, Kcache, Vcache, Hkv, dh, cache_off=0,
                  ws=None, stream=None):
    lib = _lib()
    B, N, d = H.shape
    Ncache = Kcache.shape[1]
    w, wn = _ws(ws)
    st = lib.cdll.ps_refresh_kv(
        lib.handle(), _ptr(H), _dtype(H), _ptr(pos), _ptr(npos), _ptr(Wk), _ptr(Wv),
        B, N, d, Hkv, dh, _ptr(Kcache), _ptr(Vcache), Ncache, cache_off, w, wn,
        _stream(stream))
    _check(st, "ps_refresh_kv")


def ps_commit(logits, role, undecided, D_blk, d_ld, d_sum, d_cnt, d_prev,
              suffix_sel, sel_ld, params, token, conf, commit, ws=None,
              stream=None):
    lib = _lib()
    B, P, V = logits.shape
    w, wn = _ws(ws)
    if not isinstance(params, CommitParams):
        params = CommitParams(*params)
    st = lib.cdll.ps_commit(
        lib.handle(), _ptr(logits), _dtype(logits), B, P, V, _ptr(role), _ptr(undecided), _ptr(D_blk),
        d_ld, _ptr(d_sum), _ptr(d_cnt), _ptr(d_prev), _ptr(suffix_sel), sel_ld, params,
        _ptr(token), _ptr(conf), _ptr(commit), w, wn, _stream(stream))
    _check(st, "ps_commit")


def ps_drift_score(A_cur, A_prev, scorer, D, stream=None):
    """Ablation drift signal (SCORER_*) of distributions A_cur [B][N][C]
    against A_prev (or None) into D [B][N]."""
    lib = _lib()
    B, N, C = A_cur.shape
    st = lib.cdll.ps_drift_score(lib.handle(), _ptr(A_cur), _ptr(A_prev), B, N, C, int(scorer),
                                 _ptr(D), _stream(stream))
    _check(st, "ps_drift_score")


def ps_nvfp4_residual_noalloc(H, mu, assign, rho, codes, scales, tensor_scale,
                              stream=None):
    """ps_nvfp4_residual without a workspace: for callers that cannot
    allocate device memory; the library's fixed device array holds the
    scratch (B <= 16384; overlapping calls on one device race)."""
    lib = _lib()
    fn = lib.cdll.ps_nvfp4_residual_noalloc
    fn.restype = _i
    fn.argtypes = [_p, _p, _i, _p, _p, _p, _i, _i, _i, _i, _p, _p, _p, _p]
    B, N, d = H.shape
    C = mu.shape[1] if mu is not None else 1
    st = fn(lib.handle(), _ptr(H), _dtype(H), _ptr(mu), _ptr(assign), _ptr(rho), B, N,
            d, C, _ptr(codes), _ptr(scales), _ptr(tensor_scale), _stream(stream))
    _check(st, "ps_nvfp4_residual_noalloc")


def ps_trace_enable(enable=True):
    """Start (clearing earlier records) or stop the library's kernel trace."""
    lib = _lib()
    _check(lib.cdll.ps_trace_enable(lib.handle(), int(bool(enable))), "ps_trace_enable")


def ps_trace_records():
    """[(kernel name, ms)] for every kernel launched since tracing was enabled,
    in launch order (waits for them to finish)."""
    lib = _lib()
    out = []
    for i in range(lib.cdll.ps_trace_count(lib.handle())):
        name = ctypes.c_char_p()
        ms = ctypes.c_float()
        _check(lib.cdll.ps_trace_get(lib.handle(), i, ctypes.byref(name), ctypes.byref(ms)),
               "ps_trace_get")
        out.append((name.value.decode(), ms.value))
    return out


# ---- offload of the quantised clusters (include/polestar.h)
def ps_store_record_bytes(d):
    return int(_lib().cdll.ps_store_record_bytes(int(d)))


class HostStore:
    """Pinned host memory mapped into the device (ps_host_alloc): `ptr` is
    valid on host and device; `view()` is a numpy byte view of it."""

    def __init__(self, nbytes):
        lib = _lib()
        p = ctypes.c_void_p()
        _check(lib.cdll.ps_host_alloc(int(nbytes), ctypes.byref(p)), "ps_host_alloc")
        self.ptr, self.nbytes = p.value, int(nbytes)

    def view(self):
        import numpy as np
        buf = (ctypes.c_uint8 * self.nbytes).from_address(self.ptr)
        return np.frombuffer(buf, dtype=np.uint8)

    def free(self):
        if self.ptr:
            _check(_lib().cdll.ps_host_free(ctypes.c_void_p(self.ptr)), "ps_host_free")
            self.ptr = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def _store_ptr(store):
    return store.ptr if isinstance(store, HostStore) else _ptr(store)


def ps_nvfp4_pack_clusters(codes, scales, assign, C, store, order, cl_off, stream=None):
    """Cluster-grouped records of every window into `store` (a device uint8
    tensor or a HostStore), with order [B][N] and cl_off [B][C+1] (int32)."""
    lib = _lib()
    B, N, half = codes.shape
    st = lib.cdll.ps_nvfp4_pack_clusters(lib.handle(), _ptr(codes), _ptr(scales), _ptr(assign),
                                         B, N, 2 * half, int(C), _store_ptr(store), _ptr(order),
                                         _ptr(cl_off), _stream(stream))
    _check(st, "ps_nvfp4_pack_clusters")


def ps_nvfp4_fetch_dequant(store, order, cl_off, sel, mu, rho, tensor_scale, Ht, stream=None):
    """Reconstructed rows of the selected clusters, read from `store`, into
    Ht [B][N][d] (bf16); other rows untouched."""
    lib = _lib()
    B, N, d = Ht.shape
    C = mu.shape[1]
    st = lib.cdll.ps_nvfp4_fetch_dequant(lib.handle(), _store_ptr(store), _ptr(order),
                                         _ptr(cl_off), _ptr(sel), sel.shape[1], _ptr(mu),
                                         _ptr(rho), _ptr(tensor_scale), B, N, d, C, _ptr(Ht),
                                         _stream(stream))
    _check(st, "ps_nvfp4_fetch_dequant")


def ps_block_progress(commit, undecided, role, out, stream=None):
    """(tokens committed, block decided) of a decode step into `out`: a
    HostStore of >= 8 bytes (readable on the host once `stream` has reached
    it) or an int32 device tensor of 2 elements."""
    lib = _lib()
    B, P = commit.shape
    st = lib.cdll.ps_block_progress(lib.handle(), _ptr(commit), _ptr(undecided), _ptr(role),
                                    B, P, _store_ptr(out), _stream(stream))
    _check(st, "ps_block_progress")


# ---- the 4-bit KV cache (include/polestar.h)
class Kv4Cache:
    """A layer's 4-bit KV cache over caller-owned buffers: kcode, vcode
    [B][Hkv][Ncache][dh/2] and kscale, vscale [B][Hkv][Ncache][dh/16] (uint8),
    with the tensor scales of K and V."""

    _pack = struct.Struct("4P4i2f")

    def __init__(self, kcode, kscale, vcode, vscale, kmul=1.0, vmul=1.0):
        self.B, self.Hkv, self.N, half = kcode.shape
        self.dh = 2 * half
        want = {2: (kcode, vcode), 16: (kscale, vscale)}
        for div, ts in want.items():
            for t in ts:
                _plain(t, torch.uint8, (self.B, self.Hkv, self.N, self.dh // div))
        self.buffers = (kcode, kscale, vcode, vscale)
        self.kmul, self.vmul = float(kmul), float(vmul)
        self.device = kcode.device
        self.index = self.device.index  # of the device
        self._c = self._pack.pack(*(t.data_ptr() for t in self.buffers), self.B, self.Hkv,
                                  self.N, self.dh, self.kmul, self.vmul)

    @classmethod
    def empty(cls, B, Hkv, N, dh, kmul=1.0, vmul=1.0, device="cuda"):
        """A cache over new buffers."""
        mk = [torch.zeros(B, Hkv, N, dh // q, dtype=torch.uint8, device=device)
              for q in (2, 16, 2, 16)]
        return cls(*mk, kmul=kmul, vmul=vmul)


# The current stream of a device as an integer, without building a Stream
# object (0.1 us against 3 us of a call that a decode loop makes per layer).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _kv4_stream(stream, c):
    if stream is None and _raw_stream is not None:
        return _raw_stream(c.index)
    return _stream(stream)


def raw_stream(stream, device):
    """`stream` (a torch stream, a raw one, None: the device's current one) as an
    integer; 0 where the device is not a GPU."""
    if stream is None and device.type != "cuda":
        return 0
    if stream is None and _raw_stream is not None:
        return _raw_stream(device.index)
    return _stream(stream)


def _plain(t, dtype, shape, null=False):
    """Pointer of a contiguous device tensor of this dtype and shape."""
    if t is None:
        if null:
            return 0
        raise ValueError(f"expected a {dtype} device tensor of shape {tuple(shape)}, got None")
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"expected a contiguous {dtype} device tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _rows_ld(t, B, H, dh):
    """(rows, elements between sequences, elements between rows) of t
    [B][R][H][dh], whose rows may be parts of wider ones."""
    shape = t.shape
    if len(shape) != 4:
        raise ValueError(f"expected a device tensor [{B}][rows][heads][{dh}], got {tuple(shape)}")
    b, R, h, d = shape
    if b != B or h != H or d != dh or not t.is_cuda:
        raise ValueError(f"expected a device tensor [{B}][rows][{H}][{dh}], got {tuple(shape)}")
    if t.is_contiguous():
        return R, R * H * dh, H * dh
    sb, sr, sh, sd = t.stride()
    if (sd != 1 or (sh != dh and H > 1)) and t.numel() > 0:
        raise ValueError(f"rows [{H}][{dh}] must be contiguous: strides {t.stride()}")
    return R, sb if B > 1 else 0, sr if R > 1 else H * dh


def _kv4_rows(name, c, K, V, off, rows, cnt, stream, *kpos):
    R, bld, ld = _rows_ld(K, c.B, c.Hkv, c.dh)
    if (V.dtype != K.dtype or V.shape != K.shape or not V.is_cuda or
            (V.stride() != K.stride() and _rows_ld(V, c.B, c.Hkv, c.dh) != (R, bld, ld))):
        raise ValueError("K and V need one dtype, shape and strides")
    lib = _lib()
    st = getattr(lib.cdll, name)(
        lib.handle(c.index), c._c, K.data_ptr(), V.data_ptr(), _dtype(K), R, bld, ld,
        _plain(off, torch.int32, (c.B,), True), _plain(rows, torch.int32, (c.B, R), True),
        _plain(cnt, torch.int32, (c.B,), True), *kpos, _kv4_stream(stream, c))
    _check(st, name)


def ps_kv4_store(c, K, V, off=None, rows=None, cnt=None, stream=None, kpos=None):
    """Rows of K and V [B][R][Hkv][dh] (all, or the listed ones) into slots
    off[b] + r of the cache, or with kpos [B][Hkv][Ncache], the slots' ascending
    positions, into the slot of every head that holds position off[b] + r."""
    if kpos is None:
        _kv4_rows("ps_kv4_store", c, K, V, off, rows, cnt, stream)
    else:
        _kv4_rows("ps_kv4_store_pos", c, K, V, off, rows, cnt, stream,
                  _plain(kpos, torch.int32, (c.B, c.Hkv, c.N)))


def ps_kv4_load(c, K, V, off=None, rows=None, cnt=None, stream=None):
    """The reverse of ps_kv4_store: slots off[b] + r as rows of K and V."""
    _kv4_rows("ps_kv4_load", c, K, V, off, rows, cnt, stream)


_Q_PACK = struct.Struct("6P2q3i2f")


def _kv4_query(c, Q, len, span, kpos, qpos, slope, scale, cap):
    Hq = Q.shape[2] if Q.dim() == 4 else 0
    T, bld, ld = _rows_ld(Q, c.B, Hq, c.dh)
    i32 = torch.int32
    return T, Hq, _Q_PACK.pack(
        Q.data_ptr(), _plain(len, i32, (c.B,), True), _plain(span, i32, (c.B, T, 2), True),
        _plain(kpos, i32, (c.B, c.Hkv, c.N), True), _plain(qpos, i32, (c.B, T), True),
        _plain(slope, torch.float32, (Hq,), True), bld, ld, _dtype(Q), T, Hq, scale, cap)


def ps_kv4_attn(c, Q, O, lse=None, *, scale, len=None, span=None, kpos=None, qpos=None,
                slope=None, cap=0.0, ws=None, stream=None):
    """Attention of Q [B][T][Hq][dh] over the cache into O (Q's dtype) and lse
    [B][T][Hq]; what a row sees, the cap and the distance bias as in
    include/polestar.h."""
    lib = _lib()
    T, Hq, q = _kv4_query(c, Q, len, span, kpos, qpos, slope, scale, cap)
    w, wn = _ws(ws)
    st = lib.cdll.ps_kv4_attn(lib.handle(c.index), c._c, q,
                              _plain(O, Q.dtype, (c.B, T, Hq, c.dh)),
                              _plain(lse, torch.float32, (c.B, T, Hq), True), w, wn,
                              _kv4_stream(stream, c))
    _check(st, "ps_kv4_attn")


def ps_kv4_weight(c, Q, lse, w_in, w_out, *, scale, len=None, span=None, kpos=None, qpos=None,
                  slope=None, cap=0.0, ws=None, stream=None):
    """w_out = w_in (None: 0) + the attention weight that Q's rows put on each
    slot [B][Hkv][Ncache]; lse as ps_kv4_attn wrote it."""
    lib = _lib()
    T, Hq, q = _kv4_query(c, Q, len, span, kpos, qpos, slope, scale, cap)
    shape = (c.B, c.Hkv, c.N)
    w, wn = _ws(ws)
    st = lib.cdll.ps_kv4_weight(lib.handle(c.index), c._c, q,
                                _plain(lse, torch.float32, (c.B, T, Hq)),
                                _plain(w_in, torch.float32, shape, True),
                                _plain(w_out, torch.float32, shape), w, wn, _kv4_stream(stream, c))
    _check(st, "ps_kv4_weight")


def ps_kv4_evict(src, dst, w, w_dst, len_dst, keep, sink=0, recent=0, len=None, kpos=None,
                 kpos_dst=None, ws=None, stream=None, shift=None, shift_dst=None):
    """Keeps `keep` slots of every (sequence, KV head) of src -- the first
    `sink`, the last `recent` and the heaviest of the others by w -- in the
    first slots of dst.  With shift_dst [B] the slots behind them get no weight
    and the positions that come next (ps_kv4_evict_on)."""
    lib = _lib()
    f32, i32 = torch.float32, torch.int32
    a, b = (src.B, src.Hkv, src.N), (src.B, src.Hkv, dst.N)
    wsp, wn = _ws(ws)
    args = (lib.handle(src.index), src._c, dst._c, _plain(w, f32, a),
            _plain(len, i32, (src.B,), True), _plain(kpos, i32, a, True), int(keep), int(sink),
            int(recent), _plain(w_dst, f32, b), _plain(kpos_dst, i32, b, True),
            _plain(len_dst, i32, (src.B,)))
    if shift_dst is None:
        st = lib.cdll.ps_kv4_evict(*args, wsp, wn, _kv4_stream(stream, src))
    else:
        st = lib.cdll.ps_kv4_evict_on(*args, _plain(shift, i32, (src.B,), True),
                                      _plain(shift_dst, i32, (src.B,)), wsp, wn,
                                      _kv4_stream(stream, src))
    _check(st, "ps_kv4_evict")


# ---- rotary positions (include/polestar.h)
class RopeTable:
    """What rotates heads of dh elements: the first `rot` of each, in pairs
    (i, i + rot/2) or with `pairs` (2i, 2i + 1), by position * freq_i, times amp.
    scaling "linear", "ntk" (factor) or "parts" (factor, low, high, orig_len)
    stretches the frequencies."""

    def __init__(self, dh, rot=None, *, base=10000.0, pairs=False, scaling="none", factor=1.0,
                 low=1.0, high=4.0, orig_len=1.0, amp=1.0, device="cuda"):
        self.dh, self.rot = int(dh), int(dh if rot is None else rot)
        self.pairs, self.amp = bool(pairs), float(amp)
        if scaling not in ROPE_SCALING:
            raise ValueError(f"unknown scaling {scaling!r}: one of {', '.join(ROPE_SCALING)}")
        host = torch.zeros(max(self.rot, 2) // 2, dtype=torch.int64)
        p = RopeParams(self.rot, ROPE_SCALING[scaling], base, factor, low, high, orig_len)
        _check(_lib().cdll.ps_rope_turns(ctypes.byref(p), host.data_ptr()), "ps_rope_turns")
        self.turns = host.to(device)
        self.device = self.turns.device
        self.index = self.device.index
        # stays as it is
        self._head = self.turns.data_ptr()


_ROPE_ROWS = struct.Struct("6P6if4x")
_ROPE_PART = struct.Struct("2P4q3i4x")
_ROPE_PARTS = [struct.Struct("2P4q3i4x" * n) for n in range(4)]


def _at(t, dtype, shape, index):
    """Pointer of a contiguous tensor of this dtype and shape on GPU `index`; 0 of None."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"expected a contiguous {dtype} device tensor of shape {tuple(shape)} on "
                         f"GPU {index}, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on "
                         f"{t.device}")
    return t.data_ptr()


def _rope_part(t, B, T, H, dh, dtype, index):
    """(pointer, elements between sequences, elements between rows, rows, heads) of rows
    [B][T][H][dh]; T, H None: any."""
    shape = t.shape
    if (len(shape) != 4 or shape[0] != B or shape[3] != dh or (T is not None and shape[1] != T) or
            (H is not None and shape[2] != H) or t.dtype != dtype or t.get_device() != index):
        raise ValueError(f"expected {dtype} rows [{B}][{'rows' if T is None else T}]"
                         f"[{'heads' if H is None else H}][{dh}] on GPU {index}, got {t.dtype} "
                         f"{tuple(shape)} on {t.device}")
    if t.is_contiguous():
        ld = shape[2] * dh
        return t.data_ptr(), shape[1] * ld, ld, shape[1], shape[2]
    R, b, ld = _rows_ld(t, B, shape[2], dh)
    return t.data_ptr(), b, ld, R, shape[2]


def ps_rope(table, Q=None, K=None, V=None, *, Q_out=None, cache=None, pos=None, off=None,
            rows=None, cnt=None, dst=None, stream=None):
    """Rotates Q [B][T][Hq][dh] into Q_out (None: in place) and K [B][T][Hkv][dh] in place,
    or with cache=(Kc, Vc) into rows dst[b][r] (None: off[b] + r) of Kc [B][N][Hkv][dh],
    V's rows into Vc's.  Row r of sequence b stands at position pos[b][r] (None:
    off[b] + r); rows and cnt name the rows that take part."""
    if V is not None and cache is None:
        raise ValueError("V is not rotated: it only goes into a cache")
    if cache is not None and K is None:
        raise ValueError("a cache takes rows of K")
    if cache is not None and (V is None) != (cache[1] is None):
        raise ValueError("V and its cache go together")
    if Q_out is not None and Q is None:
        raise ValueError("Q_out without Q")
    x = K if Q is None else Q
    if x is None:
        raise ValueError("nothing to rotate")
    if x.dim() != 4:
        raise ValueError(f"expected rows [B][T][heads][{table.dh}], got {tuple(x.shape)}")
    (B, T, _, _), dh, dtype, index = x.shape, table.dh, x.dtype, table.index
    n, parts = 0, ()
    if Q is not None:
        xp, xb, xl, _, H = _rope_part(Q, B, T, None, dh, dtype, index)
        yp, yb, yl = (xp, xb, xl) if Q_out is None else \
            _rope_part(Q_out, B, T, H, dh, dtype, index)[:3]
        n, parts = 1, (xp, yp, xb, xl, yb, yl, H, 1, 0)
    for X, c in ((K, 0), (V, 1)):
        if X is None:
            continue
        xp, xb, xl, _, H = _rope_part(X, B, T, None, dh, dtype, index)
        if cache is None:
            yp, yb, yl, slots = xp, xb, xl, 0
        else:
            yp, yb, yl, slots, _ = _rope_part(cache[c], B, None, H, dh, dtype, index)
            if slots == 0:
                continue    # a cache without slots takes nothing
        n, parts = n + 1, parts + (xp, yp, xb, xl, yb, yl, H, 1 - c, slots)
    i32, each = torch.int32, (B, T)
    head = _ROPE_ROWS.pack(
        table._head, _at(pos, i32, each, index), _at(off, i32, (B,), index),
        _at(rows, i32, each, index), _at(cnt, i32, (B,), index), _at(dst, i32, each, index),
        B, T, dh, table.rot, table.pairs, _dtype(x), table.amp)
    if n == 0:
        return
    lib = _lib()
    st = lib.cdll.ps_rope(lib.handle(index), head, _ROPE_PARTS[n].pack(*parts), n,
                          raw_stream(stream, table.device))
    _check(st, "ps_rope")


# ---- attention over packed sequences or cache rows (include/polestar.h)
_ATTN_ROWS = struct.Struct("3P4q4P10if4x")


def _heads_ld(t, H, dh, dtype, index):
    """(rows, elements between rows) of t [rows][H][dh] on GPU `index`; H None: any."""
    shape = t.shape
    if (len(shape) != 3 or shape[2] != dh or (H is not None and shape[1] != H) or
            t.dtype != dtype or index < 0 or t.get_device() != index):
        raise ValueError(f"expected a {dtype} device tensor [rows][{'heads' if H is None else H}]"
                         f"[{dh}] on GPU {index}, got {t.dtype} {tuple(shape)} on {t.device}")
    R, h, _ = shape
    if t.is_contiguous():
        return R, h * dh
    sr, sh, sd = t.stride()
    if t.numel() > 0 and (sd != 1 or (sh != dh and h > 1)):
        raise ValueError(f"rows [{h}][{dh}] must be contiguous: strides {t.stride()}")
    return R, sr if R > 1 else h * dh


def ps_attn(Q, K, V, O, lse=None, *, q_off, k_off, k_len=None, span=None, causal=False,
            scale=None, max_q=None, max_k=None, ws=None, stream=None):
    """Attention of Q [Tq][Hq][dh] over K, V [Tk][Hkv][dh] (a cache [B][N][Hkv][dh] as
    B * N rows) into O [Tq][Hq][dh] and lse [Tq][Hq]: sequence s has the rows q_off[s] up to
    q_off[s + 1] of Q and k_off[s] up to k_off[s] + k_len[s] (k_len None: k_off[s + 1]) of K.
    max_q, max_k: the most of a sequence, if the caller knows (None: all of Q's, of K's).
    ws: of these numbers, ps.workspace(ps.OP_ATTN, B=S, N=max_k, Hq=.., Hkv=.., dh=.., P=Tq,
    k=max_q); one of others, larger ones too, may not be enough."""
    dh, dtype, index = Q.shape[-1], Q.dtype, Q.get_device()
    Tq, q_ld = _heads_ld(Q, None, dh, dtype, index)
    Hq = Q.shape[1]
    Tk, k_ld = _heads_ld(K, None, dh, dtype, index)
    Hkv = K.shape[1]
    Tv, v_ld = _heads_ld(V, Hkv, dh, dtype, index)
    To, o_ld = _heads_ld(O, Hq, dh, dtype, index)
    if Tv != Tk or To != Tq:
        raise ValueError(f"K and V need as many rows ({Tk}, {Tv}), Q and O too ({Tq}, {To})")
    if q_off is None or k_off is None or q_off.dim() != 1 or q_off.shape[0] < 1:
        raise ValueError("q_off and k_off say where the sequences begin")
    if ws is not None and ws.get_device() != index:
        raise ValueError(f"the workspace is on {ws.device}, the rows on GPU {index}")
    S = q_off.shape[0] - 1
    i32 = torch.int32
    lib = _lib()
    w, wn = _ws(ws)
    head = _ATTN_ROWS.pack(
        Q.data_ptr(), K.data_ptr(), V.data_ptr(), q_ld, k_ld, v_ld, o_ld,
        _at(q_off, i32, (S + 1,), index), _at(k_off, i32, (S + (k_len is None),), index),
        _at(k_len, i32, (S,), index), _at(span, i32, (Tq, 2), index), _dtype(Q), S, Tq, Tk,
        Hq, Hkv, dh, bool(causal), max(Tq, 1) if max_q is None else max_q,
        max(Tk, 1) if max_k is None else max_k, dh ** -0.5 if scale is None else scale)
    st = lib.cdll.ps_attn(lib.handle(index), head, O.data_ptr(),
                          _at(lse, torch.float32, (Tq, Hq), index), w, wn,
                          raw_stream(stream, Q.device))
    _check(st, "ps_attn")


# ---- drawn tokens (include/polestar.h)
_SAMPLE_ROWS = struct.Struct("6Pq3i4x")


def ps_sample(logits, u, token, prob=None, n=None, *, temperature=None, top_k=None, top_p=None,
              min_p=None, stream=None):
    """Draws a token of every row of logits [R][V] (rows may lie apart) by u [R] f64 from
    what temperature, top_k, top_p and min_p ([R] each, or None) leave; prob [R], n [R]:
    its probability and how many were left."""
    if logits.dim() != 2 or not logits.is_cuda:
        raise ValueError(f"expected device logits [rows][vocabulary], got {tuple(logits.shape)}")
    R, V = logits.shape
    if V > 1 and R > 0 and logits.stride(1) != 1:
        raise ValueError(f"rows of logits must be contiguous: strides {logits.stride()}")
    if u is None or token is None:
        raise ValueError("u and token are not optional")
    f32, i32, index, each = torch.float32, torch.int32, logits.get_device(), (R,)
    lib = _lib()
    s = _SAMPLE_ROWS.pack(
        logits.data_ptr(), _at(u, torch.float64, each, index),
        _at(temperature, f32, each, index), _at(top_k, i32, each, index),
        _at(top_p, f32, each, index), _at(min_p, f32, each, index),
        logits.stride(0) if R > 1 else V, _dtype(logits), R, V)
    st = lib.cdll.ps_sample(lib.handle(index), s, _at(token, i32, each, index),
                            _at(prob, f32, each, index), _at(n, i32, each, index),
                            raw_stream(stream, logits.device))
    _check(st, "ps_sample")


def ps_commit_drawn(conf, role, undecided, D_blk, d_ld, d_sum, d_cnt, d_prev, suffix_sel, sel_ld,
                    params, commit, stream=None):
    """ps_commit's rule on tokens that were drawn, conf [B][P] their confidences, all on one
    GPU."""
    index = conf.get_device()
    for t in (role, undecided, D_blk, d_sum, d_cnt, d_prev, suffix_sel, commit):
        if t is not None and t.get_device() != index:
            raise ValueError(f"expected device tensors on GPU {index}, got one on {t.device}")
    B, P = conf.shape
    at = _plain(conf, torch.float32, (B, P))
    lib = _lib()
    st = lib.cdll.ps_commit_drawn(
        lib.handle(index), at, B, P, _ptr(role), _ptr(undecided),
        _ptr(D_blk), d_ld, _ptr(d_sum), _ptr(d_cnt), _ptr(d_prev), _ptr(suffix_sel), sel_ld,
        params, _ptr(commit), raw_stream(stream, conf.device))
    _check(st, "ps_commit_drawn")


# ---- refresh schedule of the decode loop (include/polestar.h; host only)
def ps_schedule_step(params, state, committed, block_done):
    """Actions (SCHED_* flags) of the next step; updates `state` in place."""
    act = _lib().cdll.ps_schedule_step(ctypes.byref(params), ctypes.byref(state),
                                       int(committed), int(bool(block_done)))
    if act < 0:
        raise PolestarError(-act, "ps_schedule_step")
    return act


class Schedule:
    """A decode loop's schedule: tau_upd tokens between refreshes, every
    full_period-th refresh in full, the window sliding by block_len."""

    def __init__(self, tau_upd, full_period, block_len):
        self.params = ScheduleParams(int(tau_upd), int(full_period), int(block_len))
        self.state = ScheduleState(0, 0, 0)

    def step(self, committed, block_done):
        return ps_schedule_step(self.params, self.state, committed, block_done)
