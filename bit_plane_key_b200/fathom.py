"""Python binding of libfathom (the C ABI in include/fathom.h).

Argument marshalling only: every step of the scan runs in the library's CUDA
kernels.  Tensors are torch tensors (device memory, or page-locked host memory
for host-resident stores and rows); torch is used for allocation and streams.
If libfathom.so is missing this module raises at import: there is no CPU or
fallback path.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfathom.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libfathom.so is not built; run `python -m bit_plane_key_b200.build` (needs nvcc)")

_lib = ctypes.CDLL(LIB_PATH)

OK, EINVAL, ENOMEM, ECUDA, ETIMEOUT, EUNSUPPORTED = range(6)
F32, BF16 = 0, 1
DEV_BAD_DEPTH, DEV_BAD_INDEX, DEV_TOPK_OVERFLOW, DEV_TIMEOUT = 1, 2, 4, 8
MAX_TOPK = 4096


class FathomError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = _lib.fathom_status_string(status).decode()
        super().__init__("%s: %s (status %d)" % (what, msg, status))


class fathom_store(ctypes.Structure):
    _fields_ = [("n_kv_heads", ctypes.c_int32), ("d", ctypes.c_int32), ("n", ctypes.c_int64),
                ("n_pad", ctypes.c_int64), ("host_resident", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("planes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_P, _I, _L, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_SP = ctypes.POINTER(fathom_store)


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_sig("fathom_n_pad", _L, [_L])
_sig("fathom_planes_bytes", _Z, [_I, _I, _L])
_sig("fathom_scales_bytes", _Z, [_I, _I, _L])
_sig("fathom_pack_bitplanes", _I, [_P, _I, _I, _L, _I, _P, _P, _P])
_sig("fathom_alloc_depths", _I, [_P, _I, _P, _I, _I, _I, _I, _I, _P, _P])
_sig("fathom_alloc_depths_pooled", _I, [_P, _I, _P, _I, _I, _I, _I, _P, _P])
_sig("fathom_append_keys", _I, [_SP, _P, _I, _L, _P])
_sig("fathom_topk_merge", _I, [_P, _P, _I, _I, _I, _P, _P, _P, _Z, _P])
_sig("fathom_scan_scores", _I, [_SP, _P, _I, _P, _I, _P, _P, _P])
_sig("fathom_topk_workspace_bytes", _Z, [_L, _I, _I])
_sig("fathom_topk", _I, [_P, _P, _L, _L, _I, _I, _P, _P, _P, _Z, _P])
_sig("fathom_scan_workspace_bytes", _Z, [_SP, _I, _I])
_sig("fathom_scan_topk", _I, [_SP, _P, _I, _P, _I, _I, _P, _P, _P, _Z, _P])
_sig("fathom_sparse_attend", _I, [_P, _I, _P, _P, _L, _I, _P, _I, _I, _L, _I, _I, _P, _P])
_sig("fathom_sparse_attend_partial", _I, [_P, _I, _P, _P, _L, _I, _L, _P, _I, _I, _L, _I, _I, _P, _P])
_sig("fathom_attend_merge", _I, [_P, _I, _I, _I, _P, _P])
_sig("fathom_last_device_status", _I, [_P])
_sig("fathom_status_string", ctypes.c_char_p, [_I])
_sig("fathom_read_probe", _I, [_P, _Z, _I, _P, _I, _P])
_sig("fathom_noalloc_scratch_bytes", _Z, [])
_sig("fathom_scan_batched_workspace_bytes", _Z, [_SP, _I, _I, _I])
_sig("fathom_scan_topk_batched", _I, [_SP, _I, _P, _I, _P, _I, _I, _P, _P, _P, _Z, _P])
_sig("fathom_scan_topk_noalloc", _I, [_SP, _P, _I, _P, _I, _I, _P, _P, _P])
_sig("fathom_decode_workspace_bytes", _Z, [_SP, _I, _I, _I])
_sig("fathom_decode_step", _I, [_SP, _P, _I, _P, _I, _I, _I, _I, _P, _P, _L, _L, _I, _I, _P, _P, _P, _P, _P, _Z, _P])
_F = ctypes.c_float
_sig("fathom_qk_norm_rope", _I, [_P, _I, _L, _I, _I, _I, _I, _P, _P, _I, _F, _P, _P, _I, _I, _P, _P, _P, _L, _I, _L, _L,
                                 _P])
_sig("fathom_append_rows", _I, [_SP, _SP, _P, _P, _L, _I, _L, _L, _P])
_sig("fathom_store_attend_workspace_bytes", _Z, [_I, _I, _I, _I, _I])
_sig("fathom_store_attend", _I, [_SP, _SP, _P, _I, _I, _I, _I, _P, _P, _Z, _P])
_sig("fathom_store_attend_partial", _I, [_SP, _SP, _P, _I, _I, _I, _L, _P, _P, _Z, _P])
_sig("fathom_store_attend_batched", _I, [_SP, _SP, _I, _P, _I, _I, _I, _I, _P, _P, _Z, _P])


def lib():
    """The loaded ctypes library (for calls with raw pointers)."""
    return _lib


def _check(rc, what):
    if rc != OK:
        raise FathomError(rc, what)


def _stream(stream):
    """The stream's handle (an int, which ctypes passes as a pointer); the current device's current stream by default."""
    if stream is not None:
        return stream.cuda_stream
    if not torch.cuda.is_initialized():
        torch.cuda.init()
    # torch.cuda.current_stream() builds a Stream object for 3 us; this is the handle alone
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _dtype_code(t):
    if t.dtype == torch.float32:
        return F32
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return BF16
    raise TypeError("expected float32 or bfloat16, got %s" % t.dtype)


def n_pad(n):
    return int(_lib.fathom_n_pad(int(n)))


class Store:
    """A packed bit-plane store: planes u32 [Hkv][d][4][n_pad/32], scales u16 [Hkv][d][n_pad/64].
    n = keys held; n_pad = capacity (the row stride, from the arrays' shape)."""

    def __init__(self, planes, scales, n, host_resident=None):
        self.planes, self.scales, self.n = planes, scales, int(n)
        self.n_kv_heads, self.d = int(planes.shape[0]), int(planes.shape[1])
        self.n_pad = int(planes.shape[-1]) * 32
        self.host_resident = (not planes.is_cuda) if host_resident is None else bool(host_resident)
        self._c = fathom_store(self.n_kv_heads, self.d, self.n, self.n_pad, int(self.host_resident), 0,
                               planes.data_ptr(), scales.data_ptr())

    @property
    def c(self):
        return ctypes.byref(self._c)

    @classmethod
    def empty(cls, n_kv_heads, d, capacity, device=None, host_resident=False):
        """An empty store (n = 0) with room for `capacity` keys, zero-filled,
        in device memory or page-locked host memory; grow it with append_keys."""
        cap = n_pad(capacity)
        kw = dict(pin_memory=True) if host_resident else dict(device=device)
        planes = torch.zeros((n_kv_heads, d, 4, cap // 32), dtype=torch.int32, **kw)
        scales = torch.zeros((n_kv_heads, d, cap // 64), dtype=torch.int16, **kw)
        return cls(planes, scales, 0, host_resident=host_resident)

    def to_host(self):
        """Copy of this store in page-locked host memory (host-resident)."""
        return Store(self.planes.cpu().pin_memory(), self.scales.cpu().pin_memory(), self.n, host_resident=True)

    def plane_bytes_read(self, union_depths):
        """Plane + scale bytes a scan reads for union depths U [Hkv][d] (over the
        first n_pad(n) keys, the range a scan covers)."""
        U = union_depths.to(torch.int64)
        npad = n_pad(self.n)
        return int(U.sum()) * npad // 8 + int((U > 0).sum()) * (npad // 64) * 2


def pack_bitplanes(K, planes=None, scales=None, stream=None):
    """K [Hkv][n][d] (float32 or bfloat16, cuda) -> Store."""
    Hkv, n, d = K.shape
    npad = n_pad(n)
    if planes is None:
        planes = torch.empty((Hkv, d, 4, npad // 32), dtype=torch.int32, device=K.device)
    if scales is None:
        scales = torch.empty((Hkv, d, npad // 64), dtype=torch.int16, device=K.device)
    _check(_lib.fathom_pack_bitplanes(_ptr(K), _dtype_code(K), Hkv, n, d, _ptr(planes), _ptr(scales),
                                      _stream(stream)), "fathom_pack_bitplanes")
    return Store(planes, scales, n, host_resident=False)


def append_keys(store, K_tail, n_new, stream=None):
    """Decode-time append: keys [store.n, n_new) into a store with the capacity.
    K_tail [Hkv][n_new - t][d] (cuda, float32 or bfloat16) holds the keys from
    t = (store.n // 64) * 64 on.  Updates store.n."""
    _check(_lib.fathom_append_keys(store.c, _ptr(K_tail), _dtype_code(K_tail), int(n_new), _stream(stream)),
           "fathom_append_keys")
    store.n = int(store._c.n)
    return store


def alloc_depths(q, sigma2, budget_bits, fixed_r=0, out=None, stream=None):
    """q [Hq][d], sigma2 f32 [Hkv][d] -> depths u8 [Hq][d]."""
    Hq, d = q.shape
    Hkv = sigma2.shape[0]
    if out is None:
        out = torch.empty((Hq, d), dtype=torch.uint8, device=q.device)
    _check(_lib.fathom_alloc_depths(_ptr(q), _dtype_code(q), _ptr(sigma2), Hq, Hkv, d, int(budget_bits),
                                    int(fixed_r), _ptr(out), _stream(stream)), "fathom_alloc_depths")
    return out


def alloc_depths_pooled(q, sigma2, budget_bits, out=None, stream=None):
    """Group-pooled depths (one depth vector per KV head, repeated for its query
    heads): q [Hq][d], sigma2 f32 [Hkv][d] -> depths u8 [Hq][d]."""
    Hq, d = q.shape
    Hkv = sigma2.shape[0]
    if out is None:
        out = torch.empty((Hq, d), dtype=torch.uint8, device=q.device)
    _check(_lib.fathom_alloc_depths_pooled(_ptr(q), _dtype_code(q), _ptr(sigma2), Hq, Hkv, d, int(budget_bits),
                                           _ptr(out), _stream(stream)), "fathom_alloc_depths_pooled")
    return out


def scan_scores(store, q, depths, out=None, block_max=None, stream=None):
    """Scores f32 [Hq][n_pad(n)] (padding keys -inf); block_max (optional) u32
    [Hq][n_pad(n)/64] receives the block maxima that topk() can use."""
    Hq = q.shape[0]
    if out is None:
        out = torch.empty((Hq, n_pad(store.n)), dtype=torch.float32, device=q.device)
    _check(_lib.fathom_scan_scores(store.c, _ptr(q), _dtype_code(q), _ptr(depths), Hq, _ptr(out), _ptr(block_max),
                                   _stream(stream)), "fathom_scan_scores")
    return out


def block_max_buffer(n_rows, n, device):
    """A block-maxima buffer for scan_scores / topk: u32 (as int32) [rows][n_pad(n)/64]."""
    return torch.empty((n_rows, n_pad(n) // 64), dtype=torch.int32, device=device)


def topk_workspace_bytes(n, rows, k):
    return int(_lib.fathom_topk_workspace_bytes(int(n), int(rows), int(k)))


def topk(scores, n, k, idx=None, top_scores=None, workspace=None, block_max=None, stream=None):
    """Top-k of score rows [rows][ld] over the first n columns (block_max: the
    block maxima the scan wrote with these scores, or None)."""
    rows, ld = scores.shape
    if idx is None:
        idx = torch.empty((rows, k), dtype=torch.int32, device=scores.device)
    if top_scores is None:
        top_scores = torch.empty((rows, k), dtype=torch.float32, device=scores.device)
    nb = topk_workspace_bytes(n, rows, k)
    if workspace is None:
        workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=scores.device)
    _check(_lib.fathom_topk(_ptr(scores), _ptr(block_max), int(n), int(ld), rows, int(k), _ptr(idx),
                            _ptr(top_scores), _ptr(workspace), workspace.numel(), _stream(stream)), "fathom_topk")
    return idx, top_scores


def topk_merge(cand_scores, cand_idx, k, idx=None, top_scores=None, workspace=None, stream=None):
    """Top-k of gathered per-shard lists: cand_scores f32 / cand_idx i32 [rows][n_cand]
    (shards in ascending key-range order, each list in top-k order) -> idx, scores [rows][k]."""
    rows, n_cand = cand_scores.shape
    if idx is None:
        idx = torch.empty((rows, k), dtype=torch.int32, device=cand_scores.device)
    if top_scores is None:
        top_scores = torch.empty((rows, k), dtype=torch.float32, device=cand_scores.device)
    nb = topk_workspace_bytes(n_cand, rows, k)
    if workspace is None:
        workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=cand_scores.device)
    _check(_lib.fathom_topk_merge(_ptr(cand_scores), _ptr(cand_idx), rows, n_cand, int(k), _ptr(idx),
                                  _ptr(top_scores), _ptr(workspace), workspace.numel(), _stream(stream)),
           "fathom_topk_merge")
    return idx, top_scores


def scan_workspace_bytes(store, n_q_heads, k):
    return int(_lib.fathom_scan_workspace_bytes(store.c, int(n_q_heads), int(k)))


def scan_topk(store, q, depths, k, idx=None, top_scores=None, workspace=None, stream=None):
    """idx i32 [Hq][k] and top scores f32 [Hq][k]."""
    Hq = q.shape[0]
    if idx is None:
        idx = torch.empty((Hq, k), dtype=torch.int32, device=q.device)
    if top_scores is None:
        top_scores = torch.empty((Hq, k), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(scan_workspace_bytes(store, Hq, k), 1), dtype=torch.uint8, device=q.device)
    _check(_lib.fathom_scan_topk(store.c, _ptr(q), _dtype_code(q), _ptr(depths), Hq, int(k), _ptr(idx),
                                 _ptr(top_scores), _ptr(workspace), workspace.numel(), _stream(stream)),
           "fathom_scan_topk")
    return idx, top_scores


def _store_array(stores):
    return (fathom_store * len(stores))(*[st._c for st in stores])


def scan_batched_workspace_bytes(stores, n_q_heads, k):
    arr = _store_array(stores)
    return int(_lib.fathom_scan_batched_workspace_bytes(arr, len(stores), int(n_q_heads), int(k)))


def scan_topk_batched(stores, q, depths, k, idx=None, top_scores=None, workspace=None, stream=None):
    """Sessions `stores` (list of Store), q [S][Hq][d], depths [S][Hq][d] -> idx, top scores [S][Hq][k]."""
    S, Hq = q.shape[0], q.shape[1]
    arr = _store_array(stores)
    if idx is None:
        idx = torch.empty((S, Hq, k), dtype=torch.int32, device=q.device)
    if top_scores is None:
        top_scores = torch.empty((S, Hq, k), dtype=torch.float32, device=q.device)
    if workspace is None:
        nb = int(_lib.fathom_scan_batched_workspace_bytes(arr, S, Hq, int(k)))
        workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=q.device)
    _check(_lib.fathom_scan_topk_batched(arr, S, _ptr(q), _dtype_code(q), _ptr(depths), Hq, int(k), _ptr(idx),
                                         _ptr(top_scores), _ptr(workspace), workspace.numel(), _stream(stream)),
           "fathom_scan_topk_batched")
    return idx, top_scores


def scan_scores_view(workspace, n_q_heads, n_pad_keys):
    """The scan's scores inside a fathom_scan_topk workspace: f32 [Hq][n_pad]."""
    return workspace[: 4 * n_q_heads * n_pad_keys].view(torch.float32).view(n_q_heads, n_pad_keys)


def kv_rows(n_kv_heads, n, d, device=None, pin_memory=False):
    """K and V row views [Hkv][n][d] (bf16) of one interleaved [Hkv][n][2][d]
    buffer: a key's K and V rows are adjacent, which is the layout to use for
    rows kept in page-locked host memory."""
    kv = torch.empty((n_kv_heads, n, 2, d), dtype=torch.bfloat16, device=device, pin_memory=pin_memory)
    return kv[:, :, 0, :], kv[:, :, 1, :]


def sparse_attend(q, K_rows, V_rows, idx, n_kv_heads=None, out=None, stream=None):
    """o f32 [Hq][d]; K_rows/V_rows bf16 [Hkv][n][d] views with unit channel
    stride and equal strides (two arrays, or the views of kv_rows()), on the
    device or in page-locked host memory."""
    Hq, d = q.shape
    Hkv, n, _ = K_rows.shape
    k = idx.shape[1]
    host = not K_rows.is_cuda
    if K_rows.stride() != V_rows.stride() or K_rows.stride(2) != 1 or K_rows.stride(0) != n * K_rows.stride(1):
        raise ValueError("K_rows and V_rows need strides (n*s, s, 1), the same for both")
    if out is None:
        out = torch.empty((Hq, d), dtype=torch.float32, device=q.device)
    _check(_lib.fathom_sparse_attend(_ptr(q), _dtype_code(q), _ptr(K_rows), _ptr(V_rows), int(K_rows.stride(1)),
                                     int(host), _ptr(idx), Hq, Hkv, n, d, int(k), _ptr(out), _stream(stream)),
           "fathom_sparse_attend")
    return out


def sparse_attend_partial(q, K_rows, V_rows, idx, key0, n_kv_heads=None, parts=None, stream=None):
    """Partials f32 [Hq][d + 2] (o relative to m, then m, l) of attention over
    the rows this rank holds: K_rows/V_rows as sparse_attend, holding keys
    [key0, key0 + n); idx are global key indices (others and -1 skipped)."""
    Hq, d = q.shape
    Hkv, n, _ = K_rows.shape
    k = idx.shape[1]
    host = not K_rows.is_cuda
    if K_rows.stride() != V_rows.stride() or K_rows.stride(2) != 1 or K_rows.stride(0) != n * K_rows.stride(1):
        raise ValueError("K_rows and V_rows need strides (n*s, s, 1), the same for both")
    if parts is None:
        parts = torch.empty((Hq, d + 2), dtype=torch.float32, device=q.device)
    _check(_lib.fathom_sparse_attend_partial(_ptr(q), _dtype_code(q), _ptr(K_rows), _ptr(V_rows),
                                             int(K_rows.stride(1)), int(host), int(key0), _ptr(idx), Hq, Hkv, n, d,
                                             int(k), _ptr(parts), _stream(stream)),
           "fathom_sparse_attend_partial")
    return parts


def attend_merge(parts, out=None, stream=None):
    """o f32 [Hq][d] from the ranks' partials f32 [world][Hq][d + 2]."""
    world, Hq, d2 = parts.shape
    if out is None:
        out = torch.empty((Hq, d2 - 2), dtype=torch.float32, device=parts.device)
    _check(_lib.fathom_attend_merge(_ptr(parts.contiguous()), world, Hq, d2 - 2, _ptr(out), _stream(stream)),
           "fathom_attend_merge")
    return out


def last_device_status(stream=None):
    v = _lib.fathom_last_device_status(_stream(stream))
    if v < 0:
        raise FathomError(-v, "fathom_last_device_status")
    return v


def read_probe(src, sink, ctas=None, stream=None):
    """Stream all of `src` (device or page-locked host tensor) through the SMs."""
    host = not src.is_cuda
    if ctas is None:
        ctas = torch.cuda.get_device_properties(sink.device).multi_processor_count * 8
    _check(_lib.fathom_read_probe(_ptr(src), src.numel() * src.element_size(), int(host), _ptr(sink), int(ctas),
                                  _stream(stream)), "fathom_read_probe")


def noalloc_scratch_bytes():
    return int(_lib.fathom_noalloc_scratch_bytes())


def scan_topk_noalloc(store, q, depths, k, idx, top_scores=None, stream=None):
    """fathom_scan_topk on the library's fixed scratch array (no workspace; idx preallocated)."""
    _check(_lib.fathom_scan_topk_noalloc(store.c, _ptr(q), _dtype_code(q), _ptr(depths), q.shape[0], int(k),
                                         _ptr(idx), _ptr(top_scores), _stream(stream)), "fathom_scan_topk_noalloc")
    return idx, top_scores


def decode_workspace_bytes(store, n_q_heads, k, kv_groups):
    return int(_lib.fathom_decode_workspace_bytes(store.c, int(n_q_heads), int(k), int(kv_groups)))


def decode_step(store, q, sigma2, budget_bits, k, K_rows, V_rows, fixed_r=0, kv_groups=1, depths=None, idx=None,
                top_scores=None, out=None, workspace=None, stream=None, want_top_scores=True):
    """One decode step (depths, scan, top-k, attention) in one C-ABI call,
    pipelined over kv_groups groups of KV heads.  Returns (depths, idx,
    top_scores or None, out)."""
    Hq, d = q.shape
    dev = q.device
    rows_n = K_rows.shape[1]
    if K_rows.stride() != V_rows.stride() or K_rows.stride(2) != 1 or K_rows.stride(0) != rows_n * K_rows.stride(1):
        raise ValueError("K_rows and V_rows need strides (rows*s, s, 1), the same for both")
    if depths is None:
        depths = torch.empty((Hq, d), dtype=torch.uint8, device=dev)
    if idx is None:
        idx = torch.empty((Hq, k), dtype=torch.int32, device=dev)
    if top_scores is None and want_top_scores:
        top_scores = torch.empty((Hq, k), dtype=torch.float32, device=dev)
    if out is None:
        out = torch.empty((Hq, d), dtype=torch.float32, device=dev)
    need = decode_workspace_bytes(store, Hq, k, kv_groups)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check(_lib.fathom_decode_step(store.c, _ptr(q), _dtype_code(q), _ptr(sigma2), Hq, int(budget_bits), int(fixed_r),
                                   int(k), _ptr(K_rows), _ptr(V_rows), int(rows_n), int(K_rows.stride(1)),
                                   int(not K_rows.is_cuda), int(kv_groups), _ptr(depths), _ptr(idx),
                                   _ptr(top_scores), _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "fathom_decode_step")
    return depths, idx, top_scores, out


_BF16_BITS = (torch.bfloat16, torch.int16, torch.uint16)


def _check_rows(K_rows, V_rows):
    """Strides of a row cache, K_rows and V_rows [Hkv][rows][d]; returns (row stride, rows, host-resident)."""
    Hkv, rows_n, _ = shape = K_rows.shape
    strides = K_rows.stride()
    if K_rows.dtype not in _BF16_BITS or V_rows.dtype is not K_rows.dtype:
        raise TypeError("K_rows and V_rows hold bfloat16")
    cuda = K_rows.is_cuda
    if (shape != V_rows.shape or strides != V_rows.stride() or strides[2] != 1
            or (Hkv > 1 and strides[0] != rows_n * strides[1]) or cuda != V_rows.is_cuda):
        raise ValueError("K_rows and V_rows need strides (rows*s, s, 1), the same for both")
    return strides[1], rows_n, int(not cuda)


def _check_is(t, shape, dtype, what):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous %s %s" % (what, dtype, tuple(shape)))


def qk_norm_rope(qkv, n_q_heads, n_kv_heads, inv_freq, K_rows, V_rows, row0, q_weight=None, k_weight=None, eps=1e-6,
                 positions=None, interleaved=False, out=None, stream=None):
    """Norms (when weights are given) and rotation of a projection's query and
    key heads: qkv [T][Hq + 2 Hkv][d] (float32 or bfloat16, a token's heads
    contiguous), inv_freq f32 [rot_dim / 2].  Returns the queries [T][Hq][d] and
    writes token t's key and value rows at row0 + t of the row cache (bf16 views
    as sparse_attend).  positions i32 [T], default row0 + t."""
    T, H, d = qkv.shape
    ts, hs, cs = qkv.stride()
    if H != n_q_heads + 2 * n_kv_heads or cs != 1 or (H > 1 and hs != d):
        raise ValueError("qkv must be [T][Hq + 2 Hkv][d] with a token's heads contiguous")
    stride, rows_n, host = _check_rows(K_rows, V_rows)
    if K_rows.shape[0] != n_kv_heads or K_rows.shape[2] != d:
        raise ValueError("K_rows and V_rows must be [Hkv][rows][d]")
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be contiguous float32 [rot_dim / 2]")
        rot = 2 * inv_freq.shape[0]
    w_dtype = F32
    if k_weight is not None and q_weight is None:
        raise ValueError("q_weight and k_weight go together")
    for w in (q_weight, k_weight):
        if w is not None:
            if w.shape != (d,) or not w.is_contiguous() or w.dtype is not q_weight.dtype:
                raise ValueError("q_weight and k_weight must be contiguous [d] of one dtype")
            w_dtype = _dtype_code(w)
    if positions is not None:
        _check_is(positions, (T,), torch.int32, "positions")
    if out is None:
        out = _empty(qkv, (T, n_q_heads, d), qkv.dtype, stream)
    else:
        _check_is(out, (T, n_q_heads, d), qkv.dtype, "out")
    if T == 0:
        return out
    # a single token has no stride of its own
    rc = _lib.fathom_qk_norm_rope(qkv.data_ptr(), _dtype_code(qkv), ts if T > 1 else H * d, T, int(n_q_heads), int(n_kv_heads), d,
                                  _ptr(q_weight), _ptr(k_weight), w_dtype, float(eps), _ptr(positions), _ptr(inv_freq), rot,
                                  bool(interleaved), out.data_ptr(), K_rows.data_ptr(), V_rows.data_ptr(), stride, host,
                                  rows_n, int(row0), _stream(stream))
    if rc:
        _check(rc, "fathom_qk_norm_rope")
    return out


def append_rows(k_store, v_store, K_rows, V_rows, n_new, stream=None):
    """Grows the K store and the V store to n_new keys from the row cache (views
    as sparse_attend, key i of the store = row i); v_store and V_rows None: the K
    store alone."""
    if (v_store is None) != (V_rows is None):
        raise ValueError("v_store and V_rows go together")
    stride, rows_n, host = _check_rows(K_rows, K_rows if V_rows is None else V_rows)
    if K_rows.shape[0] != k_store.n_kv_heads or K_rows.shape[2] != k_store.d:
        raise ValueError("K_rows must be [Hkv][rows][d] of the store")
    _check(_lib.fathom_append_rows(k_store.c, v_store.c if v_store is not None else None, _ptr(K_rows), _ptr(V_rows),
                                   stride, host, rows_n, int(n_new), _stream(stream)), "fathom_append_rows")
    for st in (k_store, v_store):
        if st is not None:
            st.n = int(st._c.n)
    return k_store, v_store


def store_attend_workspace_bytes(store, n_sessions, n_tokens, n_q_heads):
    return int(_lib.fathom_store_attend_workspace_bytes(int(n_sessions), int(n_tokens), int(n_q_heads),
                                                        store.n_kv_heads, store.d))


def _empty(like, shape, dtype, stream):
    """New memory that belongs to the stream of the call: once freed, it is used again behind the call alone."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _attend_args(store, q, lead, out, width, workspace, stream):
    """Checks q [lead...][Hq][d] and makes out f32 [lead...][Hq][width] and the workspace."""
    shape = q.shape
    if len(shape) != lead + 2 or lead < 0 or shape[-1] != store.d or not q.is_contiguous():
        raise ValueError("q must be contiguous [...][Hq][d] with d = %d" % store.d)
    want = shape if width == store.d else shape[:-1] + (width,)
    if out is None:
        out = _empty(q, want, torch.float32, stream)
    else:
        _check_is(out, want, torch.float32, "out")
    T = shape[-3] if lead else 1
    if workspace is None:
        nb = store_attend_workspace_bytes(store, shape[0] if lead == 2 else 1, T, shape[-2])
        workspace = _empty(q, (max(nb, 1),), torch.uint8, stream)
    return out, T, workspace


def _attend_lead(q):
    if q.dim() not in (2, 3):
        raise ValueError("q must be [Hq][d] or [T][Hq][d]")
    return q.dim() - 2


def store_attend(k_store, v_store, q, causal=True, out=None, workspace=None, stream=None):
    """Attention over every key of the K store and the 4-bit values of the V
    store: q [Hq][d] or [T][Hq][d] -> f32 of the same shape.  causal: the stores'
    last T keys are the T tokens' own, each sees its past and itself; else every
    token sees all keys."""
    out, T, workspace = _attend_args(k_store, q, _attend_lead(q), out, k_store.d, workspace, stream)
    _check(_lib.fathom_store_attend(k_store.c, v_store.c, _ptr(q), _dtype_code(q), T, q.shape[-2], int(bool(causal)),
                                    _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "fathom_store_attend")
    return out


def store_attend_partial(k_store, v_store, q, visible, parts=None, workspace=None, stream=None):
    """Partials f32 [..][Hq][d + 2] (as sparse_attend_partial) of attention over
    this range's keys; token t sees those below visible + t."""
    parts, T, workspace = _attend_args(k_store, q, _attend_lead(q), parts, k_store.d + 2, workspace, stream)
    _check(_lib.fathom_store_attend_partial(k_store.c, v_store.c, _ptr(q), _dtype_code(q), T, q.shape[-2],
                                            int(visible), _ptr(parts), _ptr(workspace), workspace.numel(),
                                            _stream(stream)), "fathom_store_attend_partial")
    return parts


def store_attend_batched(k_stores, v_stores, q, causal=True, out=None, workspace=None, stream=None):
    """store_attend of the sessions (k_stores[s], v_stores[s]) in one pass: q
    [S][T][Hq][d] -> f32 of the same shape."""
    if not k_stores or len(k_stores) != q.shape[0] or len(v_stores) != q.shape[0]:
        raise ValueError("one K store and one V store for each session of q")
    out, T, workspace = _attend_args(k_stores[0], q, 2, out, k_stores[0].d, workspace, stream)
    _check(_lib.fathom_store_attend_batched(_store_array(k_stores), _store_array(v_stores), len(k_stores), _ptr(q),
                                            _dtype_code(q), T, q.shape[-2], int(bool(causal)), _ptr(out),
                                            _ptr(workspace), workspace.numel(), _stream(stream)),
           "fathom_store_attend_batched")
    return out
