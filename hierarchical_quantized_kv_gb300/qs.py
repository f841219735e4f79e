"""ctypes binding of libqs (include/qs.h): argument marshalling only.

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: each step of the hot path runs in the CUDA library.
PyTorch supplies device memory and the current stream.  If ``libqs.so`` has
not been built this module raises on first use -- there is no fallback.
"""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqs.so")

QS_DRAFT_UPPER4, QS_VERIFY_INT8 = 0, 1
(QS_OK, QS_ERR_ARG, QS_ERR_SHAPE, QS_ERR_ALIGN, QS_ERR_CUDA, QS_ERR_UNSUPPORTED, QS_ERR_WORKSPACE,
 QS_ERR_TOO_LARGE) = range(8)
QS_STATIC_WS_BYTES = 8 << 20
DEV_OVERFLOW, DEV_OVER_ROLLBACK, DEV_FLUSH_UNCOMMITTED, DEV_CAPACITY, DEV_NQ_GT_FILL, DEV_TIMEOUT = (
    1, 2, 4, 8, 16, 32)
DEV_PREFILL, DEV_PAGE, DEV_SELECT, DEV_TREE = 64, 128, 256, 512
QS_PAGED = 0x100
ST_N_GROUPS, ST_FILL, ST_PENDING, ST_HALF_BASE, ST_ERR, ST_TICKET = range(6)
STATE_WORDS = 8
QS_FP16, QS_BF16, QS_FP32 = range(3)
QS_MAX_TREE, QS_MAX_VOCAB = 64, 368640
META_K_SCALE, META_K_ZERO, META_V_SCALE, META_V_ZERO = range(4)

_P = ctypes.c_void_p
_I32 = ctypes.c_int32


class QsCacheStruct(ctypes.Structure):
    _fields_ = [("B", _I32), ("H", _I32), ("D", _I32), ("G", _I32), ("cap_groups", _I32),
                ("upper_bits", _I32), ("k_upper", _P), ("k_lower", _P), ("v_upper", _P), ("v_lower", _P),
                ("meta", _P), ("buf_k", _P), ("buf_v", _P), ("state", _P), ("arrive", _P)]


class QsPagesStruct(ctypes.Structure):
    _fields_ = [("table", _P), ("n_pages", _I32)]


class QsRowsStruct(ctypes.Structure):
    _fields_ = [("data", _P), ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_t", ctypes.c_int64)]


class QsCacheBytes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("k_upper", "k_lower", "v_upper", "v_lower", "meta", "buf_k", "buf_v", "state",
                 "arrive")]


class QsError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (fn, status_string(status), status))


class QsArgumentError(AssertionError, ValueError):
    """A tensor that does not fit the call: its shape, type, device or layout."""


_lib = None

# exported entry points and their argument types
_SIGS = {
    "qs_cache_bytes": [_I32, _I32, _I32, _I32, _I32, ctypes.POINTER(QsCacheBytes)],
    "qs_paged_cache_bytes": [_I32, _I32, _I32, _I32, _I32, ctypes.POINTER(QsCacheBytes)],
    "qs_quantize_flush_paged": [ctypes.POINTER(QsCacheStruct), ctypes.POINTER(QsPagesStruct), _P, _P],
    "qs_quantize_flush_due_paged": [ctypes.POINTER(QsCacheStruct), ctypes.POINTER(QsPagesStruct),
                                    _I32, _P],
    "qs_prefill_paged": [ctypes.POINTER(QsCacheStruct), ctypes.POINTER(QsPagesStruct), _P, _P, _I32,
                         _P, _P],
    "qs_state_reset": [ctypes.POINTER(QsCacheStruct), _P],
    "qs_buffer_append": [ctypes.POINTER(QsCacheStruct), _P, _P, _I32, _P],
    "qs_buffer_rollback": [ctypes.POINTER(QsCacheStruct), _P, _P],
    "qs_need_flush": [ctypes.POINTER(QsCacheStruct), _I32, _P, _P],
    "qs_quantize_flush": [ctypes.POINTER(QsCacheStruct), _P, _P],
    "qs_quantize_flush_due": [ctypes.POINTER(QsCacheStruct), _I32, _P],
    "qs_attn_workspace_size": [ctypes.POINTER(QsCacheStruct), _I32, ctypes.POINTER(ctypes.c_size_t)],
    "qs_attn_decode": [ctypes.POINTER(QsCacheStruct), ctypes.c_int, _P, _I32, ctypes.c_float, _P,
                       _P, _P, ctypes.c_size_t, _P],
    "qs_get_errors": [ctypes.POINTER(QsCacheStruct), _P, _P],
    "qs_attn_workspace_size_gqa": [ctypes.POINTER(QsCacheStruct), _I32, _I32,
                                   ctypes.POINTER(ctypes.c_size_t)],
    "qs_attn_decode_gqa": [ctypes.POINTER(QsCacheStruct), ctypes.c_int, _P, _I32, _I32, ctypes.c_float,
                           _P, _P, _P, ctypes.c_size_t, _P],
    "qs_prefill": [ctypes.POINTER(QsCacheStruct), _P, _P, _I32, _P, _P],
    "qs_attn_decode_paged": [ctypes.POINTER(QsCacheStruct), ctypes.POINTER(QsPagesStruct),
                             ctypes.c_int, _P, _P, _I32, _P, _I32, _I32, ctypes.c_float, _P, _P, _P,
                             ctypes.c_size_t, _P],
    "qs_attn_decode_sparse": [ctypes.POINTER(QsCacheStruct), ctypes.POINTER(QsPagesStruct),
                              ctypes.c_int, _P, _I32, _P, _P, _I32, _P, _I32, _I32, ctypes.c_float,
                              _P, _P, _P, ctypes.c_size_t, _P],
    "qs_select_groups": [ctypes.POINTER(QsCacheStruct), ctypes.POINTER(QsPagesStruct), _P, _I32, _I32,
                         _I32, _P, _P],
    "qs_cache_read": [ctypes.POINTER(QsCacheStruct), ctypes.POINTER(QsPagesStruct), ctypes.c_int,
                      _I32, _I32, _P, _P, _P],
    "qs_spec_accept": [_P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P],
    "qs_attn_decode_static_ws": [ctypes.POINTER(QsCacheStruct), ctypes.c_int, _P, _I32,
                                 ctypes.c_float, _P, _P, _P],
    "qs_attn_decode_append": [ctypes.POINTER(QsCacheStruct), ctypes.c_int, _P, _P, _I32, _P, _I32,
                              _I32, ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P],
    "qs_buffer_append_rotary": [ctypes.POINTER(QsCacheStruct), _P, _P, _P, _P, _I32, _I32, _P, _P, _I32,
                                _I32, _P],
    "qs_attn_tree_workspace_size": [ctypes.POINTER(QsCacheStruct), _I32, _I32,
                                    ctypes.POINTER(ctypes.c_size_t)],
    "qs_attn_decode_tree": [ctypes.POINTER(QsCacheStruct), ctypes.POINTER(QsPagesStruct), ctypes.c_int,
                            _P, _I32, _P, _I32, _I32, ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P],
    "qs_tree_accept": [ctypes.POINTER(QsCacheStruct), _P, _P, _P, _I32, _P, _P, _P, _P],
    "qs_sample": [_P, ctypes.c_int, _I32, _I32, ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P, _P],
}


def lib():
    """Load libqs.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libqs.so is not built (run __graft_entry__.build()); "
                               "there is no CPU fallback")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.qs_status_string.argtypes = [ctypes.c_int]
        L.qs_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(s):
    return lib().qs_status_string(int(s)).decode()


def _check(fn, status):
    if status != QS_OK:
        raise QsError(fn, status)


_current_raw_stream = None


def _current_stream_handle():
    """cudaStream_t of torch's current stream on the current device.  Through
    torch._C._cuda_getCurrentRawStream (the lookup torch's own generated code
    makes: about 0.3 us a call, against 3 us for torch.cuda.current_stream()
    on the Grace host) where this torch has it, else the public call."""
    global _current_raw_stream
    if _current_raw_stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        dev = getattr(torch._C, "_cuda_getDevice", None)
        if raw is not None and dev is not None:
            torch.cuda.init()
            _current_raw_stream = lambda: raw(dev())
        else:
            _current_raw_stream = lambda: torch.cuda.current_stream().cuda_stream
    return _current_raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream_handle()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t):
    # (a plain integer: ctypes converts it for a void * argument, a c_void_p
    # object per pointer cost 0.2 us each)
    return None if t is None else t.data_ptr()


# -------------------------------------------------------------------- cache

def qs_cache_bytes(B, H, cap_groups, D=128, G=128):
    out = QsCacheBytes()
    _check("qs_cache_bytes", lib().qs_cache_bytes(B, H, D, G, cap_groups, ctypes.byref(out)))
    return {n: getattr(out, n) for n, _ in QsCacheBytes._fields_}


class Cache:
    """A hierarchical quantized KV cache in torch-owned device memory, laid
    out as include/qs.h describes (shapes below are the C layouts)."""

    def __init__(self, B, H, cap_groups, device="cuda", D=128, G=128, upper_bits=4):
        """upper_bits: the top bits of each 8-bit code the draft reads (4, or
        2 for the two-bit draft layout of include/qs.h)."""
        qs_cache_bytes(B, H, cap_groups, D, G)  # validates the sizes
        self._alloc(B, H, cap_groups, device, D, G, upper_bits, (B, H, cap_groups))
        self.struct = self._struct(upper_bits)
        self._ref = ctypes.byref(self.struct)

    def _alloc(self, B, H, cap_groups, device, D, G, upper_bits, slots):
        import torch
        self.B, self.H, self.D, self.G, self.cap = B, H, D, G, cap_groups
        self.upper_bits = upper_bits
        self._f32 = torch.float32
        u8 = dict(dtype=torch.uint8, device=device)
        f16 = dict(dtype=torch.float16, device=device)
        self.k_upper = torch.zeros(slots + (G, D // 2), **u8)
        self.k_lower = torch.zeros(slots + (G, D // 2), **u8)
        self.v_upper = torch.zeros(slots + (G // 32, D, 16), **u8)
        self.v_lower = torch.zeros(slots + (G // 32, D, 16), **u8)
        self.meta = torch.zeros(slots + (4, 128), **f16)
        self.buf_k = torch.zeros((B, H, 2 * G, D), **f16)
        self.buf_v = torch.zeros((B, H, 2 * G, D), **f16)
        self.state = torch.zeros((B, STATE_WORDS), dtype=torch.int32, device=device)
        self.arrive = torch.zeros((B, H), dtype=torch.int32, device=device)
        self._f16, self._i32, self._dev = self.buf_k.dtype, self.state.dtype, self.state.get_device()

    def _struct(self, upper_bits):
        return QsCacheStruct(self.B, self.H, self.D, self.G, self.cap, upper_bits,
                             self.k_upper.data_ptr(), self.k_lower.data_ptr(),
                             self.v_upper.data_ptr(), self.v_lower.data_ptr(),
                             self.meta.data_ptr(), self.buf_k.data_ptr(),
                             self.buf_v.data_ptr(), self.state.data_ptr(),
                             self.arrive.data_ptr())

    # the qs_pages argument of the calls that take an optional one: none
    _pages_ref = None

    def nbytes(self):
        return sum(t.numel() * t.element_size() for t in
                   (self.k_upper, self.k_lower, self.v_upper, self.v_lower, self.meta,
                    self.buf_k, self.buf_v, self.state, self.arrive))


class PagedCache(Cache):
    """A cache whose groups lie in a pool of n_pages pages (include/qs.h,
    qs_pages): the group arrays are [n_pages, H, ...], ``table`` (int32 [B,
    cap_groups], filled with -1) names the page of each sequence's groups and
    is the caller's to fill or to replace.  The calls for contiguous caches
    refuse it."""

    def __init__(self, B, H, cap_groups, n_pages, device="cuda", D=128, G=128, upper_bits=4):
        import torch
        qs_cache_bytes(B, H, cap_groups, D, G)  # validates the sizes
        qs_paged_cache_bytes(B, H, n_pages, D, G)
        self.n_pages = n_pages
        self._alloc(B, H, cap_groups, device, D, G, upper_bits, (n_pages, H))
        self.pages_struct = QsPagesStruct(None, n_pages)
        self._pages_ref = ctypes.byref(self.pages_struct)
        self.table = torch.full((B, cap_groups), -1, dtype=torch.int32, device=device)
        self.struct = self._struct(upper_bits | QS_PAGED)
        self._ref = ctypes.byref(self.struct)

    @property
    def table(self):
        """The page table: write into it, or assign another int32 [B,
        cap_groups] tensor (a captured graph keeps the one it was captured
        with)."""
        return self._table

    @table.setter
    def table(self, t):
        if (t.dtype != self.state.dtype or t.device != self.state.device or
                tuple(t.shape) != (self.B, self.cap) or not t.is_contiguous()):
            raise ValueError("the page table is a contiguous int32 [%d, %d] tensor on %s"
                             % (self.B, self.cap, self.state.device))
        self._table = t
        self.pages_struct.table = t.data_ptr()

    def nbytes(self):
        return super().nbytes() + self.table.numel() * self.table.element_size()


def qs_paged_cache_bytes(B, H, n_pages, D=128, G=128):
    out = QsCacheBytes()
    _check("qs_paged_cache_bytes", lib().qs_paged_cache_bytes(B, H, D, G, n_pages, ctypes.byref(out)))
    return {n: getattr(out, n) for n, _ in QsCacheBytes._fields_}


def qs_state_reset(cache, stream=None):
    _check("qs_state_reset", lib().qs_state_reset(cache._ref, _stream(stream)))


def qs_buffer_append(cache, k_new, v_new, stream=None):
    """k_new, v_new: fp16 [B, H, n_new, D] contiguous device tensors."""
    assert k_new.is_contiguous() and v_new.is_contiguous() and k_new.shape == v_new.shape
    n_new = k_new.shape[2]
    _check("qs_buffer_append", lib().qs_buffer_append(cache._ref, _ptr(k_new), _ptr(v_new),
                                                      n_new, _stream(stream)))


def qs_buffer_rollback(cache, n_drop, stream=None):
    """n_drop: int32 [B] device tensor."""
    _check("qs_buffer_rollback", lib().qs_buffer_rollback(cache._ref, _ptr(n_drop), _stream(stream)))


def qs_need_flush(cache, n_next, mask, stream=None):
    """mask: uint8 [B] device tensor (written)."""
    _check("qs_need_flush", lib().qs_need_flush(cache._ref, int(n_next), _ptr(mask), _stream(stream)))


def qs_quantize_flush(cache, mask=None, stream=None):
    """mask: uint8 [B] device tensor or None (every sequence)."""
    _check("qs_quantize_flush", lib().qs_quantize_flush(cache._ref, _ptr(mask), _stream(stream)))


def qs_quantize_flush_due(cache, n_next, stream=None):
    """Flush every sequence whose buffer cannot take n_next more tokens."""
    _check("qs_quantize_flush_due", lib().qs_quantize_flush_due(cache._ref, int(n_next),
                                                                _stream(stream)))


def qs_prefill(cache, k, v, lens, stream=None):
    """k, v: fp16 [B, H, T, D] contiguous device tensors; lens: int32 [B]
    device tensor of prompt lengths."""
    assert k.is_contiguous() and v.is_contiguous() and k.shape == v.shape
    _check("qs_prefill", lib().qs_prefill(cache._ref, _ptr(k), _ptr(v), int(k.shape[2]), _ptr(lens),
                                          _stream(stream)))


def qs_quantize_flush_paged(cache, mask=None, stream=None):
    """qs_quantize_flush on a PagedCache."""
    if mask is not None and not (mask.numel() == cache.B and mask.element_size() == 1 and
                                 mask.is_contiguous() and mask.get_device() == cache._dev):
        raise QsArgumentError("mask: uint8 [B] on the cache's device")
    _check("qs_quantize_flush_paged", lib().qs_quantize_flush_paged(
        cache._ref, cache._pages_ref, _ptr(mask), _stream(stream)))


def qs_quantize_flush_due_paged(cache, n_next, stream=None):
    """qs_quantize_flush_due on a PagedCache."""
    _check("qs_quantize_flush_due_paged", lib().qs_quantize_flush_due_paged(
        cache._ref, cache._pages_ref, int(n_next), _stream(stream)))


def _check_f16(cache, t, name):
    if not (t.dtype is cache._f16 and t.is_contiguous() and t.get_device() == cache._dev):
        raise QsArgumentError("%s: contiguous float16 on the cache's device" % name)


def qs_prefill_paged(cache, k, v, lens, stream=None):
    """qs_prefill on a PagedCache."""
    if k is None or v is None or not (k.shape == v.shape and k.dim() == 4 and
                                      k.shape[:2] == (cache.B, cache.H) and k.shape[3] == cache.D):
        raise QsArgumentError("k, v: [B, H, T, D]")
    _check_f16(cache, k, "k")
    _check_f16(cache, v, "v")
    if not (lens.numel() == cache.B and lens.dtype is cache._i32 and lens.is_contiguous() and
            lens.get_device() == cache._dev):
        raise QsArgumentError("lens: int32 [B] on the cache's device")
    _check("qs_prefill_paged", lib().qs_prefill_paged(cache._ref, cache._pages_ref, _ptr(k), _ptr(v),
                                                      int(k.shape[2]), _ptr(lens), _stream(stream)))


def qs_cache_read(cache, mode, k, v, tok0=0, stream=None):
    """Tokens [tok0, tok0 + T) of each sequence as fp16 rows into k, v: fp16
    [B, H, T, D] contiguous device tensors, one of them may be None.  Rows past
    a sequence's last token stay as they were."""
    shape = () if k is None and v is None else (v if k is None else k).shape
    T = shape[2] if len(shape) == 4 else 0
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            if t.shape != (cache.B, cache.H, T, cache.D):
                raise QsArgumentError("%s: [B, H, T, D]" % name)
            _check_f16(cache, t, name)
    _check("qs_cache_read", lib().qs_cache_read(cache._ref, cache._pages_ref, int(mode), int(tok0),
                                                int(T), _ptr(k), _ptr(v), _stream(stream)))


def qs_spec_accept(p, q, draft, u, e, n_accept, token, n_drop, stream=None):
    """p [B, g+1, V], q [B, g, V], u [B, g], e [B, V]: float32 device tensors;
    draft [B, g] int32; outputs n_accept, token, n_drop: int32 [B] tensors."""
    B, g1, V = p.shape
    for t in (p, q, draft, u, e):
        assert t.is_contiguous()
    _check("qs_spec_accept", lib().qs_spec_accept(_ptr(p), _ptr(q), _ptr(draft), _ptr(u), _ptr(e), B,
                                                  g1 - 1, V, _ptr(n_accept), _ptr(token),
                                                  _ptr(n_drop), _stream(stream)))


def qs_attn_workspace_size(cache, n_q):
    n = ctypes.c_size_t()
    _check("qs_attn_workspace_size", lib().qs_attn_workspace_size(cache._ref, int(n_q), ctypes.byref(n)))
    return n.value


def qs_attn_decode(cache, mode, q, softmax_scale, out, lse=None, workspace=None, stream=None):
    """q, out: fp16 [B, H, n_q, D]; lse: float32 [B, H, n_q] or None;
    workspace: a uint8 device tensor of at least qs_attn_workspace_size bytes."""
    n_q = q.shape[2]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("qs_attn_decode", lib().qs_attn_decode(
        cache._ref, int(mode), _ptr(q), n_q, float(softmax_scale), _ptr(out), _ptr(lse),
        _ptr(workspace), ws_bytes, _stream(stream)))


def qs_attn_workspace_size_gqa(cache, n_q, group):
    n = ctypes.c_size_t()
    _check("qs_attn_workspace_size_gqa", lib().qs_attn_workspace_size_gqa(
        cache._ref, int(n_q), int(group), ctypes.byref(n)))
    return n.value


def qs_attn_decode_gqa(cache, mode, q, group, softmax_scale, out, lse=None, workspace=None,
                       stream=None):
    """q, out: fp16 [B, H*group, n_q, D]; lse: float32 [B, H*group, n_q] or None."""
    n_q = q.shape[2]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("qs_attn_decode_gqa", lib().qs_attn_decode_gqa(
        cache._ref, int(mode), _ptr(q), n_q, int(group), float(softmax_scale), _ptr(out), _ptr(lse),
        _ptr(workspace), ws_bytes, _stream(stream)))


def qs_attn_decode_static_ws(cache, mode, q, softmax_scale, out, lse=None, stream=None):
    """qs_attn_decode with its scratch in the library's fixed device array
    (for callers that cannot allocate device memory); q, out, lse as for
    qs_attn_decode.  Returns the status instead of raising on
    QS_ERR_TOO_LARGE, so a caller can fall back to the allocating call."""
    n_q = q.shape[2]
    status = lib().qs_attn_decode_static_ws(cache._ref, int(mode), _ptr(q), n_q,
                                            float(softmax_scale), _ptr(out), _ptr(lse),
                                            _stream(stream))
    if status != QS_ERR_TOO_LARGE:
        _check("qs_attn_decode_static_ws", status)
    return status


def qs_attn_decode_append(cache, mode, k_new, v_new, q, softmax_scale, out, lse=None,
                          workspace=None, group=1, stream=None):
    """qs_buffer_append(k_new, v_new) then qs_attn_decode(_gqa), one launch.
    k_new, v_new: fp16 [B, H, n_new, D]; q, out: fp16 [B, H*group, n_q, D]."""
    assert k_new.is_contiguous() and v_new.is_contiguous() and k_new.shape == v_new.shape
    n_q = q.shape[2]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("qs_attn_decode_append", lib().qs_attn_decode_append(
        cache._ref, int(mode), _ptr(k_new), _ptr(v_new), k_new.shape[2], _ptr(q), n_q, int(group),
        float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, _stream(stream)))


def _n_new(cache, k_new, v_new):
    """The appended tokens: k_new and v_new fp16 [B, H, n_new, D], or neither."""
    if k_new is None and v_new is None:
        return 0
    if k_new is None or v_new is None:
        raise QsArgumentError("k_new and v_new go together")
    shape = k_new.shape
    if not (len(shape) == 4 and v_new.shape == shape and shape[0] == cache.B and
            shape[1] == cache.H and shape[3] == cache.D):
        raise QsArgumentError("k_new, v_new: [B, H, n_new, D]")
    _check_f16(cache, k_new, "k_new")
    _check_f16(cache, v_new, "v_new")
    return shape[2]


def _check_queries(cache, q, group, out=None, lse=None):
    """q (and out) fp16 [B, H * group, n_q, D] contiguous, lse fp32 of the rows."""
    shape = q.shape
    if len(shape) != 4:
        raise QsArgumentError("q: [B, H * group, n_q, D]")
    b, h, n_q, d = shape
    if b != cache.B or h != cache.H * group or d != cache.D:
        raise QsArgumentError("q: [B, H * group, n_q, D]")
    _check_f16(cache, q, "q")
    if out is not None:
        if out.shape != shape:
            raise QsArgumentError("out: the shape of q")
        _check_f16(cache, out, "out")
    if lse is not None and not (lse.numel() == b * h * n_q and lse.dtype is cache._f32 and
                                lse.is_contiguous() and lse.get_device() == cache._dev):
        raise QsArgumentError("lse: contiguous float32 [B, H * group, n_q] on the cache's device")
    return n_q


def _ws_bytes(cache, workspace):
    if workspace is None:
        return 0
    if not workspace.is_contiguous() or workspace.get_device() != cache._dev:
        raise QsArgumentError("workspace: contiguous, on the cache's device")
    return workspace.nbytes


def _check_selection(cache, sel):
    """sel: int32 [B, H, k] contiguous."""
    shape = sel.shape
    if not (len(shape) == 3 and shape[0] == cache.B and shape[1] == cache.H and
            sel.dtype is cache._i32 and sel.is_contiguous() and sel.get_device() == cache._dev):
        raise QsArgumentError("sel: contiguous int32 [B, H, k] on the cache's device")
    return shape[2]


def qs_attn_decode_paged(cache, mode, q, softmax_scale, out, lse=None, workspace=None, group=1,
                         k_new=None, v_new=None, stream=None):
    """qs_attn_decode_gqa on a PagedCache, or with k_new, v_new (fp16 [B, H,
    n_new, D]) qs_attn_decode_append on it."""
    n_q = _check_queries(cache, q, group, out, lse)
    ws_bytes = _ws_bytes(cache, workspace)
    _check("qs_attn_decode_paged", lib().qs_attn_decode_paged(
        cache._ref, cache._pages_ref, int(mode), _ptr(k_new), _ptr(v_new), _n_new(cache, k_new, v_new),
        _ptr(q), n_q, int(group), float(softmax_scale), _ptr(out), _ptr(lse),
        _ptr(workspace), ws_bytes, _stream(stream)))


def qs_select_groups(cache, q, sel, group=1, stream=None):
    """For each KV head the sel.shape[2] groups whose keys could score highest
    against q (fp16 [B, H*group, n_q, D]) into sel, int32 [B, H, k]."""
    n_q, k = _check_queries(cache, q, group), _check_selection(cache, sel)
    _check("qs_select_groups", lib().qs_select_groups(
        cache._ref, cache._pages_ref, _ptr(q), n_q, int(group), k, _ptr(sel),
        _stream(stream)))


def qs_attn_decode_sparse(cache, mode, sel, q, softmax_scale, out, lse=None, workspace=None, group=1,
                          k_new=None, v_new=None, stream=None):
    """Decode attention (cache: a Cache or a PagedCache) over the groups named
    in sel, int32 [B, H, k] (-1: none), and the buffer; k_new, v_new as for
    qs_attn_decode_paged."""
    n_q, k = _check_queries(cache, q, group, out, lse), _check_selection(cache, sel)
    ws_bytes = _ws_bytes(cache, workspace)
    _check("qs_attn_decode_sparse", lib().qs_attn_decode_sparse(
        cache._ref, cache._pages_ref, int(mode), _ptr(sel), k, _ptr(k_new), _ptr(v_new),
        _n_new(cache, k_new, v_new), _ptr(q), n_q, int(group), float(softmax_scale), _ptr(out),
        _ptr(lse), _ptr(workspace), ws_bytes, _stream(stream)))


# ------------------------------------- a round over a tree of drafted tokens

_get_device = None


def _current_device():
    global _get_device
    if _get_device is None:
        import torch
        raw = getattr(torch._C, "_cuda_getDevice", None)
        torch.cuda.init()
        _get_device = raw or torch.cuda.current_device
    return _get_device()


def _check_device(dev):
    """The library launches on the current device."""
    if dev >= 0 and dev != _current_device():
        raise QsArgumentError("the tensors lie on cuda:%d, which is not the current device" % dev)


def _rows(cache, t, name, heads, n):
    """The numbers of a qs_rows: fp16 [B, heads, n, D] with any strides, the last
    one 1."""
    shape = t.shape
    if shape != (cache.B, heads, n, cache.D) or t.dtype is not cache._f16 or t.get_device() != cache._dev:
        raise QsArgumentError("%s: float16 [%d, %d, %d, %d] on the cache's device"
                              % (name, cache.B, heads, n, cache.D))
    b, h, t_, d = t.stride()
    if d != 1:
        raise QsArgumentError("%s: the elements of a row lie side by side" % name)
    # (the stride of a dimension of one is of no account)
    return t.data_ptr(), b if cache.B > 1 else 0, h if heads > 1 else 0, t_ if n > 1 else 0


_THREE_ROWS = ctypes.c_int64 * 12


def qs_buffer_append_rotary(cache, k, v, inv_freq, q=None, q_out=None, offset=None, interleaved=False,
                            stream=None):
    """qs_buffer_append with the position rotation.  k, v: fp16 [B, H, n, D], q:
    fp16 [B, H * group, n, D] or None, all with any strides but the last (slices
    of a projection's output, say); q_out: contiguous, the shape of q; inv_freq:
    float32 [rot / 2]; offset: int32 [B, n] or None."""
    _check_device(cache._dev)
    n = k.shape[2] if k.dim() == 4 else 0
    group, q_rows = 1, (0, 0, 0, 0)
    if q is not None and q_out is not None:
        group = q.shape[1] // cache.H if q.dim() == 4 else 0
        q_rows = _rows(cache, q, "q", cache.H * group, n)
        if q_out.shape != q.shape:
            raise QsArgumentError("q_out: the shape of q")
        _check_f16(cache, q_out, "q_out")
    elif q is not None or q_out is not None:
        raise QsArgumentError("q and q_out go together")
    rows = _THREE_ROWS(*_rows(cache, k, "k", cache.H, n), *_rows(cache, v, "v", cache.H, n), *q_rows)
    if not (inv_freq.dim() == 1 and inv_freq.dtype is cache._f32 and inv_freq.is_contiguous() and
            inv_freq.get_device() == cache._dev):
        raise QsArgumentError("inv_freq: contiguous float32 [rot / 2] on the cache's device")
    if offset is not None:
        _check_i32(cache, offset, "offset", (cache.B, n))
    at = ctypes.addressof(rows)
    _check("qs_buffer_append_rotary", lib().qs_buffer_append_rotary(
        cache._ref, at, at + 32, None if q is None else at + 64, _ptr(q_out), group, n, _ptr(offset),
        _ptr(inv_freq), 2 * inv_freq.shape[0], 1 if interleaved else 0, _stream(stream)))


def _check_i32(cache, t, name, shape):
    if not (t.shape == shape and t.dtype is cache._i32 and t.is_contiguous() and
            t.get_device() == cache._dev):
        raise QsArgumentError("%s: contiguous int32 %s on the cache's device" % (name, list(shape)))


def qs_attn_tree_workspace_size(cache, n_q, group=1):
    n = ctypes.c_size_t()
    _check("qs_attn_tree_workspace_size", lib().qs_attn_tree_workspace_size(
        cache._ref, int(n_q), int(group), ctypes.byref(n)))
    return n.value


def qs_attn_decode_tree(cache, mode, parent, q, softmax_scale, out, lse=None, workspace=None, group=1,
                        stream=None):
    """Decode attention (cache: a Cache or a PagedCache) of the last n_q nodes of
    a tree, parent int32 [B, n_tree]; q, out: fp16 [B, H * group, n_q, D]."""
    _check_device(cache._dev)
    n_q = _check_queries(cache, q, group, out, lse)
    n_tree = parent.shape[1] if parent.dim() == 2 else 0
    _check_i32(cache, parent, "parent", (cache.B, n_tree))
    ws_bytes = _ws_bytes(cache, workspace)
    _check("qs_attn_decode_tree", lib().qs_attn_decode_tree(
        cache._ref, cache._pages_ref, int(mode), _ptr(parent), n_tree, _ptr(q), n_q, int(group),
        float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, _stream(stream)))


def qs_tree_accept(cache, parent, draft, target, n_keep, path, emitted, stream=None):
    """parent, draft, target, and the outputs path, emitted: int32 [B, n_tree];
    n_keep (out): int32 [B]."""
    _check_device(cache._dev)
    n_tree = parent.shape[1] if parent.dim() == 2 else 0
    for name, t in (("parent", parent), ("draft", draft), ("target", target), ("path", path),
                    ("emitted", emitted)):
        _check_i32(cache, t, name, (cache.B, n_tree))
    _check_i32(cache, n_keep, "n_keep", (cache.B,))
    _check("qs_tree_accept", lib().qs_tree_accept(
        cache._ref, _ptr(parent), _ptr(draft), _ptr(target), n_tree, _ptr(n_keep), _ptr(path),
        _ptr(emitted), _stream(stream)))


_logit_types = {}


def _sample_types():
    import torch
    if not _logit_types:
        _logit_types.update({torch.float16: QS_FP16, torch.bfloat16: QS_BF16, torch.float32: QS_FP32})
    return torch.float32, torch.int32


def _check_row(t, name, dtype, shape, dev):
    if not (t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == dev):
        raise QsArgumentError("%s: contiguous %s %s on the logits' device" % (name, dtype, list(shape)))


def qs_sample(logits, u, token, probs=None, temperature=None, top_k=None, top_p=None, min_p=None,
              stream=None):
    """A token (int32 [rows]) for each row of logits, fp16, bf16 or fp32
    [rows, V] with any row stride, by u, float32 [rows]; probs: float32 [rows, V]
    or None; temperature, top_p, min_p: float32 [rows], top_k: int32 [rows], or
    None."""
    f32, i32 = _sample_types()
    kind = _logit_types.get(logits.dtype)
    if logits.dim() != 2 or kind is None:
        raise QsArgumentError("logits: fp16, bf16 or fp32 [rows, V]")
    rows, V = logits.shape
    dev = logits.get_device()
    if dev < 0:
        raise QsArgumentError("logits: on a CUDA device")
    _check_device(dev)
    row, step = logits.stride()
    if step != 1 and V > 1:
        raise QsArgumentError("logits: the elements of a row lie side by side")
    _check_row(u, "u", f32, (rows,), dev)
    _check_row(token, "token", i32, (rows,), dev)
    if probs is not None:
        _check_row(probs, "probs", f32, (rows, V), dev)
    if temperature is not None:
        _check_row(temperature, "temperature", f32, (rows,), dev)
    if top_k is not None:
        _check_row(top_k, "top_k", i32, (rows,), dev)
    if top_p is not None:
        _check_row(top_p, "top_p", f32, (rows,), dev)
    if min_p is not None:
        _check_row(min_p, "min_p", f32, (rows,), dev)
    _check("qs_sample", lib().qs_sample(
        _ptr(logits), kind, rows, V, row if rows > 1 else V,
        _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p), _ptr(u), _ptr(token), _ptr(probs),
        _stream(stream)))


def qs_get_errors(cache, stream=None):
    """Per-sequence error words (numpy int32 [B]); clears them on the device."""
    h = np.zeros(cache.B, np.int32)
    _check("qs_get_errors", lib().qs_get_errors(cache._ref, h.ctypes.data_as(ctypes.c_void_p),
                                                _stream(stream)))
    return h
