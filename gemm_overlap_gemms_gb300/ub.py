"""ctypes binding of libubgemm (include/ub.h): argument marshalling only.

Every step of the AG-GEMM and GEMM-RS path runs in the library's kernels and copy
engine calls; this module checks tensor dtypes, devices and shapes, passes raw
device pointers and the current CUDA stream, and turns error codes into exceptions.
There is no fallback: if ``libubgemm.so`` is missing, the first call raises.

API modelled on "Support dynamic token counts in TP communication/GEMM overlap"
(TransformerEngine issue #3564), "Proposed API": ``initialize_ub([max_tokens,
hidden], tp_size, dtype=torch.bfloat16)`` registers a buffer at capacity, and
``set_ub_active_shape([T, hidden])`` sets the active shape before each microbatch.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libubgemm.so")
_lib = None

UB_OK = 0
ERRORS = {
    -1: "UB_ERR_ARG", -2: "UB_ERR_DTYPE", -3: "UB_ERR_RANK", -4: "UB_ERR_ZERO",
    -5: "UB_ERR_CAPACITY", -6: "UB_ERR_HIDDEN", -7: "UB_ERR_DIVISIBLE", -8: "UB_ERR_ALIGN",
    -9: "UB_ERR_CUDA", -10: "UB_ERR_TIMEOUT",
}
CODES = {v: k for k, v in ERRORS.items()}
OPTIONS = {"sm_margin": 1, "timeout_ns": 2, "self_rank": 3, "drop_flag": 4, "profile": 5,
           "cta_pair": 6, "streamk": 7, "copy_streams": 8, "gather_kernel": 9, "skinny": 10, "pdl": 11,
           "bulk_beside": 12, "gather_chain": 13}
OPS = {"ag": 0, "rs": 1, "ag_swiglu": 2, "ag_kn": 3, "rs_kn": 4, "wgrad": 5, "reduce_scatter": 6, "kv_append": 7,
       "attn_prompt": 8, "attn_decode": 9, "attn_tree": 10, "kv_accept": 11, "kv_pages": 12, "kv_copy": 13}
MAX_TP = 8
EXPORTS = [
    "ub_create", "ub_destroy", "ub_set_active_shape", "ub_set_active_shape_nd",
    "ub_validate_active_shape", "ub_get_active_shape", "ub_get_capacity", "ub_get_tp",
    "ub_buffer", "ag_gemm", "gemm_rs", "ub_set_option", "ub_get_option", "ub_query_status",
    "ub_clear_status", "ub_get_counters", "ub_kernel_time", "ub_grid_ctas", "ub_last_error",
    "ag_gemm_noalloc", "ag_gemm_swiglu", "ag_gemm_kn", "gemm_rs_kn", "ub_wgrad",
    "ub_allgather", "ub_reduce_scatter", "ub_plan_tail_split", "ub_plan_path",
    "ub_plan_ag_self_head", "ag_gemm_from_buffer", "ub_plan_gather_parts", "ub_stream_read",
    "ub_plan_ag_group_m", "ub_kv_append", "ub_attn_prompt", "ub_attn_decode",
    "ub_attn_prompt_window", "ub_attn_decode_window", "ub_kv_append_tree", "ub_attn_tree", "ub_kv_accept",
    "ub_kv_take", "ub_kv_free", "ub_kv_fork", "ub_kv_compact", "ub_kv_copy",
]
NOALLOC_MAX_ELEMS = 16 * 1024 * 1024
ACCEPT_MOST = 2048  # drafts of a sequence in kv_accept


class UbError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("%s (%d): %s" % (ERRORS.get(code, "UB_ERR?"), code, msg))
        self.code = code
        self.name = ERRORS.get(code, "UB_ERR?")


class Counters(ctypes.Structure):
    _fields_ = [("ag_calls", ctypes.c_int64), ("rs_calls", ctypes.c_int64),
                ("device_allocations", ctypes.c_int64), ("last_T", ctypes.c_int64),
                ("tensor_map_encodes", ctypes.c_int64), ("last_kernel", ctypes.c_int64),
                ("last_pieces", ctypes.c_int64), ("last_gather", ctypes.c_int64)]


KERNELS = {0: "single", 1: "pair", 2: "few_token"}
GATHERS = {-1: "none", 0: "copies", 1: "gather_kernel", 2: "in_gemm"}


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load libubgemm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError("libubgemm.so is not built (%s); run __graft_entry__.build()" % _LIB_PATH)
    L = ctypes.CDLL(_LIB_PATH)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    PP = ctypes.POINTER(ctypes.c_void_p)
    sig = {
        "ub_create": [I64, I64, I, I, ctypes.POINTER(P)],
        "ub_destroy": [P],
        "ub_set_active_shape": [P, I64, I64],
        "ub_set_active_shape_nd": [P, I, ctypes.POINTER(I64)],
        "ub_validate_active_shape": [I, ctypes.POINTER(I64), I64, I64, I],
        "ub_get_active_shape": [P, ctypes.POINTER(I64), ctypes.POINTER(I64)],
        "ub_get_capacity": [P, ctypes.POINTER(I64), ctypes.POINTER(I64)],
        "ub_get_tp": [P, ctypes.POINTER(I)],
        "ub_buffer": [P, PP, ctypes.POINTER(ctypes.c_size_t)],
        "ag_gemm": [P, PP, P, I64, P, P],
        "ag_gemm_swiglu": [P, PP, P, I64, P, P],
        "ag_gemm_kn": [P, PP, P, I64, P, P],
        "gemm_rs_kn": [P, PP, PP, I64, PP, P],
        "ub_wgrad": [P, P, I64, I, P, P],
        "ub_allgather": [P, PP, P],
        "ub_reduce_scatter": [P, PP, PP, P],
        "ub_stream_read": [P, P, I64, P],
        "gemm_rs": [P, PP, PP, I64, PP, P],
        "ub_set_option": [P, I, I64],
        "ub_get_option": [P, I, ctypes.POINTER(I64)],
        "ub_query_status": [P],
        "ub_clear_status": [P],
        "ub_get_counters": [P, ctypes.POINTER(Counters)],
        "ub_kernel_time": [P, I, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(I64)],
        "ub_grid_ctas": [P, ctypes.POINTER(I)],
        "ub_last_error": [],
        "ag_gemm_noalloc": [PP, I, I64, I64, P, I64, P, P],
        "ag_gemm_from_buffer": [P, P, I64, I64, P, P],
        "ub_plan_tail_split": [I64, I64, I64, I, I],
        "ub_plan_path": [I64, I64, I64, I64, I64, I, I, I, ctypes.POINTER(I), ctypes.POINTER(I)],
        "ub_plan_ag_self_head": [I64, I, I, I64, I64],
        "ub_plan_ag_group_m": [I64, I, I, I64, I64],
        "ub_kv_append": [P, ctypes.c_char_p, P],
        "ub_attn_prompt": [P, ctypes.c_char_p, P],
        "ub_attn_decode": [P, ctypes.c_char_p, P],
        "ub_attn_prompt_window": [P, ctypes.c_char_p, I, I, P],
        "ub_attn_decode_window": [P, ctypes.c_char_p, I, I, P],
        "ub_kv_append_tree": [P, ctypes.c_char_p, P, P],
        "ub_attn_tree": [P, ctypes.c_char_p, P, I, I, P],
        "ub_kv_accept": [P, ctypes.c_char_p, P, I64, P, P, P],
        "ub_kv_take": [P, ctypes.c_char_p, P, P, P],
        "ub_kv_free": [P, ctypes.c_char_p, P, P, P],
        "ub_kv_fork": [P, ctypes.c_char_p, P, P, I64, P, I64, P, P],
        "ub_kv_compact": [P, ctypes.c_char_p, P, P, I64, P, I64, P, P],
        "ub_kv_copy": [P, ctypes.c_char_p, P, I64, P],
        "ub_plan_gather_parts": [I, I, I64, I64, ctypes.POINTER(I), ctypes.POINTER(I64), ctypes.POINTER(I64),
                                 ctypes.POINTER(I)],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        if name == "ub_last_error":
            fn.restype = ctypes.c_char_p
        elif name in ("ub_plan_tail_split", "ub_plan_ag_self_head"):
            fn.restype = ctypes.c_int64
        else:
            fn.restype = ctypes.c_int
    _lib = L
    return L


def last_error() -> str:
    return load().ub_last_error().decode(errors="replace")


# ---------------------------------------------------------------- planning queries (host only)

def _plan_check(v: int) -> int:
    if v < 0:
        _check(int(v))
    return int(v)


def plan_tail_split(tiles: int, pairs: int, k_blocks: int, widest: bool = False, gathered: bool = False) -> int:
    """k-pieces per tile of the CTA-pair kernel's last, partial wave (1: whole tiles);
    `gathered` for an AG-GEMM whose rows come through the all-gather."""
    return _plan_check(load().ub_plan_tail_split(tiles, pairs, k_blocks, 1 if widest else 0, 1 if gathered else 0))


def plan_path(single_tiles: int, pair_tiles: int, k_blocks: int, slots: int, pairs: int,
              cta_pair: int = -1, streamk: int = -1, gathered: bool = False) -> tuple:
    """(pair, split) for a tile-kernel call: CTA pairs or single CTAs, split last wave."""
    pr, sp = ctypes.c_int(0), ctypes.c_int(0)
    rc = load().ub_plan_path(single_tiles, pair_tiles, k_blocks, slots, pairs, cta_pair, streamk,
                             1 if gathered else 0, ctypes.byref(pr), ctypes.byref(sp))
    _check(rc)
    return bool(pr.value), bool(sp.value)


def plan_gather_parts(tp: int, self_rank: int, c: int, head: int) -> list:
    """The gather's copies in issue order: (chunk, row_lo, row_hi, publishes_flag)."""
    n_max = MAX_TP + 1
    ch = (ctypes.c_int * n_max)()
    lo = (ctypes.c_int64 * n_max)()
    hi = (ctypes.c_int64 * n_max)()
    fl = (ctypes.c_int * n_max)()
    n = load().ub_plan_gather_parts(tp, self_rank, c, head, ch, lo, hi, fl)
    if n < 0:
        _check(n)
    return [(ch[i], lo[i], hi[i], bool(fl[i])) for i in range(n)]


def plan_ag_self_head(T: int, tp: int, self_rank: int, n_tiles: int, pairs: int) -> int:
    """Rows of the self chunk the CTA-pair AG kernel reads in place."""
    return _plan_check(load().ub_plan_ag_self_head(T, tp, self_rank, n_tiles, pairs))


def plan_ag_group_m(T: int, tp: int, self_rank: int, n_tiles: int, pairs: int) -> int:
    """Tile rows per group of a CTA-pair AG call's tile order (0: N fastest)."""
    return _plan_check(load().ub_plan_ag_group_m(T, tp, self_rank, n_tiles, pairs))


def _check(rc: int):
    if rc != UB_OK:
        raise UbError(rc, last_error())
    return rc


def validate_active_shape(shape, max_tokens: int, hidden: int, tp: int) -> int:
    """UB_OK or the UB_ERR_* code of the first violated active-shape constraint."""
    dims = (ctypes.c_int64 * max(1, len(shape)))(*[int(d) for d in shape])
    return load().ub_validate_active_shape(len(shape), dims, max_tokens, hidden, tp)


def _stream_ptr(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptrs(tensors):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _bf16_cuda(t: torch.Tensor, name: str, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError("%s must be a CUDA bfloat16 tensor, got %s on %s" % (name, t.dtype, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the user buffer on %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


# ub_attn_t of include/ub.h, packed by one struct call instead of a ctypes structure (a
# decoding step's call takes microseconds): 8 ints, scale, reserved, 4 sizes, four
# [data, row, head], two [data, page, head, row], six pointers.
_ATTN = struct.Struct("=I7ifI4q" + "Q2q" * 4 + "Q3q" * 2 + "6Q")
# ub_pool_t: four ints, three sizes, two pointers.
_POOL = struct.Struct("=I2iI3q2Q")
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
# What a wrong argument raises while its view is read; the checks below are on the path of
# every decoding step, so each argument is read once and its faults are named afterwards.
_UNREADABLE = (AttributeError, TypeError, ValueError)


def _attn_error(t, name: str, dtype, device: int, what: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype or not t.is_cuda:
        raise TypeError("%s must be a CUDA %s tensor, got %s on %s" % (name, dtype, t.dtype, t.device))
    if t.get_device() != device:
        raise ValueError("%s is on %s, the user buffer on cuda:%d" % (name, t.device, device))
    raise ValueError("%s must be %s, got %s with strides %s" % (name, what, tuple(t.shape), t.stride()))


def _heads_view(t: torch.Tensor, name: str, T: int, D: int, device: int):
    """(data, row, head, heads) of a [T, heads, D] bf16 view with a contiguous head dimension."""
    try:
        n, heads, d = t.shape
        row, head, one = t.stride()
        if n == T and d == D and one == 1 and t.dtype is _BF16 and t.get_device() == device:
            return t.data_ptr(), row, head, heads
    except _UNREADABLE:
        pass
    _attn_error(t, name, _BF16, device, "[%d, heads, %d] with a contiguous last dimension" % (T, D))


def _head_dim(q) -> int:
    try:
        return q.shape[2]
    except (AttributeError, IndexError, TypeError):
        return -1  # no [T, heads, D] view: named by the check of q


def _pages_view(t: torch.Tensor, name: str, D: int, device: int):
    """(data, page, head, row, pages, kv_heads, page_size) of a cache."""
    try:
        pages, heads, size, d = t.shape
        page, head, row, one = t.stride()
        if d == D and one == 1 and t.dtype is _BF16 and t.get_device() == device:
            return t.data_ptr(), page, head, row, pages, heads, size
    except _UNREADABLE:
        pass
    _attn_error(t, name, _BF16, device, "[pages, kv_heads, page_size, %d] with a contiguous last dimension" % D)


def _caches(k_cache, v_cache, D: int, device: int):
    """(k data and strides, v data and strides, pages, kv_heads, page_size)."""
    kp, k0, k1, k2, pages, heads, size = _pages_view(k_cache, "k_cache", D, device)
    vp, v0, v1, v2, pages_v, heads_v, size_v = _pages_view(v_cache, "v_cache", D, device)
    if pages_v != pages or heads_v != heads or size_v != size:
        raise ValueError("v_cache has shape %s, k_cache %s" % (tuple(v_cache.shape), tuple(k_cache.shape)))
    return (kp, k0, k1, k2, vp, v0, v1, v2), pages, heads, size


def _ints(t: torch.Tensor, name: str, n: int | None, device: int):
    """(data, length) of a contiguous int32 vector (of n entries, if given)."""
    try:
        (length,) = t.shape
        if ((n is None or length == n) and (length < 2 or t.stride(0) == 1) and t.dtype is _I32
                and t.get_device() == device):
            return t.data_ptr(), length
    except _UNREADABLE:
        pass
    _attn_error(t, name, _I32, device, "[%s] and contiguous" % ("n" if n is None else n))


def _table(t: torch.Tensor, n: int, device: int, name: str = "page_table"):
    """(data, entries, row) of a page table."""
    try:
        rows, width = t.shape
        row, one = t.stride()
        if rows == n and (one == 1 or width < 2) and t.dtype is _I32 and t.get_device() == device:
            return t.data_ptr(), width, row
    except _UNREADABLE:
        pass
    _attn_error(t, name, _I32, device, "[%d, entries] with a contiguous last dimension" % n)


def _tall(t, name: str) -> int:
    """The rows of a table (what else is wrong with it _table says)."""
    try:
        return t.shape[0]
    except _UNREADABLE + (IndexError,):
        raise TypeError("%s must be a torch.Tensor [rows, entries]" % name) from None


def _pairs(t: torch.Tensor, name: str, n: int | None, device: int):
    """(data, pairs) of a contiguous int32 [pairs, 2]."""
    try:
        length, two = t.shape
        if two == 2 and (n is None or length == n) and t.is_contiguous() and t.dtype is _I32 and t.get_device() == device:
            return t.data_ptr(), length
    except _UNREADABLE:
        pass
    _attn_error(t, name, _I32, device, "[%s, 2] and contiguous" % ("n" if n is None else n))


def _sight(window, sinks) -> bool:
    """Whether a window is asked for; window and sinks are checked here, for struct and ctypes do not."""
    if window is None or window < 0 or sinks < 0 or window > 0x7fffffff or sinks > 0x7fffffff:
        raise ValueError("window %r, sinks %r: counts of tokens are needed (window 0: all)" % (window, sinks))
    return window > 0


def _rotations(t: torch.Tensor, name: str, shape, device: int):
    """(data, positions, rotated elements) of a table of cosines or sines."""
    try:
        positions, half = t.shape
        if (t.is_contiguous() and t.dtype is _F32 and t.get_device() == device
                and (shape is None or shape == (positions, half))):
            return t.data_ptr(), positions, 2 * half
    except _UNREADABLE:
        pass
    _attn_error(t, name, _F32, device, "[positions, rot / 2] and contiguous, cos like sin")


class _DeviceArray:
    """Exposes the registered buffer to torch through __cuda_array_interface__."""

    def __init__(self, owner, ptr: int, shape):
        self._owner = owner
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": "<i2",
                                         "data": (ptr, False), "version": 3, "strides": None}


class UserBuffer:
    """A user buffer registered at capacity [max_tokens, hidden] for tp virtual ranks."""

    def __init__(self, shape, tp_size: int, dtype=torch.bfloat16):
        if len(shape) != 2:
            raise UbError(CODES["UB_ERR_RANK"], "capacity shape must be [max_tokens, hidden]")
        if dtype != torch.bfloat16:
            raise UbError(CODES["UB_ERR_DTYPE"], "only torch.bfloat16 user buffers are supported")
        L = load()
        h = ctypes.c_void_p()
        _check(L.ub_create(int(shape[0]), int(shape[1]), int(tp_size), 0, ctypes.byref(h)))
        self._h = h
        self.max_tokens, self.hidden, self.tp = int(shape[0]), int(shape[1]), int(tp_size)
        self._active = None
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._dev = self.device.index

    # -- lifetime
    def close(self):
        if getattr(self, "_h", None):
            load().ub_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    # -- shapes
    def set_active_shape(self, shape):
        dims = (ctypes.c_int64 * max(1, len(shape)))(*[int(d) for d in shape])
        _check(load().ub_set_active_shape_nd(self._h, len(shape), dims))
        self._active = (int(shape[0]), int(shape[1]))

    @property
    def active_shape(self):
        """[T, hidden] as last set (kept on this side: every call reads it)."""
        if self._active is None:
            T, H = ctypes.c_int64(), ctypes.c_int64()
            _check(load().ub_get_active_shape(self._h, ctypes.byref(T), ctypes.byref(H)))
            self._active = (T.value, H.value)
        return self._active

    @property
    def capacity_shape(self):
        M, H = ctypes.c_int64(), ctypes.c_int64()
        _check(load().ub_get_capacity(self._h, ctypes.byref(M), ctypes.byref(H)))
        return (M.value, H.value)

    def buffer(self) -> torch.Tensor:
        """The whole registered buffer as a [max_tokens, hidden] bf16 CUDA tensor (a view)."""
        p = ctypes.c_void_p()
        n = ctypes.c_size_t()
        _check(load().ub_buffer(self._h, ctypes.byref(p), ctypes.byref(n)))
        arr = _DeviceArray(self, p.value, (self.max_tokens, self.hidden))
        return torch.as_tensor(arr, device=self.device).view(torch.bfloat16)

    def buffer_ptr(self) -> int:
        p = ctypes.c_void_p()
        _check(load().ub_buffer(self._h, ctypes.byref(p), None))
        return p.value

    # -- options / status
    def set_option(self, key: str, value: int):
        _check(load().ub_set_option(self._h, OPTIONS[key], int(value)))

    def get_option(self, key: str) -> int:
        v = ctypes.c_int64()
        _check(load().ub_get_option(self._h, OPTIONS[key], ctypes.byref(v)))
        return v.value

    def query_status(self) -> int:
        """Sticky device status (UB_OK or UB_ERR_*); synchronise the stream first."""
        return load().ub_query_status(self._h)

    def clear_status(self):
        _check(load().ub_clear_status(self._h))

    def counters(self) -> dict:
        c = Counters()
        _check(load().ub_get_counters(self._h, ctypes.byref(c)))
        return {f: getattr(c, f) for f, _ in Counters._fields_}

    def kernel_time(self, op: str):
        """(total_ms, launches) of the GEMM kernels of ``op`` since the last query
        (needs the ``profile`` option)."""
        ms, n = ctypes.c_double(), ctypes.c_int64()
        _check(load().ub_kernel_time(self._h, OPS[op], ctypes.byref(ms), ctypes.byref(n)))
        return ms.value, n.value

    def grid_ctas(self) -> int:
        g = ctypes.c_int()
        _check(load().ub_grid_ctas(self._h, ctypes.byref(g)))
        return g.value

    # -- the two operations
    def ag_gemm(self, shards, Wt: torch.Tensor, Y: torch.Tensor | None = None, stream=None):
        """Y[T, N] = concat_r(shards[r]) @ Wt.T; the gathered input stays in the buffer."""
        T, H = self.active_shape
        if len(shards) != self.tp:
            raise ValueError("expected %d shards, got %d" % (self.tp, len(shards)))
        c = T // self.tp
        for r, s in enumerate(shards):
            _bf16_cuda(s, "shards[%d]" % r, (c, H), device=self.device)
        _bf16_cuda(Wt, "Wt", device=self.device)
        if Wt.dim() != 2 or Wt.shape[1] != H:
            raise ValueError("Wt must be [N, %d], got %s" % (H, tuple(Wt.shape)))
        N = Wt.shape[0]
        if Y is None:
            Y = torch.empty((T, N), dtype=torch.bfloat16, device=Wt.device)
        _bf16_cuda(Y, "Y", device=self.device)
        if Y.dim() != 2 or Y.shape[0] < T or Y.shape[1] != N:
            raise ValueError("Y must be [>=%d, %d], got %s" % (T, N, tuple(Y.shape)))
        _check(load().ag_gemm(self._h, _ptrs(shards), ctypes.c_void_p(Wt.data_ptr()), N,
                              ctypes.c_void_p(Y.data_ptr()), _stream_ptr(stream)))
        return Y

    def ag_gemm_swiglu(self, shards, Wt: torch.Tensor, Z: torch.Tensor | None = None, stream=None):
        """Z[T, F] = silu(G @ Wt[:F].T) * (G @ Wt[F:].T), G = concat_r(shards[r]); Wt is
        [2F, hidden] with the gate rows first. The gathered input stays in the buffer."""
        T, H = self.active_shape
        if len(shards) != self.tp:
            raise ValueError("expected %d shards, got %d" % (self.tp, len(shards)))
        c = T // self.tp
        for r, s in enumerate(shards):
            _bf16_cuda(s, "shards[%d]" % r, (c, H), device=self.device)
        _bf16_cuda(Wt, "Wt", device=self.device)
        if Wt.dim() != 2 or Wt.shape[1] != H or Wt.shape[0] % 2:
            raise ValueError("Wt must be [2F, %d], got %s" % (H, tuple(Wt.shape)))
        F = Wt.shape[0] // 2
        if Z is None:
            Z = torch.empty((T, F), dtype=torch.bfloat16, device=Wt.device)
        _bf16_cuda(Z, "Z", device=self.device)
        if Z.dim() != 2 or Z.shape[0] < T or Z.shape[1] != F:
            raise ValueError("Z must be [>=%d, %d], got %s" % (T, F, tuple(Z.shape)))
        _check(load().ag_gemm_swiglu(self._h, _ptrs(shards), ctypes.c_void_p(Wt.data_ptr()), F,
                                     ctypes.c_void_p(Z.data_ptr()), _stream_ptr(stream)))
        return Z

    def ag_gemm_kn(self, shards, W: torch.Tensor, Y: torch.Tensor | None = None, stream=None):
        """Y[T, N] = concat_r(shards[r]) @ W with W stored [hidden, N] (e.g. the
        row-parallel input gradient dS @ Bt_j). The gathered input stays in the buffer."""
        T, H = self.active_shape
        if len(shards) != self.tp:
            raise ValueError("expected %d shards, got %d" % (self.tp, len(shards)))
        c = T // self.tp
        for r, s in enumerate(shards):
            _bf16_cuda(s, "shards[%d]" % r, (c, H), device=self.device)
        _bf16_cuda(W, "W", device=self.device)
        if W.dim() != 2 or W.shape[0] != H:
            raise ValueError("W must be [%d, N], got %s" % (H, tuple(W.shape)))
        N = W.shape[1]
        if Y is None:
            Y = torch.empty((T, N), dtype=torch.bfloat16, device=W.device)
        _bf16_cuda(Y, "Y", device=self.device)
        if Y.dim() != 2 or Y.shape[0] < T or Y.shape[1] != N:
            raise ValueError("Y must be [>=%d, %d], got %s" % (T, N, tuple(Y.shape)))
        _check(load().ag_gemm_kn(self._h, _ptrs(shards), ctypes.c_void_p(W.data_ptr()), N,
                                 ctypes.c_void_p(Y.data_ptr()), _stream_ptr(stream)))
        return Y

    def gemm_rs_kn(self, A, B, Y_shards=None, stream=None):
        """Y_shards[r] = rows [r*c, (r+1)*c) of sum_j A[j] @ B[j], B[j] stored [K, hidden]
        (e.g. the column-parallel input gradient sum_j dY_j @ Wt_j)."""
        T, H = self.active_shape
        if len(A) != self.tp or len(B) != self.tp:
            raise ValueError("expected %d A and B operands" % self.tp)
        K = A[0].shape[1] if A[0].dim() == 2 else -1
        for j in range(self.tp):
            _bf16_cuda(A[j], "A[%d]" % j, (T, K), device=self.device)
            _bf16_cuda(B[j], "B[%d]" % j, (K, H), device=self.device)
        c = T // self.tp
        if Y_shards is None:
            Y_shards = [torch.empty((c, H), dtype=torch.bfloat16, device=A[0].device)
                        for _ in range(self.tp)]
        for r, y in enumerate(Y_shards):
            _bf16_cuda(y, "Y_shards[%d]" % r, device=self.device)
            if y.dim() != 2 or y.shape[0] < c or y.shape[1] != H:
                raise ValueError("Y_shards[%d] must be [>=%d, %d]" % (r, c, H))
        _check(load().gemm_rs_kn(self._h, _ptrs(A), _ptrs(B), K, _ptrs(Y_shards),
                                 _stream_ptr(stream)))
        return Y_shards

    def wgrad(self, D: torch.Tensor, ub_is_a: bool = False, out: torch.Tensor | None = None,
              stream=None):
        """Weight gradient over the T active rows of the gathered buffer G:
        ub_is_a=False -> out [M, hidden] = D.T @ G; ub_is_a=True -> out [hidden, M] = G.T @ D."""
        T, H = self.active_shape
        _bf16_cuda(D, "D", device=self.device)
        if D.dim() != 2 or D.shape[0] != T:
            raise ValueError("D must be [%d, M], got %s" % (T, tuple(D.shape)))
        M = D.shape[1]
        shape = (H, M) if ub_is_a else (M, H)
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=D.device)
        _bf16_cuda(out, "out", shape, device=self.device)
        _check(load().ub_wgrad(self._h, ctypes.c_void_p(D.data_ptr()), M, int(bool(ub_is_a)),
                               ctypes.c_void_p(out.data_ptr()), _stream_ptr(stream)))
        return out

    def ag_gemm_from_buffer(self, Wt: torch.Tensor, Y: torch.Tensor | None = None, swiglu: bool = False,
                            stream=None):
        """Y[T, N] = UB[:T] @ Wt.T over the buffer as it stands (no gather, no flag wait);
        with swiglu, Wt is [2F, hidden] (gate rows first) and Y[T, F] = silu(gate) * up.
        The buffer must already hold the chunks: an allgather() of this active shape on
        this handle, ordered before this call (same stream, or an event)."""
        T, H = self.active_shape
        _bf16_cuda(Wt, "Wt", device=self.device)
        if Wt.dim() != 2 or Wt.shape[1] != H or (swiglu and Wt.shape[0] % 2):
            raise ValueError("Wt must be [%s, %d], got %s" % ("2F" if swiglu else "N", H, tuple(Wt.shape)))
        N = Wt.shape[0]
        n_out = N // 2 if swiglu else N
        if Y is None:
            Y = torch.empty((T, n_out), dtype=torch.bfloat16, device=Wt.device)
        _bf16_cuda(Y, "Y", device=self.device)
        if Y.dim() != 2 or Y.shape[0] < T or Y.shape[1] != n_out:
            raise ValueError("Y must be [>=%d, %d], got %s" % (T, n_out, tuple(Y.shape)))
        _check(load().ag_gemm_from_buffer(self._h, ctypes.c_void_p(Wt.data_ptr()), N, n_out if swiglu else 0,
                                          ctypes.c_void_p(Y.data_ptr()), _stream_ptr(stream)))
        return Y

    def allgather(self, shards, stream=None):
        """Bulk all-gather: UB[r*c + i] = shards[r][i] for the active shape, no GEMM."""
        T, H = self.active_shape
        if len(shards) != self.tp:
            raise ValueError("expected %d shards, got %d" % (self.tp, len(shards)))
        c = T // self.tp
        for r, s in enumerate(shards):
            _bf16_cuda(s, "shards[%d]" % r, (c, H), device=self.device)
        _check(load().ub_allgather(self._h, _ptrs(shards), _stream_ptr(stream)))

    def reduce_scatter(self, P, Y_shards=None, stream=None):
        """Bulk reduce-scatter: Y_shards[r] = rows [r*c, (r+1)*c) of sum_j P[j]."""
        T, H = self.active_shape
        if len(P) != self.tp:
            raise ValueError("expected %d partials" % self.tp)
        for j, x in enumerate(P):
            _bf16_cuda(x, "P[%d]" % j, (T, H), device=self.device)
        c = T // self.tp
        if Y_shards is None:
            Y_shards = [torch.empty((c, H), dtype=torch.bfloat16, device=P[0].device)
                        for _ in range(self.tp)]
        for r, y in enumerate(Y_shards):
            _bf16_cuda(y, "Y_shards[%d]" % r, device=self.device)
            if y.dim() != 2 or y.shape[0] < c or y.shape[1] != H:
                raise ValueError("Y_shards[%d] must be [>=%d, %d]" % (r, c, H))
        _check(load().ub_reduce_scatter(self._h, _ptrs(P), _ptrs(Y_shards), _stream_ptr(stream)))
        return Y_shards

    def stream_read(self, t: torch.Tensor, stream=None):
        """Read the bytes of contiguous CUDA tensor `t` once and discard them (ub_stream_read:
        the cost of one kernel reading them, the floor of a call whose work is that read)."""
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise TypeError("t must be a contiguous CUDA tensor")
        if t.device != self.device:
            raise ValueError("t is on %s, the user buffer on %s" % (t.device, self.device))
        _check(load().ub_stream_read(self._h, ctypes.c_void_p(t.data_ptr()), t.numel() * t.element_size(),
                                     _stream_ptr(stream)))

    def gemm_rs(self, A, Bt, Y_shards=None, stream=None):
        """Y_shards[r] = rows [r*c, (r+1)*c) of sum_j A[j] @ Bt[j].T (c = T / tp)."""
        T, H = self.active_shape
        if len(A) != self.tp or len(Bt) != self.tp:
            raise ValueError("expected %d A and Bt operands" % self.tp)
        K = A[0].shape[1] if A[0].dim() == 2 else -1
        for j in range(self.tp):
            _bf16_cuda(A[j], "A[%d]" % j, (T, K), device=self.device)
            _bf16_cuda(Bt[j], "Bt[%d]" % j, (H, K), device=self.device)
        c = T // self.tp
        if Y_shards is None:
            Y_shards = [torch.empty((c, H), dtype=torch.bfloat16, device=A[0].device)
                        for _ in range(self.tp)]
        if len(Y_shards) != self.tp:
            raise ValueError("expected %d output shards" % self.tp)
        for r, y in enumerate(Y_shards):
            _bf16_cuda(y, "Y_shards[%d]" % r, device=self.device)
            if y.dim() != 2 or y.shape[0] < c or y.shape[1] != H:
                raise ValueError("Y_shards[%d] must be [>=%d, %d]" % (r, c, H))
        _check(load().gemm_rs(self._h, _ptrs(A), _ptrs(Bt), K, _ptrs(Y_shards),
                              _stream_ptr(stream)))
        return Y_shards


    # -- attention between the QKV and the attention-out projections
    def _new(self, shape, dtype, stream):
        """A new tensor of the stream that the call runs on, so that its memory is not reused too early."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _raw_stream(self, stream) -> int:
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self._dev)
        return stream.cuda_stream

    def _out(self, out, name, T, H, D, stream):
        if out is None:
            out = self._new((T, H, D), _BF16, stream)
        data, row, head, heads = _heads_view(out, name, T, D, self._dev)
        if heads != H:
            raise ValueError("%s has %d heads, q has %d" % (name, heads, H))
        return out, data, row, head

    def _lse(self, lse, T, H, stream):
        """(lse, its pointer); True allocates it."""
        if lse is None or lse is False:
            return None, 0
        if lse is True:
            lse = self._new((T, H), _F32, stream)
        if (not isinstance(lse, torch.Tensor) or lse.dtype != _F32 or lse.device != self.device
                or tuple(lse.shape) != (T, H) or not lse.is_contiguous()):
            _attn_error(lse, "lse", _F32, self._dev, "(%d, %d) and contiguous" % (T, H))
        return lse, lse.data_ptr()

    def kv_append(self, q, k, v, cos, sin, seq_starts, kv_lens, page_table, k_cache, v_cache, q_out=None,
                  interleaved: bool = False, stream=None, parents=None):
        """Rotate q and k of the active tokens by their positions and store k and v in the paged
        cache (ub_kv_append). Returns the rotated queries.

        q [T, heads, D], k and v [T, kv_heads, D]: views of the QKV output, any token and head
        strides that are multiples of 8; D 64 or 128. cos, sin: fp32 [positions, rot / 2], rot a
        multiple of 16 up to D (None: no rotation). seq_starts int32 [n + 1], kv_lens int32 [n]
        (the tokens of this call included), page_table int32 [n, entries], on the device.
        k_cache, v_cache [pages, kv_heads, page_size, D]. q_out: like q, q itself allowed.
        parents: int32 [T], the tokens are drafts (ub_kv_append_tree; see attn_tree), each rotated
        by its position along its path."""
        dev = self._dev
        T, _ = self._active or self.active_shape
        D = _head_dim(q)
        qp, q0, q1, H = _heads_view(q, "q", T, D, dev)
        kp, k0, k1, G = _heads_view(k, "k", T, D, dev)
        vp, v0, v1, Gv = _heads_view(v, "v", T, D, dev)
        caches, pages, Gc, page = _caches(k_cache, v_cache, D, dev)
        if Gv != G or Gc != G:
            raise ValueError("k has %d heads, v %d, the caches %d" % (G, Gv, Gc))
        lens, n = _ints(kv_lens, "kv_lens", None, dev)
        starts, _ = _ints(seq_starts, "seq_starts", n + 1, dev)
        table, width, table_row = _table(page_table, n, dev)
        rot = positions = cp = sp = 0
        if cos is not None or sin is not None:
            cp, positions, rot = _rotations(cos, "cos", None, dev)
            sp, _, _ = _rotations(sin, "sin", (positions, rot // 2), dev)
        q_out, op, o0, o1 = self._out(q_out, "q_out", T, H, D, stream)
        a = _ATTN.pack(_ATTN.size, n, H, G, D, page, rot, 1 if interleaved else 0, 1.0, 0, pages, width, table_row,
                       positions, qp, q0, q1, kp, k0, k1, vp, v0, v1, op, o0, o1, *caches, starts, lens, table, cp, sp, 0)
        if parents is None:
            rc = (_lib or load()).ub_kv_append(self._h, a, self._raw_stream(stream))
        else:
            rc = (_lib or load()).ub_kv_append_tree(self._h, a, _ints(parents, "parents", T, dev)[0], self._raw_stream(stream))
        if rc:
            _check(rc)
        return q_out

    def attn_prompt(self, q, k, v, seq_starts, out=None, lse=None, scale: float | None = None, stream=None,
                    window: int = 0, sinks: int = 0):
        """Causal attention of whole packed prompts (ub_attn_prompt): sequence s is rows
        [seq_starts[s], seq_starts[s + 1]) of q [T, heads, D] and of k, v [T, kv_heads, D].
        scale: 1 / sqrt(D) if None. lse: an fp32 [T, heads] tensor, or True for a new one.
        Returns out, or (out, lse) where lse is asked for. Rows of no sequence stay as they are.
        window > 0: a token sees the last `window` tokens, itself included, and the first `sinks`
        of its sequence (ub_attn_prompt_window)."""
        near = _sight(window, sinks)
        dev = self._dev
        T, _ = self._active or self.active_shape
        D = _head_dim(q)
        qp, q0, q1, H = _heads_view(q, "q", T, D, dev)
        kp, k0, k1, G = _heads_view(k, "k", T, D, dev)
        vp, v0, v1, Gv = _heads_view(v, "v", T, D, dev)
        if Gv != G:
            raise ValueError("k has %d heads, v %d" % (G, Gv))
        starts, n = _ints(seq_starts, "seq_starts", None, dev)
        out, op, o0, o1 = self._out(out, "out", T, H, D, stream)
        lse, lp = self._lse(lse, T, H, stream)
        a = _ATTN.pack(_ATTN.size, n - 1, H, G, D, 0, 0, 0, D ** -0.5 if scale is None else scale, 0, 0, 0, 0, 0,
                       qp, q0, q1, kp, k0, k1, vp, v0, v1, op, o0, o1, 0, 0, 0, 0, 0, 0, 0, 0, starts, 0, 0, 0, 0, lp)
        if near:
            rc = (_lib or load()).ub_attn_prompt_window(self._h, a, window, sinks, self._raw_stream(stream))
        else:
            rc = (_lib or load()).ub_attn_prompt(self._h, a, self._raw_stream(stream))
        if rc:
            _check(rc)
        return out if lse is None else (out, lse)

    def attn_prompt_paged(self, q, k_cache, v_cache, seq_starts, kv_lens, page_table, out=None, lse=None,
                          scale: float | None = None, stream=None, window: int = 0, sinks: int = 0):
        """Causal attention of prompts, or of chunks of prompts, over the paged cache that holds
        their keys and values (after kv_append); arguments as there and in attn_prompt. With a
        window, entries of page_table whose pages no token sees are not looked at."""
        near = _sight(window, sinks)
        dev = self._dev
        T, _ = self._active or self.active_shape
        D = _head_dim(q)
        qp, q0, q1, H = _heads_view(q, "q", T, D, dev)
        caches, pages, G, page = _caches(k_cache, v_cache, D, dev)
        if page == 0:
            raise ValueError("pages of no rows")
        lens, n = _ints(kv_lens, "kv_lens", None, dev)
        starts, _ = _ints(seq_starts, "seq_starts", n + 1, dev)
        table, width, table_row = _table(page_table, n, dev)
        out, op, o0, o1 = self._out(out, "out", T, H, D, stream)
        lse, lp = self._lse(lse, T, H, stream)
        a = _ATTN.pack(_ATTN.size, n, H, G, D, page, 0, 0, D ** -0.5 if scale is None else scale, 0, pages, width,
                       table_row, 0, qp, q0, q1, 0, 0, 0, 0, 0, 0, op, o0, o1, *caches, starts, lens, table, 0, 0, lp)
        if near:
            rc = (_lib or load()).ub_attn_prompt_window(self._h, a, window, sinks, self._raw_stream(stream))
        else:
            rc = (_lib or load()).ub_attn_prompt(self._h, a, self._raw_stream(stream))
        if rc:
            _check(rc)
        return out if lse is None else (out, lse)

    def attn_decode(self, q, k_cache, v_cache, kv_lens, page_table, out=None, lse=None, scale: float | None = None,
                    stream=None, window: int = 0, sinks: int = 0):
        """Attention of one new token per sequence over the paged cache (ub_attn_decode): row s of
        q [T, heads, D] is sequence s, n = kv_lens.shape[0] <= T; arguments as in kv_append and
        attn_prompt (window and sinks: ub_attn_decode_window). Rows from n on stay as they are."""
        near = _sight(window, sinks)
        dev = self._dev
        T, _ = self._active or self.active_shape
        D = _head_dim(q)
        qp, q0, q1, H = _heads_view(q, "q", T, D, dev)
        caches, pages, G, page = _caches(k_cache, v_cache, D, dev)
        lens, n = _ints(kv_lens, "kv_lens", None, dev)
        table, width, table_row = _table(page_table, n, dev)
        out, op, o0, o1 = self._out(out, "out", T, H, D, stream)
        lse, lp = self._lse(lse, T, H, stream)
        a = _ATTN.pack(_ATTN.size, n, H, G, D, page, 0, 0, D ** -0.5 if scale is None else scale, 0, pages, width,
                       table_row, 0, qp, q0, q1, 0, 0, 0, 0, 0, 0, op, o0, o1, *caches, 0, lens, table, 0, 0, lp)
        if near:
            rc = (_lib or load()).ub_attn_decode_window(self._h, a, window, sinks, self._raw_stream(stream))
        else:
            rc = (_lib or load()).ub_attn_decode(self._h, a, self._raw_stream(stream))
        if rc:
            _check(rc)
        return out if lse is None else (out, lse)

    def attn_tree(self, q, k_cache, v_cache, seq_starts, kv_lens, page_table, parents, out=None, lse=None,
                  scale: float | None = None, stream=None, window: int = 0, sinks: int = 0):
        """Attention of drafted tokens over the paged cache that holds the text and them
        (ub_attn_tree): rows [seq_starts[s], seq_starts[s + 1]) of q are the drafts of sequence s,
        the last of its kv_lens[s] cached tokens. parents int32 [T]: the draft that each token
        follows, counted within its sequence and before it, or -1: the text. A draft sees the text,
        its ancestors and itself. Other arguments as in attn_prompt_paged."""
        near = _sight(window, sinks)
        dev = self._dev
        T, _ = self._active or self.active_shape
        D = _head_dim(q)
        qp, q0, q1, H = _heads_view(q, "q", T, D, dev)
        caches, pages, G, page = _caches(k_cache, v_cache, D, dev)
        lens, n = _ints(kv_lens, "kv_lens", None, dev)
        starts, _ = _ints(seq_starts, "seq_starts", n + 1, dev)
        up, _ = _ints(parents, "parents", T, dev)
        table, width, table_row = _table(page_table, n, dev)
        out, op, o0, o1 = self._out(out, "out", T, H, D, stream)
        lse, lp = self._lse(lse, T, H, stream)
        a = _ATTN.pack(_ATTN.size, n, H, G, D, page, 0, 0, D ** -0.5 if scale is None else scale, 0, pages, width,
                       table_row, 0, qp, q0, q1, 0, 0, 0, 0, 0, 0, op, o0, o1, *caches, starts, lens, table, 0, 0, lp)
        rc = (_lib or load()).ub_attn_tree(self._h, a, up, window, sinks if near else 0, self._raw_stream(stream))
        if rc:
            _check(rc)
        return out if lse is None else (out, lse)

    def kv_accept(self, k_cache, v_cache, seq_starts, kv_lens, page_table, parents, leaves, new_lens=None, stream=None):
        """Keep the accepted drafts (ub_kv_accept): leaves int32 [n] names the last accepted draft of
        each sequence, -1 for none; the cached rows of its path move together behind the text.
        Returns new_lens int32 [n], the lengths with the accepted drafts. parents has an entry per
        draft, whatever the active shape is now; kv_lens stays as it is, for the other layers'
        caches."""
        dev = self._dev
        try:
            D = k_cache.shape[3]
        except (AttributeError, IndexError, TypeError):
            D = -1
        caches, pages, G, page = _caches(k_cache, v_cache, D, dev)
        lens, n = _ints(kv_lens, "kv_lens", None, dev)
        starts, _ = _ints(seq_starts, "seq_starts", n + 1, dev)
        up, tokens = _ints(parents, "parents", None, dev)
        last, _ = _ints(leaves, "leaves", n, dev)
        table, width, table_row = _table(page_table, n, dev)
        if new_lens is None:
            new_lens = self._new((n,), _I32, stream)
        to, _ = _ints(new_lens, "new_lens", n, dev)
        a = _ATTN.pack(_ATTN.size, n, G, G, D, page, 0, 0, 1.0, 0, pages, width, table_row, 0, *[0] * 12, *caches,
                       starts, lens, table, 0, 0, 0)
        rc = (_lib or load()).ub_kv_accept(self._h, a, up, tokens, last, to, self._raw_stream(stream))
        if rc:
            _check(rc)
        return new_lens

    # -- pages of the cache
    def _pool(self, refs, page_table, page_size: int, n: int):
        refs_p, pages = _ints(refs, "refs", None, self._dev)
        table, width, row = _table(page_table, n, self._dev)
        return _POOL.pack(_POOL.size, n, page_size, 0, pages, width, row, refs_p, table), pages, width

    def kv_take(self, refs, page_table, begin, end, page_size: int, stream=None):
        """Pages for the cache rows [begin[s], end[s]) of every sequence (ub_kv_take): each missing
        entry (-1) of page_table int32 [n, entries] among them gets a free page, the lowest first.
        refs int32 [pages]: how many table entries name a page, 0: free. In place."""
        n = _tall(page_table, "page_table")
        pool, _, _ = self._pool(refs, page_table, page_size, n)
        b, _ = _ints(begin, "begin", n, self._dev)
        e, _ = _ints(end, "end", n, self._dev)
        rc = (_lib or load()).ub_kv_take(self._h, pool, b, e, self._raw_stream(stream))
        if rc:
            _check(rc)

    def kv_free(self, refs, page_table, begin, end, page_size: int, stream=None):
        """Give up the pages that lie wholly within the cache rows [begin[s], end[s]) of every sequence
        (ub_kv_free): their entries become -1, their counts go down. `end` may lie past the table."""
        n = _tall(page_table, "page_table")
        pool, _, _ = self._pool(refs, page_table, page_size, n)
        b, _ = _ints(begin, "begin", n, self._dev)
        e, _ = _ints(end, "end", n, self._dev)
        rc = (_lib or load()).ub_kv_free(self._h, pool, b, e, self._raw_stream(stream))
        if rc:
            _check(rc)

    def kv_fork(self, refs, page_table, kv_lens, source, new_table, page_size: int, copies=None, stream=None):
        """Fork sequences (ub_kv_fork): row i of new_table int32 [children, entries] becomes row
        source[i] of page_table, whole pages shared, a last page that is filled in part replaced by
        a free one. Returns copies int32 [children, 2], (from, to) of those or (-1, -1): the data to
        copy with kv_copy, in every layer's cache. new_table overlaps page_table nowhere."""
        dev = self._dev
        pool, _, width = self._pool(refs, page_table, page_size, _tall(page_table, "page_table"))
        lens, _ = _ints(kv_lens, "kv_lens", page_table.shape[0], dev)
        src, m = _ints(source, "source", None, dev)
        to, new_width, new_row = _table(new_table, m, dev, "new_table")
        if new_width != width:
            raise ValueError("new_table has %d entries per row, page_table %d" % (new_width, width))
        if copies is None:
            copies = self._new((m, 2), _I32, stream)
        pairs, _ = _pairs(copies, "copies", m, dev)
        rc = (_lib or load()).ub_kv_fork(self._h, pool, lens, src, m, to, new_row, pairs, self._raw_stream(stream))
        if rc:
            _check(rc)
        return copies

    def kv_compact(self, refs, page_table, refs_out=None, table_out=None, moves=None, used=None, stream=None):
        """Move the pages in use together into the first ones (ub_kv_compact). Returns (moves, used):
        moves int32 [>= pages / 2, 2], (from, to) and then (-1, -1), for kv_copy; used int32 [1],
        the number of pages in use. refs and page_table change in place unless refs_out and
        table_out are given. Every table on the pool has to be rows of page_table."""
        dev = self._dev
        n = _tall(page_table, "page_table")
        pool, pages, width = self._pool(refs, page_table, 8, n)  # the page size plays no part
        r, _ = _ints(refs if refs_out is None else refs_out, "refs_out", pages, dev)
        t, new_width, row = _table(page_table if table_out is None else table_out, n, dev, "table_out")
        if new_width != width:
            raise ValueError("table_out has %d entries per row, page_table %d" % (new_width, width))
        if moves is None:
            moves = self._new((pages // 2, 2), _I32, stream)
        if used is None:
            used = self._new((1,), _I32, stream)
        m, room = _pairs(moves, "moves", None, dev)
        u, _ = _ints(used, "used", 1, dev)
        rc = (_lib or load()).ub_kv_compact(self._h, pool, r, t, row, m, room, u, self._raw_stream(stream))
        if rc:
            _check(rc)
        return moves, used

    def kv_copy(self, k_cache, v_cache, pairs, stream=None):
        """Copy pages (ub_kv_copy): page pairs[i, 0] of both caches to page pairs[i, 1]; pairs int32
        [n, 2] on the device, (-1, -1) is skipped."""
        dev = self._dev
        try:
            D = k_cache.shape[3]
        except (AttributeError, IndexError, TypeError):
            D = -1
        caches, pages, G, page = _caches(k_cache, v_cache, D, dev)
        p, n = _pairs(pairs, "pairs", None, dev)
        a = _ATTN.pack(_ATTN.size, 1, G, G, D, page, 0, 0, 1.0, 0, pages, 1, 1, 0, *[0] * 12, *caches, *[0] * 6)
        rc = (_lib or load()).ub_kv_copy(self._h, a, p, n, self._raw_stream(stream))
        if rc:
            _check(rc)


def ag_gemm_noalloc(shards, Wt: torch.Tensor, Y: torch.Tensor | None = None, stream=None):
    """AG-GEMM through the allocation-free entry point (no handle): for callers that
    cannot allocate device memory. Uses the library's fixed 32 MiB device scratch, so
    T * hidden <= NOALLOC_MAX_ELEMS, and calls on one device must not overlap.

    The C entry point cannot see tensor sizes (it builds its tensor maps from T, hidden
    and N alone), so every shape and the device of every tensor are checked here, and
    the call runs with the tensors' device current: the library picks that device's
    copy of the scratch and launches there."""
    tp = len(shards)
    if not 1 <= tp <= MAX_TP:
        raise ValueError("expected 1..%d shards, got %d" % (MAX_TP, tp))
    _bf16_cuda(shards[0], "shards[0]")
    if shards[0].dim() != 2:
        raise ValueError("shards[0] must be [c, hidden], got %s" % (tuple(shards[0].shape),))
    c, H = shards[0].shape
    for r, s in enumerate(shards):
        _bf16_cuda(s, "shards[%d]" % r, (c, H))
    _bf16_cuda(Wt, "Wt")
    if Wt.dim() != 2 or Wt.shape[1] != H:
        raise ValueError("Wt must be [N, %d], got %s" % (H, tuple(Wt.shape)))
    N = Wt.shape[0]
    T = c * tp
    device = Wt.device
    if Y is None:
        Y = torch.empty((T, N), dtype=torch.bfloat16, device=device)
    _bf16_cuda(Y, "Y")
    if Y.dim() != 2 or Y.shape[0] < T or Y.shape[1] != N:
        raise ValueError("Y must be [>=%d, %d], got %s" % (T, N, tuple(Y.shape)))
    for name, t in [("shards[%d]" % r, s) for r, s in enumerate(shards)] + [("Y", Y)]:
        if t.device != device:
            raise ValueError("%s is on %s, Wt on %s: all tensors must share one device" % (name, t.device, device))
    with torch.cuda.device(device):
        _check(load().ag_gemm_noalloc(_ptrs(shards), tp, T, H, ctypes.c_void_p(Wt.data_ptr()), N,
                                      ctypes.c_void_p(Y.data_ptr()), _stream_ptr(stream)))
    return Y


# ---------------------------------------------------------------- module-level manager

_default: UserBuffer | None = None


def initialize_ub(shape, tp_size: int, dtype=torch.bfloat16) -> UserBuffer:
    """Register the default user buffer at capacity ``shape`` = [max_tokens, hidden]."""
    global _default
    if _default is not None:
        _default.close()
    _default = UserBuffer(shape, tp_size, dtype)
    return _default


def set_ub_active_shape(shape):
    """Set the active shape [T, hidden] of the default user buffer."""
    if _default is None:
        raise RuntimeError("initialize_ub() has not been called")
    _default.set_active_shape(shape)


def get_ub() -> UserBuffer:
    if _default is None:
        raise RuntimeError("initialize_ub() has not been called")
    return _default


def destroy_ub():
    global _default
    if _default is not None:
        _default.close()
        _default = None
