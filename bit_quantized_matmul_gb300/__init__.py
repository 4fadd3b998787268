"""Thin Python binding over the C ABI of ``libq4mm.so`` (``include/q4mm.h``).

Argument marshalling only: tensors are passed as raw device pointers with the
current PyTorch CUDA stream, and every step of the computation runs in the
library's CUDA kernels.  There is no CPU or PyTorch fallback: if the library
is missing, importing this package raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch  # device memory and streams; loads the CUDA runtime first

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq4mm.so")

Q4_OK = 0
Q4_ERR_INVALID_ARG = 1
Q4_ERR_SHAPE = 2
Q4_ERR_ALIGN = 3
Q4_ERR_NONFINITE = 4
Q4_ERR_RANGE = 5
Q4_ERR_CUDA = 6
Q4_ERR_TIMEOUT = 7
Q4_ERR_NOMEM = 8
Q4_ERR_UNSUPPORTED = 9

Q4MM_BATCH_INVARIANT = 0x1
Q4MM_FORCE_SIMT = 0x2
Q4MM_FORCE_TC = 0x4
Q4MM_ROW_BY_ROW = 0x8
Q4MM_FORCE_MMA = 0x10
Q4MM_M_MAX = 4096
Q4MM_GROUP_MAX = 4
Q4MM_NOALLOC_PARTIAL_BYTES = 2457600
Q4MM_PATH_SIMT = 1
Q4MM_PATH_TC = 2
Q4MM_PATH_ROW_BY_ROW = 3
Q4MM_PATH_MMA = 4
Q4_DTYPE_F32 = 0
Q4_DTYPE_F16 = 1
Q4_DTYPE_BF16 = 2

BLOCK = 32
BLOCK_BYTES = 18

# Every symbol the header declares; the CPU test checks the library exports them.
EXPORTS = (
    "q4_quantize", "q4_import_blocks", "q4_export_blocks", "q4_weight_free", "q4_weight_shape",
    "q4_weight_device_bytes", "q4mm_forward", "q4mm_forward_ex", "q4mm_argmax", "q4mm_argmax_ex",
    "q4mm_forward_noalloc", "q4mm_forward_group", "q4mm_forward_gated", "q4mm_argmax_rows", "q4_verify_greedy",
    "q4mm_select_path", "q4mm_plan_info", "q4mm_set_m_threshold", "q4mm_get_m_threshold", "q4mm_set_group_m_threshold",
    "q4mm_get_group_m_threshold", "q4_device_status", "q4mm_set_wait_limit_ns", "q4mm_set_stall_for_test",
    "q4_status_string", "q4_scratch_bytes",
    "q4_kv_append",
    "q4_kvq_cache_bytes", "q4_kvq_append", "q4_kvq_read", "q4_kvq_attention", "q4_kvq_evict",
    "q4_prompt_attention",
)

if not os.path.exists(LIB_PATH):
    raise ImportError("libq4mm.so is not built (%s); run __graft_entry__.build() or "
                      "python bit_quantized_matmul_gb300/build.py" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)
_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_u32 = ctypes.c_uint32
_int = ctypes.c_int
_sig = {
    "q4_quantize": [_p, _i64, _i64, ctypes.POINTER(_p), _p],
    "q4_import_blocks": [_p, _i64, _i64, ctypes.POINTER(_p), _p],
    "q4_export_blocks": [_p, _p, ctypes.c_size_t],
    "q4_weight_free": [_p],
    "q4_weight_shape": [_p, ctypes.POINTER(_i64), ctypes.POINTER(_i64)],
    "q4_weight_device_bytes": [_p, ctypes.POINTER(ctypes.c_size_t)],
    "q4mm_forward": [_p, _p, _p, _i64, _p],
    "q4mm_forward_ex": [_p, _p, _p, _i64, _u32, _p],
    "q4mm_argmax": [_p, _p, _p, _p, _i64, _p],
    "q4mm_argmax_ex": [_p, _p, _p, _p, _i64, _u32, _p],
    "q4mm_forward_noalloc": [_p, _p, _p, _i64, _p],
    "q4mm_forward_group": [_p, ctypes.c_int, _p, _p, _i64, _u32, _p],
    "q4mm_forward_gated": [_p, _p, _p, _p, _i64, _u32, _p],
    "q4mm_argmax_rows": [_p, _p, _i64, _p, _i64, _p, _p, _p],
    "q4_verify_greedy": [_p, _p, _i64, _p, _i64, _p, _p],
    "q4_kv_append": [_p, _p, _p, _p, _i64, _i64, _i64, _i64, _i64, ctypes.c_int, ctypes.POINTER(_i64),
                     ctypes.POINTER(_i64), _p, _p, _p, _i64, _i64, _p],
    "q4_kvq_cache_bytes": [_i64] * 4 + [ctypes.POINTER(ctypes.c_size_t)],
    "q4_kvq_append": [_p, _p, _p, _int] + [_i64] * 4 + [_p] * 5 + [_i64, _i64, _p],
    "q4_kvq_read": [_p, _p, _p, _int] + [_i64] * 4 + [_p] * 3 + [_i64, _i64, _p],
    "q4_kvq_attention": [_p, _p, _p, _p, _int] + [_i64] * 5 + [_p, ctypes.c_float] + [_p] * 3 + [_i64, _i64, _p],
    "q4_kvq_evict": [_p, _p] + [_i64] * 4 + [_p] * 3 + [_i64] * 3 + [_p] * 3,
    "q4_prompt_attention": [_p] * 4 + [_int] + [_i64] * 3 + [_p] * 3 + [ctypes.c_float, _int, _p, _p] + [_i64] * 3 +
                           [_p],
    "q4mm_select_path": [_p, _i64, _u32],
    "q4mm_plan_info": [_p, _i64, _u32, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                       ctypes.POINTER(ctypes.c_int)],
    "q4mm_set_m_threshold": [_i64],
    "q4mm_get_m_threshold": [],
    "q4mm_set_group_m_threshold": [_i64],
    "q4mm_get_group_m_threshold": [],
    "q4_device_status": [],
    "q4mm_set_wait_limit_ns": [ctypes.c_uint64],
    "q4mm_set_stall_for_test": [ctypes.c_int],
    "q4_status_string": [ctypes.c_int],
    "q4_scratch_bytes": [ctypes.POINTER(ctypes.c_size_t)] * 4,
}
for _name, _args in _sig.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int
_lib.q4mm_get_m_threshold.restype = ctypes.c_int64
_lib.q4mm_get_group_m_threshold.restype = ctypes.c_int64
_lib.q4_status_string.restype = ctypes.c_char_p


class Q4Error(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        msg = "%s: %s (status %d)" % (what, q4_status_string(status), status)
        super().__init__(msg)
        self.status = status


def _check(status: int, what: str):
    if status != Q4_OK:
        raise Q4Error(status, what)


def q4_status_string(status: int) -> str:
    return _lib.q4_status_string(int(status)).decode()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev_f32(t: torch.Tensor, name: str) -> torch.Tensor:
    if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()):
        raise ValueError("%s must be a contiguous float32 CUDA tensor" % name)
    return t


class Q4Weight:
    """Owning wrapper of a ``q4_weight*`` handle (freed on ``free()`` / GC)."""

    def __init__(self, handle: int, N: int, K: int, device: torch.device):
        self._h = ctypes.c_void_p(handle)
        self.N, self.K, self.device = N, K, device

    @property
    def handle(self) -> ctypes.c_void_p:
        if not self._h:
            raise ValueError("Q4Weight already freed")
        return self._h

    def free(self):
        if self._h:
            torch.cuda.synchronize(self.device)
            _check(_lib.q4_weight_free(self._h), "q4_weight_free")
            self._h = ctypes.c_void_p(0)

    def __del__(self):
        try:
            if self._h:
                _lib.q4_weight_free(self._h)
        except Exception:
            pass

    def device_bytes(self) -> int:
        b = ctypes.c_size_t(0)
        _check(_lib.q4_weight_device_bytes(self.handle, ctypes.byref(b)), "q4_weight_device_bytes")
        return int(b.value)

    @property
    def packed_bytes(self) -> int:
        """Algorithmic size of the Q4_0 weights: N*K/32 blocks of 18 bytes."""
        return self.N * (self.K // BLOCK) * BLOCK_BYTES


def q4_quantize(w: torch.Tensor, stream=None) -> Q4Weight:
    """Quantize an fp32 [N, K] CUDA tensor into a library-owned Q4_0 weight."""
    _dev_f32(w, "w")
    N, K = w.shape
    h = ctypes.c_void_p(0)
    with torch.cuda.device(w.device):
        _check(_lib.q4_quantize(w.data_ptr(), N, K, ctypes.byref(h), _stream(stream)), "q4_quantize")
    return Q4Weight(h.value, N, K, w.device)


def q4_import_blocks(blocks, N: int, K: int, device=None, stream=None) -> Q4Weight:
    """Create a weight from canonical blocks (uint8 numpy array / bytes, N*K/32*18 bytes)."""
    import numpy as np

    arr = np.ascontiguousarray(np.frombuffer(bytes(blocks), np.uint8) if isinstance(blocks, (bytes, bytearray))
                               else blocks, dtype=np.uint8)
    if arr.size != N * (K // BLOCK) * BLOCK_BYTES:
        raise ValueError("blocks size does not match N, K")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    h = ctypes.c_void_p(0)
    with torch.cuda.device(device):
        _check(_lib.q4_import_blocks(arr.ctypes.data_as(ctypes.c_void_p), N, K, ctypes.byref(h),
                                     _stream(stream)), "q4_import_blocks")
    return Q4Weight(h.value, N, K, device)


def q4_export_blocks(W: Q4Weight):
    """Canonical blocks of W as a uint8 numpy array [N, K/32, 18]."""
    import numpy as np

    out = np.empty((W.N, W.K // BLOCK, BLOCK_BYTES), np.uint8)
    with torch.cuda.device(W.device):
        _check(_lib.q4_export_blocks(W.handle, out.ctypes.data_as(ctypes.c_void_p), out.nbytes),
               "q4_export_blocks")
    return out


def q4_weight_free(W: Q4Weight):
    W.free()


def q4mm_forward_ex(W: Q4Weight, x: torch.Tensor, flags: int = 0, y: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """y[M, N] = x[M, K] @ W^T (fp32) with Q4MM_* flags."""
    _dev_f32(x, "x")
    M = x.shape[0]
    if x.dim() != 2 or x.shape[1] != W.K:
        raise ValueError("x must be [M, %d]" % W.K)
    if y is None:
        y = torch.empty((M, W.N), dtype=torch.float32, device=x.device)
    _dev_f32(y, "y")
    if tuple(y.shape) != (M, W.N):
        raise ValueError("y must be [M, %d]" % W.N)
    with torch.cuda.device(x.device):
        _check(_lib.q4mm_forward_ex(W.handle, x.data_ptr(), y.data_ptr(), M, int(flags), _stream(stream)),
               "q4mm_forward_ex")
    return y


def q4mm_forward(W: Q4Weight, x: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _dev_f32(x, "x")
    M = x.shape[0]
    if x.dim() != 2 or x.shape[1] != W.K:
        raise ValueError("x must be [M, %d]" % W.K)
    if y is None:
        y = torch.empty((M, W.N), dtype=torch.float32, device=x.device)
    _dev_f32(y, "y")
    if tuple(y.shape) != (M, W.N):
        raise ValueError("y must be [M, %d]" % W.N)
    with torch.cuda.device(x.device):
        _check(_lib.q4mm_forward(W.handle, x.data_ptr(), y.data_ptr(), M, _stream(stream)), "q4mm_forward")
    return y


def q4mm_forward_noalloc(W: Q4Weight, x: torch.Tensor, y: torch.Tensor, stream=None) -> torch.Tensor:
    """y[M, N] = x[M, K] @ W^T into the caller's y, allocating no device memory.

    For callers that must not allocate mid-step (their memory is all in their
    own pool, or a device-wide wait is unacceptable).  The first call on a
    device sets up the fixed scratch and synchronizes once; calls whose kernels
    overlap on the GPU race on that scratch.  Raises Q4Error(Q4_ERR_SHAPE) when
    the split-K partial sums exceed Q4MM_NOALLOC_PARTIAL_BYTES.
    """
    _dev_f32(x, "x")
    M = x.shape[0]
    if x.dim() != 2 or x.shape[1] != W.K:
        raise ValueError("x must be [M, %d]" % W.K)
    _dev_f32(y, "y")
    if tuple(y.shape) != (M, W.N):
        raise ValueError("y must be [M, %d]" % W.N)
    with torch.cuda.device(x.device):
        _check(_lib.q4mm_forward_noalloc(W.handle, x.data_ptr(), y.data_ptr(), M, _stream(stream)),
               "q4mm_forward_noalloc")
    return y


def q4mm_forward_group(Ws, x: torch.Tensor, ys=None, flags: int = 0, stream=None):
    """[x @ W_i^T for W_i in Ws] in one launch per 16 token rows (weights sharing K)."""
    _dev_f32(x, "x")
    M = x.shape[0]
    if not 1 <= len(Ws) <= Q4MM_GROUP_MAX:
        raise ValueError("1 to %d weights" % Q4MM_GROUP_MAX)
    if x.dim() != 2 or any(W.K != x.shape[1] for W in Ws):
        raise ValueError("x must be [M, K] with the K of every weight")
    if ys is None:
        ys = [torch.empty((M, W.N), dtype=torch.float32, device=x.device) for W in Ws]
    if len(ys) != len(Ws):
        raise ValueError("one output per weight")
    for W, y in zip(Ws, ys):
        _dev_f32(y, "y")
        if tuple(y.shape) != (M, W.N):
            raise ValueError("y must be [M, %d]" % W.N)
    hw = (ctypes.c_void_p * len(Ws))(*[W.handle for W in Ws])
    hy = (ctypes.c_void_p * len(ys))(*[y.data_ptr() for y in ys])
    with torch.cuda.device(x.device):
        _check(_lib.q4mm_forward_group(hw, len(Ws), x.data_ptr(), hy, M, int(flags), _stream(stream)),
               "q4mm_forward_group")
    return ys


def q4mm_forward_gated(Wg: Q4Weight, Wu: Q4Weight, x: torch.Tensor, h: torch.Tensor | None = None,
                       flags: int = 0, stream=None) -> torch.Tensor:
    """h = SiLU(x @ Wg^T) * (x @ Wu^T) (the gated MLP step; q4mm_forward_gated)."""
    _dev_f32(x, "x")
    M = x.shape[0]
    if x.dim() != 2 or x.shape[1] != Wg.K:
        raise ValueError("x must be [M, %d]" % Wg.K)
    if (Wu.N, Wu.K) != (Wg.N, Wg.K):
        raise ValueError("gate and up projections must have one shape")
    if h is None:
        h = torch.empty((M, Wg.N), dtype=torch.float32, device=x.device)
    _dev_f32(h, "h")
    if tuple(h.shape) != (M, Wg.N):
        raise ValueError("h must be [M, %d]" % Wg.N)
    with torch.cuda.device(x.device):
        _check(_lib.q4mm_forward_gated(Wg.handle, Wu.handle, x.data_ptr(), h.data_ptr(), M, int(flags),
                                       _stream(stream)), "q4mm_forward_gated")
    return h


def q4mm_argmax_rows(W: Q4Weight, x: torch.Tensor, rows: torch.Tensor, want_max: bool = True,
                     stream=None):
    """Greedy pick (idx int32 [R], max fp32 [R] or None) for the x rows listed in `rows`."""
    _dev_f32(x, "x")
    if x.dim() != 2 or x.shape[1] != W.K:
        raise ValueError("x must be [rows, %d]" % W.K)
    if rows.dtype != torch.int32 or not rows.is_cuda or not rows.is_contiguous():
        raise ValueError("rows must be a contiguous int32 CUDA tensor")
    R = rows.numel()
    idx = torch.empty((R,), dtype=torch.int32, device=x.device)
    mx = torch.empty((R,), dtype=torch.float32, device=x.device) if want_max else None
    with torch.cuda.device(x.device):
        _check(_lib.q4mm_argmax_rows(W.handle, x.data_ptr(), x.shape[0], rows.data_ptr(), R, idx.data_ptr(),
                                     mx.data_ptr() if mx is not None else None, _stream(stream)),
               "q4mm_argmax_rows")
    return idx, mx


def q4_verify_greedy(idx: torch.Tensor, draft: torch.Tensor, offsets: torch.Tensor, stream=None):
    """accepted[s]: leading positions of segment s where idx == draft (-1: malformed segment)."""
    for t, n in ((idx, "idx"), (draft, "draft"), (offsets, "offsets")):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("%s must be a contiguous int32 CUDA tensor" % n)
    if idx.numel() != draft.numel():
        raise ValueError("idx and draft differ in length")
    S = offsets.numel() - 1
    acc = torch.empty((max(S, 0),), dtype=torch.int32, device=idx.device)
    with torch.cuda.device(idx.device):
        _check(_lib.q4_verify_greedy(idx.data_ptr(), draft.data_ptr(), idx.numel(), offsets.data_ptr(), max(S, 0),
                                     acc.data_ptr(), _stream(stream)), "q4_verify_greedy")
    return acc


def q4_kv_append(k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                 offsets: torch.Tensor, slot: torch.Tensor, pos: torch.Tensor, stream=None):
    """Write the step's new K/V rows into a preallocated cache, in place.

    k_cache, v_cache: contiguous [layers, slots, heads, capacity, head_dim];
    k_new, v_new: [layers, total, heads, head_dim] views (head_dim contiguous,
    any other strides) of the same dtype (2- or 4-byte elements);
    offsets int32 [S + 1], slot and pos int32 [S], all on the cache's device.
    """
    if k_cache.dim() != 5 or v_cache.shape != k_cache.shape or not k_cache.is_contiguous() or \
            not v_cache.is_contiguous():
        raise ValueError("caches must be contiguous [layers, slots, heads, capacity, head_dim] of one shape")
    if k_new.dim() != 4 or v_new.shape != k_new.shape:
        raise ValueError("new rows must be [layers, total, heads, head_dim] views of one shape")
    L, slots, H, cap, D = k_cache.shape
    if k_new.shape[0] != L or k_new.shape[2] != H or k_new.shape[3] != D or k_new.stride(3) != 1 or \
            v_new.stride(3) != 1:
        raise ValueError("new rows do not match the cache shape (or head_dim is not contiguous)")
    for t in (v_cache, k_new, v_new):
        if t.dtype != k_cache.dtype or t.device != k_cache.device:
            raise ValueError("caches and new rows must share dtype and device")
    for t, n in ((offsets, "offsets"), (slot, "slot"), (pos, "pos")):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.device != k_cache.device:
            raise ValueError("%s must be a contiguous int32 tensor on the cache's device" % n)
    S = slot.numel()
    if offsets.numel() != S + 1 or pos.numel() != S:
        raise ValueError("offsets must have S + 1 entries and pos S")
    with torch.cuda.device(k_cache.device):
        ks = (_i64 * 3)(*k_new.stride()[:3])
        vs = (_i64 * 3)(*v_new.stride()[:3])
        _check(_lib.q4_kv_append(k_cache.data_ptr(), v_cache.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
                                 L, slots, H, D, cap, k_cache.element_size(), ks, vs, offsets.data_ptr(),
                                 slot.data_ptr(), pos.data_ptr(), S, k_new.shape[1], _stream(stream)),
               "q4_kv_append")


# The calls of a decode step are a few microseconds of GPU work each, so what
# their bindings cost on the host is kept small: one pass over each tensor's
# attributes, and PyTorch's raw stream and device getters.
_DTYPES = {torch.float32: Q4_DTYPE_F32, torch.float16: Q4_DTYPE_F16, torch.bfloat16: Q4_DTYPE_BF16}
_I64x2 = _i64 * 2
_f32, _i32 = torch.float32, torch.int32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(fn, what: str, index: int, stream, *args):
    """fn(*args, stream) with CUDA device `index` current; raises on a status that is not Q4_OK."""
    if stream is None and _get_device() == index and _raw_stream is not None:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _stream(stream))
    if status != Q4_OK:
        raise Q4Error(status, what)


def _dtype_code(dtype, name: str) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("%s must be float32, float16 or bfloat16" % name)
    return code


@functools.lru_cache(maxsize=1024)
def _strides(s0: int, s1: int):
    return _I64x2(s0, s1)  # read by the library only


def _rows3(t: torch.Tensor, name: str, heads: int, head_dim: int, dtype, index: int):
    """(rows, the two outer strides) of a [rows, heads, head_dim] view with contiguous head_dim on device `index`."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim:
        raise ValueError("%s must be a [rows, %d, %d] view" % (name, heads, head_dim))
    s0, s1, s2 = t.stride()
    if s2 != 1 and t.numel():
        raise ValueError("%s must have contiguous rows of head_dim values" % name)
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError("%s must be %s on CUDA device %d" % (name, dtype, index))
    return shape[0], _strides(s0, s1)


def _ints(index: int, t: torch.Tensor, name: str) -> int:
    """Length of a contiguous int32 tensor on device `index`."""
    if t.dtype is not _i32 or t.get_device() != index or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor on CUDA device %d" % (name, index))
    return t.numel()


def _out3(t, shape, dtype, device, name: str) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(t.shape) != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s" % (name, dtype, shape, device))
    return t


class Q4KVCache:
    """A 4-bit KV cache of one decoder layer: slots x heads x capacity positions of head_dim values.

    Owns the device buffer (``data``) that the ``q4_kvq_*`` calls work on; its layout is the library's.
    """

    def __init__(self, slots: int, heads: int, head_dim: int, capacity: int, device=None):
        self.slots, self.heads, self.head_dim, self.capacity = int(slots), int(heads), int(head_dim), int(capacity)
        n = ctypes.c_size_t(0)
        _check(_lib.q4_kvq_cache_bytes(self.slots, self.heads, self.head_dim, self.capacity, ctypes.byref(n)),
               "q4_kvq_cache_bytes")
        device = torch.device("cuda" if device is None else device)
        self.data = torch.zeros(n.value, dtype=torch.uint8, device=device)
        self.device = self.data.device
        self._dims = (self.slots, self.heads, self.head_dim, self.capacity)
        self._index = self.data.get_device()

    @property
    def nbytes(self) -> int:
        return self.data.numel()

    def new_mass(self) -> torch.Tensor:
        """Zeroed attention weights, fp32 [slots, heads, capacity]."""
        return torch.zeros((self.slots, self.heads, self.capacity), dtype=torch.float32, device=self.device)


def _step(cache: Q4KVCache, offsets, slot, pos) -> int:
    index = cache._index
    S = _ints(index, slot, "slot")
    if _ints(index, offsets, "offsets") != S + 1 or _ints(index, pos, "pos") != S:
        raise ValueError("offsets must have S + 1 entries and pos S")
    return S


def _mass(cache: Q4KVCache, mass: torch.Tensor) -> int:
    if tuple(mass.shape) != (cache.slots, cache.heads, cache.capacity) or mass.dtype != _f32 or \
            mass.device != cache.device or not mass.is_contiguous():
        raise ValueError("mass must be a contiguous float32 [slots, heads, capacity] tensor on the cache's device")
    return mass.data_ptr()


def q4_kvq_append(cache: Q4KVCache, k_new: torch.Tensor, v_new: torch.Tensor, offsets: torch.Tensor,
                  slot: torch.Tensor, pos: torch.Tensor, stream=None):
    """Quantize the step's new K/V rows ([total, heads, head_dim] views) into the cache.

    offsets int32 [S + 1], slot and pos int32 [S]: row offsets[s] + j of the packed
    step becomes position pos[s] + j of slot[s].
    """
    S = _step(cache, offsets, slot, pos)
    dtype, index = k_new.dtype, cache._index
    code = _dtype_code(dtype, "k_new")
    slots, heads, d, cap = cache._dims
    total, ks = _rows3(k_new, "k_new", heads, d, dtype, index)
    total_v, vs = _rows3(v_new, "v_new", heads, d, dtype, index)
    if total_v != total:
        raise ValueError("k_new and v_new differ in rows")
    _call(_lib.q4_kvq_append, "q4_kvq_append", index, stream, cache.data.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), code,
          slots, heads, d, cap, ks, vs, offsets.data_ptr(), slot.data_ptr(), pos.data_ptr(), S, total)


def q4_kvq_read(cache: Q4KVCache, offsets: torch.Tensor, slot: torch.Tensor, pos: torch.Tensor, total: int,
                dtype=torch.float32, k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None):
    """(k, v), each [total, heads, head_dim]: the rows that the cache holds for a step's requests."""
    S = _step(cache, offsets, slot, pos)
    code = _dtype_code(dtype, "dtype")
    slots, heads, d, cap = cache._dims
    device = cache.device
    shape = (int(total), heads, d)
    k = _out3(k, shape, dtype, device, "k")
    v = _out3(v, shape, dtype, device, "v")
    _call(_lib.q4_kvq_read, "q4_kvq_read", cache._index, stream, cache.data.data_ptr(), k.data_ptr(), v.data_ptr(), code, slots, heads,
          d, cap, offsets.data_ptr(), slot.data_ptr(), pos.data_ptr(), S, shape[0])
    return k, v


def q4_kvq_attention(cache: Q4KVCache, q: torch.Tensor, offsets: torch.Tensor, slot: torch.Tensor,
                     pos: torch.Tensor, scale: float | None = None, mass: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of the step's query rows over the cache, [total, q_heads, head_dim] of q's dtype.

    Row j of request s sees positions 0 .. pos[s] + j of its slot (append the
    step's rows first).  scale defaults to 1 / sqrt(head_dim).  mass, fp32
    [slots, heads, capacity], collects the weight that each position got.  out
    may be q itself (contiguous) where no mass is asked for, and overlaps nothing else.
    Uses the library's scratch, which the device's streams share: order calls on
    one stream.  The first call, or one of many more requests, allocates some.
    """
    S = _step(cache, offsets, slot, pos)
    dtype, device = q.dtype, cache.device
    code = _dtype_code(dtype, "q")
    slots, heads, d, cap = cache._dims
    hq = q.shape[1] if q.dim() == 3 else 0
    if hq == 0 or hq % heads:
        raise ValueError("q must be [total, q_heads, head_dim] with q_heads a multiple of %d" % heads)
    total, qs = _rows3(q, "q", hq, d, dtype, cache._index)
    out = _out3(out, (total, hq, d), dtype, device, "out")
    _call(_lib.q4_kvq_attention, "q4_kvq_attention", cache._index, stream, cache.data.data_ptr(), q.data_ptr(), out.data_ptr(),
          None if mass is None else _mass(cache, mass), code, slots, heads, hq, d, cap, qs,
          d ** -0.5 if scale is None else scale, offsets.data_ptr(), slot.data_ptr(), pos.data_ptr(), S, total)
    return out


def q4_kvq_evict(cache: Q4KVCache, mass: torch.Tensor, src: torch.Tensor, dst: torch.Tensor, length: torch.Tensor,
                 keep: int, recent: int = 0, stream=None):
    """Thin out slots by attention weight: (new_length int32 [S], kept int32 [S, heads, keep]).

    Each head of slot src[s] (length[s] positions) keeps its last `recent`
    positions and the others of largest mass, `keep` in all, moved in order
    to the front of slot dst[s] (the same slot: in place), mass alike.
    """
    device, index, keep = cache.device, cache._index, int(keep)
    S = _ints(index, src, "src")
    if _ints(index, dst, "dst") != S or _ints(index, length, "length") != S:
        raise ValueError("src, dst and length differ in length")
    mass_ptr = _mass(cache, mass)
    slots, heads, d, cap = cache._dims
    new_length = torch.empty((S,), dtype=_i32, device=device)
    kept = torch.empty((S, heads, max(keep, 0)), dtype=_i32, device=device)
    _call(_lib.q4_kvq_evict, "q4_kvq_evict", index, stream, cache.data.data_ptr(), mass_ptr, slots, heads, d, cap,
          src.data_ptr(), dst.data_ptr(), length.data_ptr(), S, keep, int(recent), new_length.data_ptr(),
          kept.data_ptr())
    return new_length, kept


def q4_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
                        k_offsets: torch.Tensor | None = None, causal: bool = True, scale: float | None = None,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention over packed prompts: q [q_total, q_heads, D], k and v [k_total, kv_heads, D] views
    (float16 or bfloat16), sequence s being rows offsets[s] .. offsets[s + 1].

    Causal rows are the last of their sequence's keys; k_offsets defaults to
    q_offsets and scale to 1 / sqrt(D).  out may be q itself (contiguous), and
    overlaps nothing else.
    """
    if q.dim() != 3 or k.dim() != 3 or k.shape[1] == 0 or q.shape[1] == 0 or q.shape[1] % k.shape[1]:
        raise ValueError("q must be [rows, q_heads, D] with q_heads a multiple of k's heads")
    dtype, device = q.dtype, q.device
    if dtype not in (torch.float16, torch.bfloat16) or not q.is_cuda:
        raise ValueError("q must be a float16 or bfloat16 CUDA tensor")
    if k_offsets is None:
        k_offsets = q_offsets
    index, hq, hk, d = q.get_device(), q.shape[1], k.shape[1], q.shape[2]
    tq, qs = _rows3(q, "q", hq, d, dtype, index)
    tk, ks = _rows3(k, "k", hk, d, dtype, index)
    tv, vs = _rows3(v, "v", hk, d, dtype, index)
    if tv != tk:
        raise ValueError("k and v differ in rows")
    S = _ints(index, q_offsets, "q_offsets") - 1
    if _ints(index, k_offsets, "k_offsets") != S + 1:
        raise ValueError("q_offsets and k_offsets differ in length")
    out = _out3(out, (tq, hq, d), dtype, device, "out")
    _call(_lib.q4_prompt_attention, "q4_prompt_attention", index, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          out.data_ptr(), _DTYPES[dtype], hq, hk, d, qs, ks, vs, d ** -0.5 if scale is None else scale,
          1 if causal else 0, q_offsets.data_ptr(), k_offsets.data_ptr(), S, tq, tk)
    return out


def q4mm_argmax_ex(W: Q4Weight, x: torch.Tensor, flags: int = 0, want_max: bool = True, stream=None):
    """Fused greedy pick: (idx int32 [M], maxval fp32 [M] or None)."""
    _dev_f32(x, "x")
    M = x.shape[0]
    if x.dim() != 2 or x.shape[1] != W.K:
        raise ValueError("x must be [M, %d]" % W.K)
    idx = torch.empty(M, dtype=torch.int32, device=x.device)
    mx = torch.empty(M, dtype=torch.float32, device=x.device) if want_max else None
    with torch.cuda.device(x.device):
        _check(_lib.q4mm_argmax_ex(W.handle, x.data_ptr(), idx.data_ptr(), mx.data_ptr() if mx is not None else None,
                                   M, int(flags), _stream(stream)), "q4mm_argmax_ex")
    return idx, mx


def q4mm_argmax(W: Q4Weight, x: torch.Tensor, want_max: bool = True, stream=None):
    _dev_f32(x, "x")
    M = x.shape[0]
    if x.dim() != 2 or x.shape[1] != W.K:
        raise ValueError("x must be [M, %d]" % W.K)
    idx = torch.empty(M, dtype=torch.int32, device=x.device)
    mx = torch.empty(M, dtype=torch.float32, device=x.device) if want_max else None
    with torch.cuda.device(x.device):
        _check(_lib.q4mm_argmax(W.handle, x.data_ptr(), idx.data_ptr(), mx.data_ptr() if mx is not None else None,
                                M, _stream(stream)), "q4mm_argmax")
    return idx, mx


def q4mm_select_path(W: Q4Weight, M: int, flags: int = 0) -> int:
    with torch.cuda.device(W.device):
        r = _lib.q4mm_select_path(W.handle, M, int(flags))
    if r < 0:
        raise Q4Error(-r, "q4mm_select_path")
    return r


def q4mm_plan_info(W: Q4Weight, M: int, flags: int = 0):
    """(path, kernel launches, K splits) that a call would use."""
    p, l, s = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    with torch.cuda.device(W.device):
        _check(_lib.q4mm_plan_info(W.handle, M, int(flags), ctypes.byref(p), ctypes.byref(l), ctypes.byref(s)),
               "q4mm_plan_info")
    return p.value, l.value, s.value


def q4mm_set_m_threshold(m: int):
    _check(_lib.q4mm_set_m_threshold(int(m)), "q4mm_set_m_threshold")


def q4mm_get_m_threshold() -> int:
    return int(_lib.q4mm_get_m_threshold())


def q4mm_set_group_m_threshold(m: int):
    _check(_lib.q4mm_set_group_m_threshold(int(m)), "q4mm_set_group_m_threshold")


def q4mm_get_group_m_threshold() -> int:
    return int(_lib.q4mm_get_group_m_threshold())


def q4mm_set_wait_limit_ns(ns: int):
    """Bound of the kernels' waits in ns for later launches (0: the default, 1 s)."""
    _check(_lib.q4mm_set_wait_limit_ns(int(ns)), "q4mm_set_wait_limit_ns")


def q4mm_set_stall_for_test(on: bool):
    """Test setting: later launches withhold their first hand-off so that waits run out."""
    _check(_lib.q4mm_set_stall_for_test(1 if on else 0), "q4mm_set_stall_for_test")


def q4_device_status() -> int:
    return int(_lib.q4_device_status())


def q4_scratch_bytes() -> tuple:
    """(partial, xop, gu, xpre): bytes of the library's scratch now held on the current device."""
    v = [ctypes.c_size_t(0) for _ in range(4)]
    _check(_lib.q4_scratch_bytes(*[ctypes.byref(a) for a in v]), "q4_scratch_bytes")
    return tuple(int(a.value) for a in v)


def raw_library() -> ctypes.CDLL:
    """The loaded ctypes library (for callers that marshal pointers themselves)."""
    return _lib
