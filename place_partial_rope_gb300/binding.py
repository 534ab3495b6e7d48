"""ctypes binding of ``librope_partial.so`` (C ABI: ``include/rope_partial.h``
and ``include/rope_serving.h``).

Argument marshalling only: every step of the operation runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  If the
library has not been built, loading raises -- there is no CPU fallback.

    rope_partial_inplace_fwd(x, r1, r2, start, end, stream=None)
    rope_partial_inplace_bwd(grad, r1, r2, start, end, stream=None)
    rope_partial_inplace_fwd_host(...), rope_partial_inplace_bwd_host(...)   (host tensors)

``x`` / ``grad``: contiguous CUDA tensor (B, S, N, D) of bf16, fp16 or fp32,
modified in place.  ``r1`` (cos) and ``r2`` (sin): 4-D CUDA tensors of the
same dtype and device that broadcast against ``x[..., start:end]`` (any
strides with a contiguous last dim; size-1 dims broadcast).  Both calls are
asynchronous on ``stream`` (default: torch's current stream of x's device).

Around them, for models with several position axes and for decoding over a
paged cache:

    rope_partial_inplace_fwd_axes / _bwd_axes(x, positions, sections, start, end, ...)
    KVCache(k, v, k_scale, v_scale)
    rope_partial_cache_write(cache, k, v, slots, cos, sin, start, end, mode)
    rope_partial_cache_read(cache, slots, k, v)
    rope_partial_tree_attention(q, cache, q_start, kv_len, page_table, out, ...)
    rope_partial_tree_mask(parents), tree_attention_workspace(q, cache, max_q)
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "librope_partial.so")

ROPE_OK, ROPE_ERR_NULLPTR, ROPE_ERR_INVALID, ROPE_ERR_CUDA = 0, 1, 2, 3
ROPE_BF16, ROPE_FP16, ROPE_FP32 = 0, 1, 2
ROPE_MODE_INTERLEAVE, ROPE_MODE_HALF = 1, 2
MODE_CODE = {"interleave": ROPE_MODE_INTERLEAVE, "half": ROPE_MODE_HALF}
ORDER_CODE = {"blocked": 0, "interleaved": 1}
SPECTRUM_CODE = {"shared": 0, "own": 1}
CACHE_CODE = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 3, torch.int8: 4}
DTYPE_CODE = {torch.bfloat16: ROPE_BF16, torch.float16: ROPE_FP16, torch.float32: ROPE_FP32}

_lib = None


class RopePlan(ctypes.Structure):
    """Mirror of ``rope_plan_t``."""
    _fields_ = [("path", ctypes.c_int32), ("vec_bytes", ctypes.c_int32),
                ("heads_per_thread", ctypes.c_int32), ("threads_per_block", ctypes.c_int32),
                ("blocks", ctypes.c_int64), ("tasks", ctypes.c_int64),
                ("chunks_per_row", ctypes.c_int32), ("r_per_head", ctypes.c_int32),
                ("launches", ctypes.c_int64)]


class RopeTokenRun(ctypes.Structure):
    """Mirror of ``rope_token_run_t``."""
    _fields_ = [("b0", ctypes.c_int64), ("s0", ctypes.c_int64), ("nb", ctypes.c_int64),
                ("ns", ctypes.c_int64)]


class RopeKVCache(ctypes.Structure):
    """Mirror of ``rope_kv_cache_t``."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("k_dim", ctypes.c_int64), ("v_dim", ctypes.c_int64),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("k_scale_stride", ctypes.c_int64 * 3), ("v_scale_stride", ctypes.c_int64 * 3),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class RopeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load the CUDA library once; raise if it is missing (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is not built; build it with `python -m place_partial_rope_gb300.build` "
            "(needs nvcc). There is no CPU fallback.")
    lib = ctypes.CDLL(_LIB_PATH)
    i64p = ctypes.POINTER(ctypes.c_int64)
    args = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
            ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, i64p, i64p, i64p, i64p,
            ctypes.c_int64, ctypes.c_int64]
    for name in ("rope_partial_inplace_fwd", "rope_partial_inplace_bwd",
                 "rope_partial_inplace_fwd_host", "rope_partial_inplace_bwd_host"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = args + [ctypes.c_void_p]
    for name in ("rope_partial_inplace_fwd_mode", "rope_partial_inplace_bwd_mode"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = args + [ctypes.c_int, ctypes.c_void_p]
    lib.rope_partial_plan_mode.restype = ctypes.c_int
    lib.rope_partial_plan_mode.argtypes = args + [ctypes.c_int, ctypes.c_int32,
                                                  ctypes.POINTER(RopePlan)]
    pos_args = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int] + [ctypes.c_int64] * 4 + \
        [i64p, i64p, ctypes.c_double, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]
    for name in ("rope_partial_inplace_fwd_pos", "rope_partial_inplace_bwd_pos"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = pos_args
    qk = [ctypes.c_void_p] * 4 + [ctypes.c_int] + [ctypes.c_int64] * 10 + [i64p] * 4 + [ctypes.c_void_p]
    for name in ("rope_partial_inplace_fwd_qk", "rope_partial_inplace_bwd_qk"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = qk
    lib.rope_partial_plan.restype = ctypes.c_int
    lib.rope_partial_plan.argtypes = args + [ctypes.c_int32, ctypes.POINTER(RopePlan)]
    lib.rope_partial_token_shard.restype = ctypes.c_int
    lib.rope_partial_token_shard.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                             ctypes.c_int32, i64p, i64p,
                                             ctypes.POINTER(RopeTokenRun), ctypes.POINTER(ctypes.c_int32)]
    vp, i64, i32, d = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double
    for name in ("rope_partial_inplace_fwd_axes", "rope_partial_inplace_bwd_axes"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [vp, vp, ctypes.c_int, i64, i64, i64, i64, i32, vp, i64p, i64p, ctypes.c_int,
                       ctypes.c_int, d, i64, i64, ctypes.c_int, vp]
    for name, argtypes in (
            ("rope_partial_cache_write", [vp, vp, vp, ctypes.c_int, i64, i64p, i64p, vp, vp, vp, i64, i64,
                                          i64, i64, ctypes.c_int, vp]),
            ("rope_partial_cache_read", [vp, vp, i64, vp, vp, ctypes.c_int, i64p, i64p, vp]),
            ("rope_partial_tree_attention", [vp, vp, ctypes.c_int, i64, i64, i64p, vp, vp, i64, i64, vp,
                                             i64, i64, vp, i64, vp, i64p, vp, d, vp, i64, vp]),
            ("rope_partial_tree_attention_workspace", [vp, ctypes.c_int, i64, i64, i32, i64p]),
            ("rope_partial_tree_mask", [vp, i64, i64, vp])):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = argtypes
    lib.rope_status_str.restype = ctypes.c_char_p
    lib.rope_status_str.argtypes = [ctypes.c_int]
    lib.rope_last_error_message.restype = ctypes.c_char_p
    lib.rope_last_error_message.argtypes = []
    _lib = lib
    return lib


def _i64x4(vals):
    return (ctypes.c_int64 * 4)(*[int(v) for v in vals])


def _raise_for(lib, status: int):
    if status != ROPE_OK:
        name = lib.rope_status_str(status).decode()
        msg = lib.rope_last_error_message().decode()
        raise RopeError(status, f"{name}: {msg}")


def _stream_handle(stream, device) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _marshal(x: torch.Tensor, r1: torch.Tensor, r2: torch.Tensor, host: bool = False):
    if x.dim() != 4:
        raise RopeError(ROPE_ERR_INVALID, f"x must be 4-D (B, S, N, D), got {x.dim()}-D")
    if r1.dim() != 4 or r2.dim() != 4:
        raise RopeError(ROPE_ERR_INVALID, "r1 and r2 must be 4-D")
    if x.dtype not in DTYPE_CODE:
        raise RopeError(ROPE_ERR_INVALID, f"unsupported dtype {x.dtype}")
    if r1.dtype != x.dtype or r2.dtype != x.dtype:
        raise RopeError(ROPE_ERR_INVALID, "r1, r2 and x must share one dtype")
    if not x.is_contiguous():
        raise RopeError(ROPE_ERR_INVALID, "x must be contiguous")
    for t in (x, r1, r2):
        if host and t.is_cuda:
            raise RopeError(ROPE_ERR_INVALID, "the *_host calls take CPU (host) tensors")
        if not host and (not t.is_cuda or t.device != x.device):
            raise RopeError(ROPE_ERR_INVALID, "x, r1 and r2 must be CUDA tensors on one device")
    return (x.data_ptr(), r1.data_ptr(), r2.data_ptr(), DTYPE_CODE[x.dtype], *x.shape,
            _i64x4(r1.shape), _i64x4(r1.stride()), _i64x4(r2.shape), _i64x4(r2.stride()))


def _mode_code(mode) -> int:
    if mode in MODE_CODE:
        return MODE_CODE[mode]
    raise RopeError(ROPE_ERR_INVALID, f"rotary mode {mode!r} is not 'interleave' or 'half'")


def _call(name: str, x, r1, r2, start: int, end: int, stream=None, mode=None) -> None:
    lib = load_library()
    margs = _marshal(x, r1, r2)
    extra = () if mode is None else (_mode_code(mode),)
    with torch.cuda.device(x.device):
        st = getattr(lib, name)(*margs, int(start), int(end), *extra,
                                _stream_handle(stream, x.device))
    _raise_for(lib, st)


def rope_partial_inplace_fwd(x: torch.Tensor, r1: torch.Tensor, r2: torch.Tensor, start: int,
                             end: int, stream=None) -> None:
    """Rotate ``x[..., start:end]`` in place (forward)."""
    _call("rope_partial_inplace_fwd", x, r1, r2, start, end, stream)


def rope_partial_inplace_bwd(grad: torch.Tensor, r1: torch.Tensor, r2: torch.Tensor, start: int,
                             end: int, stream=None) -> None:
    """Overwrite ``grad[..., start:end]`` with the transposed rotation (backward)."""
    _call("rope_partial_inplace_bwd", grad, r1, r2, start, end, stream)


def rope_partial_inplace_fwd_mode(x, r1, r2, start: int, end: int, mode: str = "interleave",
                                  stream=None) -> None:
    """The forward in rotary mode ``"interleave"`` or ``"half"`` (pairs
    (i, i + L/2))."""
    _call("rope_partial_inplace_fwd_mode", x, r1, r2, start, end, stream, mode)


def rope_partial_inplace_bwd_mode(grad, r1, r2, start: int, end: int, mode: str = "interleave",
                                  stream=None) -> None:
    """The backward in rotary mode ``"interleave"`` or ``"half"``."""
    _call("rope_partial_inplace_bwd_mode", grad, r1, r2, start, end, stream, mode)


def _call_host(name: str, x, r1, r2, start: int, end: int, stream=None) -> None:
    lib = load_library()
    margs = _marshal(x, r1, r2, host=True)
    handle = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else (
        torch.cuda.current_stream().cuda_stream if stream is None else int(stream))
    st = getattr(lib, name)(*margs, int(start), int(end), handle)
    _raise_for(lib, st)


def rope_partial_inplace_fwd_host(x: torch.Tensor, r1: torch.Tensor, r2: torch.Tensor,
                                  start: int, end: int, stream=None) -> None:
    """Forward on host tensors, read and written in place by the GPU (zero
    copy).  x, r1 and r2 are CPU tensors the current CUDA device can reach
    (pinned memory, or any memory on devices with pageable-memory access).
    Asynchronous: synchronise the stream before reading x on the host."""
    _call_host("rope_partial_inplace_fwd_host", x, r1, r2, start, end, stream)


def rope_partial_inplace_bwd_host(grad: torch.Tensor, r1: torch.Tensor, r2: torch.Tensor,
                                  start: int, end: int, stream=None) -> None:
    """Backward on host tensors (zero copy); see rope_partial_inplace_fwd_host."""
    _call_host("rope_partial_inplace_bwd_host", grad, r1, r2, start, end, stream)


def _qk_args(q, k, r1, r2, q_slice, k_slice, stream):
    if q.dim() != 4 or k.dim() != 4:
        raise RopeError(ROPE_ERR_INVALID, "q and k must be 4-D (B, S, N, D)")
    if q.shape[:2] != k.shape[:2]:
        raise RopeError(ROPE_ERR_INVALID, "q and k must share B and S")
    if k.dtype != q.dtype or not k.is_contiguous() or not k.is_cuda or k.device != q.device:
        raise RopeError(ROPE_ERR_INVALID, "k must be a contiguous CUDA tensor of q's dtype and device")
    m = _marshal(q, r1, r2)
    B, S, Nq, Dq = q.shape
    Nk, Dk = k.shape[2], k.shape[3]
    return (q.data_ptr(), k.data_ptr(), r1.data_ptr(), r2.data_ptr(), m[3], B, S, Nq, Dq,
            int(q_slice[0]), int(q_slice[1]), Nk, Dk, int(k_slice[0]), int(k_slice[1]),
            m[8], m[9], m[10], m[11], _stream_handle(stream, q.device))


def rope_partial_inplace_fwd_qk(q, k, r1, r2, q_slice, k_slice, stream=None) -> None:
    """Rotate ``q[..., q_slice]`` and ``k[..., k_slice]`` in place in one
    launch with the same cos/sin rows (shape (B|1, S|1, 1, L))."""
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.rope_partial_inplace_fwd_qk(*_qk_args(q, k, r1, r2, q_slice, k_slice, stream))
    _raise_for(lib, st)


def rope_partial_inplace_bwd_qk(dq, dk, r1, r2, q_slice, k_slice, stream=None) -> None:
    """Backward of rope_partial_inplace_fwd_qk on the two gradients, in place."""
    lib = load_library()
    with torch.cuda.device(dq.device):
        st = lib.rope_partial_inplace_bwd_qk(*_qk_args(dq, dk, r1, r2, q_slice, k_slice, stream))
    _raise_for(lib, st)


def _pos_args(x, positions, start, end, base, mode, stream):
    if x.dim() != 4:
        raise RopeError(ROPE_ERR_INVALID, f"x must be 4-D (B, S, N, D), got {x.dim()}-D")
    if x.dtype not in DTYPE_CODE:
        raise RopeError(ROPE_ERR_INVALID, f"unsupported dtype {x.dtype}")
    if not x.is_contiguous() or not x.is_cuda:
        raise RopeError(ROPE_ERR_INVALID, "x must be a contiguous CUDA tensor")
    if positions.dim() != 2 or positions.dtype != torch.int32:
        raise RopeError(ROPE_ERR_INVALID, "positions must be a 2-D int32 tensor (B|1, S|1)")
    if not positions.is_cuda or positions.device != x.device:
        raise RopeError(ROPE_ERR_INVALID, "positions must be on x's device")
    p_shape = (ctypes.c_int64 * 2)(*positions.shape)
    p_stride = (ctypes.c_int64 * 2)(*positions.stride())
    return (x.data_ptr(), positions.data_ptr(), DTYPE_CODE[x.dtype], *x.shape, p_shape, p_stride,
            float(base), int(start), int(end), _mode_code(mode), _stream_handle(stream, x.device))


def rope_partial_inplace_fwd_pos(x, positions, start: int, end: int, base: float = 10000.0,
                                 mode: str = "interleave", stream=None) -> None:
    """Forward with cos/sin computed in the kernel from int32 positions of
    shape (B|1, S|1): theta_k = p / base^(2k/L)."""
    lib = load_library()
    with torch.cuda.device(x.device):
        st = lib.rope_partial_inplace_fwd_pos(*_pos_args(x, positions, start, end, base, mode, stream))
    _raise_for(lib, st)


def rope_partial_inplace_bwd_pos(grad, positions, start: int, end: int, base: float = 10000.0,
                                 mode: str = "interleave", stream=None) -> None:
    """Backward of rope_partial_inplace_fwd_pos, in place on the gradient."""
    lib = load_library()
    with torch.cuda.device(grad.device):
        st = lib.rope_partial_inplace_bwd_pos(*_pos_args(grad, positions, start, end, base, mode,
                                                          stream))
    _raise_for(lib, st)


def _on_device(dev: int, fn, args) -> int:
    """Call fn(*args) with `dev` as the current CUDA device (the device the
    prepared tensors and stream belong to)."""
    if torch.cuda.current_device() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


class PreparedPos:
    """rope_partial_inplace_{fwd,bwd}_pos with arguments marshalled once."""

    def __init__(self, direction: str, x, positions, start, end, base=10000.0, mode="interleave",
                 stream=None):
        self._lib = load_library()
        self._fn = getattr(self._lib, f"rope_partial_inplace_{direction}_pos")
        self._keep = (x, positions)
        self._args = _pos_args(x, positions, start, end, base, mode, stream)
        self._dev = x.device.index

    def __call__(self) -> None:
        st = _on_device(self._dev, self._fn, self._args)
        if st != ROPE_OK:
            _raise_for(self._lib, st)


class PreparedQK:
    """rope_partial_inplace_{fwd,bwd}_qk with arguments marshalled once."""

    def __init__(self, direction: str, q, k, r1, r2, q_slice, k_slice, stream=None):
        self._lib = load_library()
        self._fn = getattr(self._lib, f"rope_partial_inplace_{direction}_qk")
        self._keep = (q, k, r1, r2)
        self._args = _qk_args(q, k, r1, r2, q_slice, k_slice, stream)
        self._dev = q.device.index

    def __call__(self) -> None:
        st = _on_device(self._dev, self._fn, self._args)
        if st != ROPE_OK:
            _raise_for(self._lib, st)


class PreparedCall:
    """One forward or backward call with its arguments marshalled once.

    Calling the object launches the kernel again on the same tensors and
    stream (for loops that launch the same call many times, where per-call
    marshalling would cost more host time than the kernel takes).  It keeps
    references to the tensors so their memory stays alive.
    """

    def __init__(self, name: str, x, r1, r2, start: int, end: int, stream=None, mode=None):
        self._lib = load_library()
        self._fn = getattr(self._lib, name)
        self._keep = (x, r1, r2)
        host = name.endswith("_host")
        dev = torch.device("cuda", torch.cuda.current_device()) if host else x.device
        extra = () if mode is None else (_mode_code(mode),)
        self._args = (*_marshal(x, r1, r2, host=host), int(start), int(end), *extra,
                      _stream_handle(stream, dev))
        self._dev = dev.index if dev.index is not None else torch.cuda.current_device()

    def __call__(self) -> None:
        st = _on_device(self._dev, self._fn, self._args)
        if st != ROPE_OK:
            _raise_for(self._lib, st)


def prepare_fwd(x, r1, r2, start: int, end: int, stream=None, mode=None) -> PreparedCall:
    """``rope_partial_inplace_fwd`` (``_fwd_mode`` when a mode is given) with
    its arguments marshalled once."""
    name = "rope_partial_inplace_fwd" if mode is None else "rope_partial_inplace_fwd_mode"
    return PreparedCall(name, x, r1, r2, start, end, stream, mode)


def prepare_bwd(grad, r1, r2, start: int, end: int, stream=None, mode=None) -> PreparedCall:
    """``rope_partial_inplace_bwd`` (``_bwd_mode`` when a mode is given) with
    its arguments marshalled once."""
    name = "rope_partial_inplace_bwd" if mode is None else "rope_partial_inplace_bwd_mode"
    return PreparedCall(name, grad, r1, r2, start, end, stream, mode)


def prepare_fwd_host(x, r1, r2, start: int, end: int, stream=None) -> PreparedCall:
    """``rope_partial_inplace_fwd_host`` with its arguments marshalled once."""
    return PreparedCall("rope_partial_inplace_fwd_host", x, r1, r2, start, end, stream)


def prepare_bwd_host(grad, r1, r2, start: int, end: int, stream=None) -> PreparedCall:
    """``rope_partial_inplace_bwd_host`` with its arguments marshalled once."""
    return PreparedCall("rope_partial_inplace_bwd_host", grad, r1, r2, start, end, stream)


def rope_partial_plan(x: torch.Tensor, r1: torch.Tensor, r2: torch.Tensor, start: int, end: int,
                      sm_count: int = 0, mode: str = "interleave") -> RopePlan:
    """The launch plan the forward would use (no launch).  Works on CPU
    tensors as well when ``sm_count`` > 0, since only shapes, strides and
    pointer alignment are read."""
    lib = load_library()
    plan = RopePlan()
    args = (x.data_ptr(), r1.data_ptr(), r2.data_ptr(), DTYPE_CODE[x.dtype], *x.shape,
            _i64x4(r1.shape), _i64x4(r1.stride()), _i64x4(r2.shape), _i64x4(r2.stride()))
    st = lib.rope_partial_plan_mode(*args, int(start), int(end), _mode_code(mode), int(sm_count),
                                    ctypes.byref(plan))
    _raise_for(lib, st)
    return plan


def rope_partial_token_shard(B: int, S: int, rank: int, world: int):
    """Rank ``rank`` of ``world``'s tokens of a (B, S) grid: ``(t0, t1, runs)``
    with runs as ``(b0, s0, nb, ns)`` tuples (host only, no CUDA call)."""
    lib = load_library()
    t0, t1, n = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32()
    runs = (RopeTokenRun * 3)()
    st = lib.rope_partial_token_shard(B, S, rank, world, ctypes.byref(t0), ctypes.byref(t1), runs,
                                      ctypes.byref(n))
    _raise_for(lib, st)
    return t0.value, t1.value, [(r.b0, r.s0, r.nb, r.ns) for r in runs[:n.value]]


# ------------------------------------------------------------------------
# rotary positions with several axes, the paged cache and attention over it
# ------------------------------------------------------------------------

_I64x2 = ctypes.c_int64 * 2
_I64x3 = ctypes.c_int64 * 3
# the handle of torch's current stream of a device, without a Stream object
# around it (a microsecond less per call); the public way where it is missing
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch(fn, args, stream, device) -> None:
    """Call fn(*args, stream) with `device` current; raise on an error status."""
    if stream is None and _raw_stream is not None:
        handle = _raw_stream(device.index)
    else:
        handle = _stream_handle(stream, device)
    if torch.cuda.current_device() == device.index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != ROPE_OK:
        _raise_for(_lib, st)


def _require(cond, message: str) -> None:
    if not cond:
        raise RopeError(ROPE_ERR_INVALID, message)


def _axes_call(name, x, positions, sections, start, end, base, mode, order, spectrum, stream):
    lib = _lib or load_library()
    _require(x.dim() == 4, "x must be 4-D (B, S, N, D)")
    _require(x.dtype in DTYPE_CODE, f"unsupported dtype {x.dtype}")
    _require(x.is_cuda and x.is_contiguous(), "x must be a contiguous CUDA tensor")
    _require(positions.dim() == 3 and positions.dtype == torch.int32,
             "positions must be a 3-D int32 tensor (axes, B|1, S|1)")
    _require(positions.device == x.device, "positions must be on x's device")
    _require(order in ORDER_CODE, f"order {order!r} is not 'blocked' or 'interleaved'")
    _require(spectrum in SPECTRUM_CODE, f"spectrum {spectrum!r} is not 'shared' or 'own'")
    n = len(sections)
    _require(n == positions.shape[0], "there must be one section for each axis of the positions")
    _launch(getattr(lib, name),
            (x.data_ptr(), positions.data_ptr(), DTYPE_CODE[x.dtype], *x.shape, n,
             (ctypes.c_int32 * n)(*sections), _I64x3(*positions.shape), _I64x3(*positions.stride()),
             ORDER_CODE[order], SPECTRUM_CODE[spectrum], base, start, end, _mode_code(mode)),
            stream, x.device)


def rope_partial_inplace_fwd_axes(x, positions, sections, start: int, end: int, base: float = 10000.0,
                                  mode: str = "interleave", order: str = "blocked",
                                  spectrum: str = "shared", stream=None) -> None:
    """Forward with several position axes: ``sections[a]`` of the slice's pairs
    turn by ``positions[a]`` (int32, shape (axes, B|1, S|1)), in blocks or
    dealt in turn (``order``), with frequencies base^(-2k/L) over the slice
    (``spectrum="shared"``) or base^(-j/sections[a]) over each axis ("own")."""
    _axes_call("rope_partial_inplace_fwd_axes", x, positions, sections, start, end, base, mode, order,
               spectrum, stream)


def rope_partial_inplace_bwd_axes(grad, positions, sections, start: int, end: int,
                                  base: float = 10000.0, mode: str = "interleave",
                                  order: str = "blocked", spectrum: str = "shared", stream=None) -> None:
    """Backward of rope_partial_inplace_fwd_axes, in place on the gradient."""
    _axes_call("rope_partial_inplace_bwd_axes", grad, positions, sections, start, end, base, mode, order,
               spectrum, stream)


class KVCache:
    """The handle of a paged cache that a program keeps beside its tensors:
    ``k`` (pages, page_size, heads, k_dim) and ``v`` (..., v_dim) of one type
    (bf16, fp16, float8_e4m3fn or int8), in any strides with a contiguous last
    dim, and for the 8-bit types fp32 ``k_scale`` and ``v_scale`` (pages,
    page_size, heads).  ``v`` may be None (keys only)."""

    def __init__(self, k, v=None, k_scale=None, v_scale=None):
        tensors = [t for t in (k, v, k_scale, v_scale) if t is not None]
        _require(k.dim() == 4 and (v is None or v.dim() == 4),
                 "k and v must be 4-D (pages, page_size, heads, dim)")
        _require(k.dtype in CACHE_CODE and (v is None or v.dtype == k.dtype),
                 f"unsupported cache dtype {k.dtype}, or v of another")
        _require(v is None or v.shape[:3] == k.shape[:3], "k and v must share pages, page_size and heads")
        _require(all(t.is_cuda and t.device == k.device for t in tensors),
                 "the cache must be CUDA tensors on one device")
        for t in (k, v):
            _require(t is None or t.shape[3] <= 1 or t.stride(3) == 1,
                     "the last dim of k and v must be contiguous")
        for t in (k_scale, v_scale):
            _require(t is None or (t.dtype == torch.float32 and t.shape == k.shape[:3]),
                     "scales must be fp32 (pages, page_size, heads)")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.device

        def ptr(t):
            return None if t is None else t.data_ptr()

        def strides(t):
            return _I64x3(*t.stride()[:3]) if t is not None else _I64x3()

        self._c = RopeKVCache(ptr(k), ptr(v), ptr(k_scale), ptr(v_scale), *k.shape,
                              0 if v is None else v.shape[3], strides(k), strides(v),
                              strides(k_scale), strides(v_scale), CACHE_CODE[k.dtype], 0)
        self._ref = ctypes.addressof(self._c)


def _rows_of(t, cache, dim, what):
    _require(t.dim() == 3 and t.shape[1] == cache._c.heads and t.shape[2] == dim,
             f"{what} must be (tokens, {cache._c.heads}, {dim})")
    _require(t.device == cache.device, f"{what} must be on the cache's device")
    _require(t.shape[2] <= 1 or t.stride(2) == 1, f"the last dim of {what} must be contiguous")
    return t.data_ptr(), _I64x2(*t.stride()[:2])


def _slots_of(slots, cache, tokens):
    _require(slots.dtype == torch.int64 and slots.dim() == 1 and slots.is_contiguous() and
             slots.device == cache.device and (tokens is None or slots.shape[0] == tokens),
             "slots must be a contiguous int64 vector on the cache's device, one per token")
    return slots.data_ptr()


def rope_partial_cache_write(cache: KVCache, k, v, slots, cos=None, sin=None, start: int = 0,
                             end: int = 0, mode: str = "interleave", stream=None) -> None:
    """Rotate lanes [start, end) of the keys ``k`` (T, heads, k_dim) by the rows
    of ``cos`` and ``sin`` ((T|1), end - start; None: no rotation) and put them
    and ``v`` (T, heads, v_dim) at ``slots`` (int64; one outside the cache
    skips its token), quantised where the cache holds 8 bits.  k and v stay as
    they are."""
    lib = _lib or load_library()
    c = cache._c
    _require(k.dtype in DTYPE_CODE and (v is None or v.dtype == k.dtype),
             f"unsupported dtype {k.dtype}, or v of another")
    kp, ks = _rows_of(k, cache, c.k_dim, "k")
    vp, vs = (None, None)
    if v is not None:
        vp, vs = _rows_of(v, cache, c.v_dim, "v")
        _require(v.shape[0] == k.shape[0], "k and v must hold the same tokens")
    T = k.shape[0]
    cp = sp = None
    cst = sst = 0
    if cos is not None or sin is not None:
        for t in (cos, sin):
            _require(t is not None and t.dim() == 2 and t.dtype == k.dtype and t.device == cache.device and
                     t.shape[0] in (1, T) and t.shape[1] == end - start and
                     (t.shape[1] <= 1 or t.stride(1) == 1),
                     "cos and sin must be (tokens or 1, end - start) of k's dtype with a contiguous last dim")
        cp, sp = cos.data_ptr(), sin.data_ptr()
        cst = cos.stride(0) if cos.shape[0] > 1 else 0
        sst = sin.stride(0) if sin.shape[0] > 1 else 0
    _launch(lib.rope_partial_cache_write,
            (cache._ref, kp, vp, DTYPE_CODE[k.dtype], T, ks, vs, _slots_of(slots, cache, T), cp, sp, cst,
             sst, start, end, _mode_code(mode)), stream, cache.device)


def rope_partial_cache_read(cache: KVCache, slots, k=None, v=None, stream=None) -> None:
    """The rows at ``slots`` as numbers, into ``k`` (T, heads, k_dim) and ``v``
    (T, heads, v_dim), either of which may be None; a slot outside the cache
    gives zeros."""
    lib = _lib or load_library()
    c = cache._c
    kp = ks = vp = vs = None
    T, dtype = slots.shape[0], None
    for t in (k, v):
        if t is not None:
            _require(t.dtype in DTYPE_CODE and dtype in (None, t.dtype), "k and v must share a dtype")
            _require(t.shape[0] == T, "k and v must have a row for each slot")
            dtype = t.dtype
    if dtype is None:
        return
    if k is not None:
        kp, ks = _rows_of(k, cache, c.k_dim, "k")
    if v is not None:
        vp, vs = _rows_of(v, cache, c.v_dim, "v")
    _launch(lib.rope_partial_cache_read,
            (cache._ref, _slots_of(slots, cache, T), T, kp, vp, DTYPE_CODE[dtype], ks, vs), stream,
            cache.device)


def rope_partial_tree_mask(parents) -> torch.Tensor:
    """The int64 tree words (n, ceil(n / 64)) of one request's drafted tokens
    from their parents (a sequence: an earlier token, or -1 for the context).
    On the host; join several requests' rows and copy them to the device."""
    lib = _lib or load_library()
    p = torch.as_tensor(parents, dtype=torch.int32, device="cpu").contiguous()
    n = p.numel()
    words = torch.zeros((n, max(1, (n + 63) // 64)), dtype=torch.int64)
    st = lib.rope_partial_tree_mask(p.data_ptr(), n, words.shape[1], words.data_ptr())
    _raise_for(lib, st)
    return words


def tree_attention_workspace(q, cache: KVCache, max_q: int) -> torch.Tensor:
    """A workspace for rope_partial_tree_attention with such a ``q``, ``cache``
    and ``max_q``.  A program keeps it: calls that follow each other on one
    stream can share it."""
    lib = _lib or load_library()
    _require(q.dim() == 3 and q.dtype in DTYPE_CODE, "q must be (tokens, heads, dim) of bf16 or fp16")
    need = ctypes.c_int64()
    with torch.cuda.device(cache.device):
        st = lib.rope_partial_tree_attention_workspace(cache._ref, DTYPE_CODE[q.dtype], q.shape[1],
                                                       int(max_q), 0, ctypes.byref(need))
    _raise_for(lib, st)
    return torch.empty(need.value, dtype=torch.uint8, device=cache.device)


def rope_partial_tree_attention(q, cache: KVCache, q_start, kv_len, page_table, out, lse=None, tree=None,
                                scale=None, max_q=None, workspace=None, stream=None) -> None:
    """Attention of drafted tokens over the cache, into ``out`` (Tq, Hq, v_dim)
    and, where given, ``lse`` (Tq, Hq) fp32.

    ``q`` (Tq, Hq, k_dim); request r has the tokens [q_start[r], q_start[r+1])
    and kv_len[r] cached rows, the last of which are those tokens' own, in the
    pages page_table[r] (int32).  ``tree`` (Tq, words) int64 holds the bits of
    the drafted tokens that each token sees (``rope_partial_tree_mask``); None
    is a chain.  ``scale`` defaults to 1 / sqrt(k_dim), ``max_q`` (the most
    tokens of a request) to Tq, and the workspace is made for the call when
    none is given."""
    lib = _lib or load_library()
    c = cache._c
    _require(q.dim() == 3 and q.shape[2] == c.k_dim and q.dtype in DTYPE_CODE,
             f"q must be (tokens, heads, {c.k_dim}) of bf16 or fp16")
    Tq, Hq = q.shape[0], q.shape[1]
    _require(out.dtype == q.dtype and out.shape == (Tq, Hq, c.v_dim),
             f"out must be ({Tq}, {Hq}, {c.v_dim}) of q's dtype")
    _require((q.stride(2) == 1 or c.k_dim == 1) and (out.stride(2) == 1 or c.v_dim == 1),
             "the last dim of q and out must be contiguous")
    R = kv_len.shape[0]
    _require(q_start.dtype == torch.int32 and kv_len.dtype == torch.int32 and
             q_start.shape == (R + 1,) and kv_len.dim() == 1 and q_start.is_contiguous() and
             kv_len.is_contiguous(), "q_start and kv_len must be contiguous int32 vectors of R + 1 and R")
    _require(page_table.dtype == torch.int32 and page_table.dim() == 2 and page_table.shape[0] == R and
             (page_table.shape[1] <= 1 or page_table.stride(1) == 1),
             "page_table must be int32 (R, pages) with a contiguous last dim")
    _require(lse is None or (lse.dtype == torch.float32 and lse.shape == (Tq, Hq) and lse.is_contiguous()),
             "lse must be contiguous fp32 (Tq, Hq)")
    _require(tree is None or (tree.dtype == torch.int64 and tree.dim() == 2 and tree.shape[0] == Tq and
                              tree.is_contiguous()), "tree must be contiguous int64 (Tq, words)")
    dev = cache.device
    for t in (q, out, q_start, kv_len, page_table, lse, tree, workspace):
        _require(t is None or t.device == dev, "every tensor must be on the cache's device")
    if max_q is None:
        max_q = max(1, Tq)
    if workspace is None:
        workspace = tree_attention_workspace(q, cache, max_q)
        if stream is not None:
            # made on the current stream, used on another: the allocator must know
            workspace.record_stream(stream if isinstance(stream, torch.cuda.Stream)
                                    else torch.cuda.ExternalStream(int(stream), device=dev))
    _require(workspace.is_contiguous(), "workspace must be contiguous")
    _launch(lib.rope_partial_tree_attention,
            (cache._ref, q.data_ptr(), DTYPE_CODE[q.dtype], Tq, Hq, _I64x2(*q.stride()[:2]),
             q_start.data_ptr(), kv_len.data_ptr(), R, max_q, page_table.data_ptr(), page_table.shape[1],
             page_table.stride(0) if R > 1 else page_table.shape[1],
             None if tree is None else tree.data_ptr(), 0 if tree is None else tree.shape[1],
             out.data_ptr(), _I64x2(*out.stride()[:2]), None if lse is None else lse.data_ptr(),
             c.k_dim ** -0.5 if scale is None else scale, workspace.data_ptr(),
             workspace.numel() * workspace.element_size()), stream, dev)
