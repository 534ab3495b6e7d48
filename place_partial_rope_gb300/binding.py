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
import struct

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
        fn.argtypes = [vp, vp, ctypes.c_int, i64, i64, i64, i64, i32, vp, vp, vp, ctypes.c_int,
                       ctypes.c_int, d, i64, i64, ctypes.c_int, vp]
    for name, argtypes in (
            ("rope_partial_cache_write", [vp, vp, vp, ctypes.c_int, i64, vp, vp, vp, vp, vp, i64, i64,
                                          i64, i64, ctypes.c_int, vp]),
            ("rope_partial_cache_read", [vp, vp, i64, vp, vp, ctypes.c_int, vp, vp, vp]),
            ("rope_partial_tree_attention", [vp, vp, ctypes.c_int, i64, i64, vp, vp, vp, i64, i64, vp,
                                             i64, i64, vp, i64, vp, vp, vp, d, vp, i64, vp]),
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


def _stream_of(stream, device):
    """The stream object of what a call takes as ``stream`` (not None)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(stream)
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


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

# Small host arrays go to the library as packed bytes: making them is a call,
# where a ctypes array is several (these calls are short enough for that to
# count).  Checks raise through _refuse only where they fail, so that no message
# is put together for a call that is right.
_pack2, _pack3 = struct.Struct("=2q").pack, struct.Struct("=3q").pack
# the handle of torch's current stream of a device, and the current device,
# without a Stream object or a context around them; the public ways where these
# are missing
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(fn, args, stream, device) -> None:
    """Call fn(*args, stream) with `device` current; raise on an error status."""
    index = device.index
    if stream is None and _raw_stream is not None:
        handle = _raw_stream(index)
    else:
        handle = _stream_handle(stream, device)
    if _current_device() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != ROPE_OK:
        _raise_for(_lib, st)


def _refuse(message: str):
    raise RopeError(ROPE_ERR_INVALID, message)


def _axes_call(name, x, positions, sections, start, end, base, mode, order, spectrum, stream):
    lib = _lib or load_library()
    if x.dim() != 4:
        _refuse("x must be 4-D (B, S, N, D)")
    dtype = DTYPE_CODE.get(x.dtype)
    if dtype is None:
        _refuse(f"unsupported dtype {x.dtype}")
    if not x.is_cuda or not x.is_contiguous():
        _refuse("x must be a contiguous CUDA tensor")
    if positions.dim() != 3 or positions.dtype is not torch.int32:
        _refuse("positions must be a 3-D int32 tensor (axes, B|1, S|1)")
    device = x.device
    if positions.device != device:
        _refuse("positions must be on x's device")
    if order not in ORDER_CODE:
        _refuse(f"order {order!r} is not 'blocked' or 'interleaved'")
    if spectrum not in SPECTRUM_CODE:
        _refuse(f"spectrum {spectrum!r} is not 'shared' or 'own'")
    if mode not in MODE_CODE:
        _mode_code(mode)
    n, shape = len(sections), positions.shape
    if n != shape[0]:
        _refuse("there must be one section for each axis of the positions")
    _launch(getattr(lib, name),
            (x.data_ptr(), positions.data_ptr(), dtype, *x.shape, n, struct.pack(f"={n}i", *sections),
             _pack3(*shape), _pack3(*positions.stride()), ORDER_CODE[order], SPECTRUM_CODE[spectrum], base,
             start, end, MODE_CODE[mode]), stream, device)


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
        if k.dim() != 4 or (v is not None and v.dim() != 4):
            _refuse("k and v must be 4-D (pages, page_size, heads, dim)")
        if k.dtype not in CACHE_CODE or (v is not None and v.dtype != k.dtype):
            _refuse(f"unsupported cache dtype {k.dtype}, or v of another")
        if v is not None and v.shape[:3] != k.shape[:3]:
            _refuse("k and v must share pages, page_size and heads")
        for t in (k, v, k_scale, v_scale):
            if t is not None and (not t.is_cuda or t.device != k.device):
                _refuse("the cache must be CUDA tensors on one device")
        for t in (k, v):
            if t is not None and t.shape[3] > 1 and t.stride(3) != 1:
                _refuse("the last dim of k and v must be contiguous")
        for t in (k_scale, v_scale):
            if t is not None and (t.dtype != torch.float32 or t.shape != k.shape[:3]):
                _refuse("scales must be fp32 (pages, page_size, heads)")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.device
        self.heads, self.k_dim, self.v_dim = k.shape[2], k.shape[3], 0 if v is None else v.shape[3]

        def ptr(t):
            return None if t is None else t.data_ptr()

        def strides(t):
            return (ctypes.c_int64 * 3)(*(t.stride()[:3] if t is not None else ()))

        self._c = RopeKVCache(ptr(k), ptr(v), ptr(k_scale), ptr(v_scale), *k.shape, self.v_dim,
                              strides(k), strides(v), strides(k_scale), strides(v_scale),
                              CACHE_CODE[k.dtype], 0)
        self._ref = ctypes.addressof(self._c)


def _rows_of(t, cache, dim, what):
    shape = t.shape
    if len(shape) != 3 or shape[1] != cache.heads or shape[2] != dim:
        _refuse(f"{what} must be (tokens, {cache.heads}, {dim})")
    if t.device != cache.device:
        _refuse(f"{what} must be on the cache's device")
    st = t.stride()
    if st[2] != 1 and dim > 1:
        _refuse(f"the last dim of {what} must be contiguous")
    return t.data_ptr(), _pack2(st[0], st[1])


def _slots_of(slots, cache, tokens):
    if (slots.dtype is not torch.int64 or slots.dim() != 1 or not slots.is_contiguous() or
            slots.device != cache.device or slots.shape[0] != tokens):
        _refuse("slots must be a contiguous int64 vector on the cache's device, one per token")
    return slots.data_ptr()


def rope_partial_cache_write(cache: KVCache, k, v, slots, cos=None, sin=None, start: int = 0,
                             end: int = 0, mode: str = "interleave", stream=None) -> None:
    """Rotate lanes [start, end) of the keys ``k`` (T, heads, k_dim) by the rows
    of ``cos`` and ``sin`` ((T|1), end - start; None: no rotation) and put them
    and ``v`` (T, heads, v_dim) at ``slots`` (int64; one outside the cache
    skips its token), quantised where the cache holds 8 bits.  k and v stay as
    they are."""
    lib = _lib or load_library()
    dtype = DTYPE_CODE.get(k.dtype)
    if dtype is None or (v is not None and v.dtype != k.dtype):
        _refuse(f"unsupported dtype {k.dtype}, or v of another")
    if mode not in MODE_CODE:
        _mode_code(mode)
    kp, ks = _rows_of(k, cache, cache.k_dim, "k")
    T = k.shape[0]
    vp = vs = cp = sp = None
    if v is not None:
        vp, vs = _rows_of(v, cache, cache.v_dim, "v")
        if v.shape[0] != T:
            _refuse("k and v must hold the same tokens")
    cst = sst = 0
    if cos is not None or sin is not None:
        for t in (cos, sin):
            if (t is None or t.dim() != 2 or t.dtype != k.dtype or t.device != cache.device or
                    t.shape[0] not in (1, T) or t.shape[1] != end - start or
                    (t.shape[1] > 1 and t.stride(1) != 1)):
                _refuse("cos and sin must be (tokens or 1, end - start) of k's dtype with a contiguous last dim")
        cp, sp = cos.data_ptr(), sin.data_ptr()
        cst = cos.stride(0) if cos.shape[0] > 1 else 0
        sst = sin.stride(0) if sin.shape[0] > 1 else 0
    _launch(lib.rope_partial_cache_write,
            (cache._ref, kp, vp, dtype, T, ks, vs, _slots_of(slots, cache, T), cp, sp, cst, sst, start, end,
             MODE_CODE[mode]), stream, cache.device)


def rope_partial_cache_read(cache: KVCache, slots, k=None, v=None, stream=None) -> None:
    """The rows at ``slots`` as numbers, into ``k`` (T, heads, k_dim) and ``v``
    (T, heads, v_dim), either of which may be None; a slot outside the cache
    gives zeros."""
    lib = _lib or load_library()
    kp = ks = vp = vs = None
    T, dtype = slots.shape[0], None
    if k is not None:
        kp, ks = _rows_of(k, cache, cache.k_dim, "k")
        dtype = k.dtype
    if v is not None:
        vp, vs = _rows_of(v, cache, cache.v_dim, "v")
        if dtype is not None and v.dtype != dtype:
            _refuse("k and v must share a dtype")
        dtype = v.dtype
    if dtype is None:
        return
    if dtype not in DTYPE_CODE:
        _refuse(f"unsupported dtype {dtype}")
    if (k is not None and k.shape[0] != T) or (v is not None and v.shape[0] != T):
        _refuse("k and v must have a row for each slot")
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
    if q.dim() != 3 or q.dtype not in DTYPE_CODE:
        _refuse("q must be (tokens, heads, dim) of bf16 or fp16")
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
    tokens of a request) to Tq, and the workspace is made for the call, on its
    stream, when none is given."""
    lib = _lib or load_library()
    dev, kd, vd = cache.device, cache.k_dim, cache.v_dim
    dtype = DTYPE_CODE.get(q.dtype)
    shape = q.shape
    if len(shape) != 3 or shape[2] != kd or dtype is None:
        _refuse(f"q must be (tokens, heads, {kd}) of bf16 or fp16")
    Tq, Hq = shape[0], shape[1]
    if out.dtype != q.dtype or out.shape != (Tq, Hq, vd):
        _refuse(f"out must be ({Tq}, {Hq}, {vd}) of q's dtype")
    qs, os_ = q.stride(), out.stride()
    if (qs[2] != 1 and kd > 1) or (os_[2] != 1 and vd > 1):
        _refuse("the last dim of q and out must be contiguous")
    R = kv_len.shape[0]
    if (q_start.dtype is not torch.int32 or kv_len.dtype is not torch.int32 or kv_len.dim() != 1 or
            q_start.shape != (R + 1,) or not q_start.is_contiguous() or not kv_len.is_contiguous()):
        _refuse("q_start and kv_len must be contiguous int32 vectors of R + 1 and R")
    pt = page_table.shape
    if page_table.dtype is not torch.int32 or len(pt) != 2 or pt[0] != R:
        _refuse("page_table must be int32 (R, pages) with a contiguous last dim")
    pst = page_table.stride()
    if pt[1] > 1 and pst[1] != 1:
        _refuse("page_table must be int32 (R, pages) with a contiguous last dim")
    lp = tp = None
    words = 0
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (Tq, Hq) or not lse.is_contiguous():
            _refuse("lse must be contiguous fp32 (Tq, Hq)")
        lp = lse.data_ptr()
    if tree is not None:
        if tree.dtype is not torch.int64 or tree.dim() != 2 or tree.shape[0] != Tq or not tree.is_contiguous():
            _refuse("tree must be contiguous int64 (Tq, words)")
        tp, words = tree.data_ptr(), tree.shape[1]
    if max_q is None:
        max_q = max(1, Tq)
    if workspace is None and stream is None:
        workspace = tree_attention_workspace(q, cache, max_q)
    elif workspace is None:
        # made on the stream that uses it: memory that another stream's work frees
        # is handed out again before that work has run
        with torch.cuda.stream(_stream_of(stream, dev)):
            workspace = tree_attention_workspace(q, cache, max_q)
    for t in (q, out, q_start, kv_len, page_table, lse, tree, workspace):
        if t is not None and t.device != dev:
            _refuse("every tensor must be on the cache's device")
    if not workspace.is_contiguous():
        _refuse("workspace must be contiguous")
    _launch(lib.rope_partial_tree_attention,
            (cache._ref, q.data_ptr(), dtype, Tq, Hq, _pack2(qs[0], qs[1]), q_start.data_ptr(),
             kv_len.data_ptr(), R, max_q, page_table.data_ptr(), pt[1], pst[0] if R > 1 else pt[1], tp, words,
             out.data_ptr(), _pack2(os_[0], os_[1]), lp, kd ** -0.5 if scale is None else scale,
             workspace.data_ptr(), workspace.nbytes), stream, dev)
