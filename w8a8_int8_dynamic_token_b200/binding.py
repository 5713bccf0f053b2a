"""ctypes binding of libw8a8.so -- argument marshalling only.

Two layers:
  * the C-ABI functions under their C names (``w8a8_linear_fused(...)`` etc.),
    taking raw pointers and sizes exactly as include/w8a8.h declares them;
  * torch-tensor helpers (``quantize_weights``, ``quant_act``, ``linear``,
    ``linear_fused``, ...) that check dtypes/devices/strides, allocate outputs
    with torch, and call the C-ABI on the current CUDA stream.

Every step of the layer runs in the library's CUDA kernels.  There is no CPU
or PyTorch fallback: if libw8a8.so is missing this module raises on first use.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import re
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libw8a8.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "w8a8.h")

W8A8_OK = 0
W8A8_ERR_INVALID_ARG = 1
W8A8_ERR_UNSUPPORTED_SHAPE = 2
W8A8_ERR_MISALIGNED = 3
W8A8_ERR_WORKSPACE = 4
W8A8_ERR_CUDA = 5
W8A8_ERR_DEVICE_TIMEOUT = 6
W8A8_ERR_UNSUPPORTED_DEVICE = 7

VARIANT_AUTO = 0
VARIANT_GEMV = 1
VARIANT_GEMM_BN128 = 2
VARIANT_GEMM_BN256 = 3
VARIANT_GEMM_PAIR = 4
VARIANT_GEMM_BN64 = 5
VARIANT_GEMV_TC = 6
VARIANT_NAMES = {0: "auto", 1: "gemv", 2: "gemm_bn128", 3: "gemm_bn256", 4: "gemm_pair",
                 5: "gemm_bn64", 6: "gemv_tc"}


DTYPE_BF16, DTYPE_FP16, DTYPE_FP32 = 0, 1, 2
ROTARY_INTERLEAVED, ROTARY_HALF = 0, 1
ACT_NONE, ACT_SILU = 0, 1
_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32}
_LAYOUTS = {"interleaved": ROTARY_INTERLEAVED, "half": ROTARY_HALF}
_ACTIVATIONS = {None: ACT_NONE, "silu": ACT_SILU}


class W8A8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class Plan(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("tile_m", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("num_tiles", ctypes.c_int32),
                ("grid", ctypes.c_int32), ("waves_x100", ctypes.c_int32),
                ("split_tiles", ctypes.c_int32), ("split_kblocks_per_pair", ctypes.c_int32),
                ("tail_tiles_nsplit", ctypes.c_int32), ("quant_in_gemm_launch", ctypes.c_int32),
                ("k_split", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f, _ in self._fields_}


class RotaryHeads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("x_batch", ctypes.c_int64), ("x_token", ctypes.c_int64),
                ("x_head", ctypes.c_int64), ("y_batch", ctypes.c_int64),
                ("y_token", ctypes.c_int64), ("y_head", ctypes.c_int64)]


# The arrays of RotaryHeads of a call, packed (as bytes: a third of the time of
# filling the structures).
_ONE_HEADS, _TWO_HEADS = struct.Struct("9q").pack, struct.Struct("18q").pack

_lib = None
_vp, _i64, _i32, _int, _sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int,
                              ctypes.c_size_t)
_f32 = ctypes.c_float

_SIGNATURES = {
    "w8a8_status_string": ([_int], ctypes.c_char_p),
    "w8a8_version": ([], ctypes.c_char_p),
    "w8a8_quantize_weights": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp], _int),
    "w8a8_quant_act": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp], _int),
    "w8a8_unpack_int32_weights": ([_vp, _i64, _i64, _vp, _vp], _int),
    "w8a8_workspace_size": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], _int),
    "w8a8_workspace_size_ex": ([_i64, _i64, _i64, _int, ctypes.POINTER(_sz)], _int),
    "w8a8_linear": ([_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _sz, _vp],
                    _int),
    "w8a8_linear_ex": ([_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _int, _vp,
                        _sz, _vp], _int),
    "w8a8_linear_fused": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp,
                           _vp, _sz, _vp], _int),
    "w8a8_linear_fused_ex": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp,
                              _vp, _sz, _int, _vp], _int),
    "w8a8_linear_fused_host": ([_vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _sz,
                                _vp], _int),
    "w8a8_linear_fused_noalloc": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp],
                                  _int),
    "w8a16_linear": ([_vp, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp], _int),
    "w8a8_input_grad_workspace_size": ([_i64, _i64, _i64, _int, ctypes.POINTER(_sz)], _int),
    "w8a8_linear_input_grad": ([_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _int, _vp, _sz,
                                _vp], _int),
    "w8a8_rotary": ([_vp, _int, _int, _i64, _i64, _i64, _i64, _int, _vp,
                     _int, _i64, _i64, _i64, _vp, _vp, _f32, _int, _vp], _int),
    "w8a8_group_norm_workspace_size": ([_i64, _i64, _i64, _i64, _int, _int, ctypes.POINTER(_sz)],
                                       _int),
    "w8a8_group_norm": ([_vp, _i64, _i64, _int, _i64, _i64, _i64, _i64, _vp, _vp, _int, _f32,
                         _int, _vp, _i64, _i64, _vp, _vp, _vp, _sz, _vp], _int),
    "w8a8_group_norm_quant": ([_vp, _i64, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _int, _f32, _int,
                               _vp, _vp, _vp, _vp, _vp, _sz, _vp], _int),
    "w8a8_group_norm_backward": ([_vp, _i64, _i64, _vp, _i64, _i64, _int, _i64, _i64, _i64, _i64,
                                  _vp, _vp, _vp, _vp, _int, _int, _vp, _i64, _i64, _vp, _vp, _vp,
                                  _sz, _vp], _int),
    "w8a8_select": ([_i64, _i64, _i64, _i32, _int, ctypes.POINTER(Plan)], _int),
    "w8a8_last_device_error": ([_vp], _int),
    "w8a8_selftest_bounded_wait": ([_i64, _vp], _int),
    "w8a8_selftest_quant_exhaustive": ([_vp, _vp], _int),
    "w8a8_debug_peek_tag": ([ctypes.POINTER(ctypes.c_uint64)], _int),
    "w8a8_bench_mma_i8_peak": ([_i64, _i32, _vp], _int),
}


def header_functions() -> list[str]:
    """Names of the functions include/w8a8.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"W8A8_API\s+[^;(]*?\b(w8a(?:8|16)_\w+)\s*\(", text)))


def lib() -> ctypes.CDLL:
    """Load libw8a8.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python -m w8a8_int8_dynamic_token_b200.build`"
                " (there is no fallback implementation)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().w8a8_status_string(int(status)).decode()


def version() -> str:
    return lib().w8a8_version().decode()


def _check(status: int, where: str) -> None:
    if status != W8A8_OK:
        raise W8A8Error(status, where)


# ------------------------------------------------------------------ raw C ABI

def w8a8_quantize_weights(W, N, K, ldw, Wq, s_w, stream) -> int:
    return lib().w8a8_quantize_weights(W, N, K, ldw, Wq, s_w, stream)


def w8a8_unpack_int32_weights(packed, N, K, Wq, stream) -> int:
    return lib().w8a8_unpack_int32_weights(packed, N, K, Wq, stream)


def w8a8_quant_act(x, M, K, ldx, q, s_a, stream) -> int:
    return lib().w8a8_quant_act(x, M, K, ldx, q, s_a, stream)


def w8a8_workspace_size(M, N, K) -> tuple[int, int]:
    out = ctypes.c_size_t(0)
    st = lib().w8a8_workspace_size(M, N, K, ctypes.byref(out))
    return st, int(out.value)


def w8a8_workspace_size_ex(M, N, K, variant) -> tuple[int, int]:
    out = ctypes.c_size_t(0)
    st = lib().w8a8_workspace_size_ex(M, N, K, variant, ctypes.byref(out))
    return st, int(out.value)


def w8a8_linear(q, s_a, M, K, Wq, s_w, bias, N, y, ldy, acc_debug, workspace, ws_bytes,
                stream) -> int:
    return lib().w8a8_linear(q, s_a, M, K, Wq, s_w, bias, N, y, ldy, acc_debug, workspace,
                             ws_bytes, stream)


def w8a8_linear_ex(q, s_a, M, K, Wq, s_w, bias, N, y, ldy, acc_debug, variant, workspace,
                   ws_bytes, stream) -> int:
    return lib().w8a8_linear_ex(q, s_a, M, K, Wq, s_w, bias, N, y, ldy, acc_debug, variant,
                                workspace, ws_bytes, stream)


def w8a8_linear_fused(x, M, K, ldx, Wq, s_w, bias, N, y, ldy, q_out, s_a_out, workspace,
                      ws_bytes, stream) -> int:
    return lib().w8a8_linear_fused(x, M, K, ldx, Wq, s_w, bias, N, y, ldy, q_out, s_a_out,
                                   workspace, ws_bytes, stream)


def w8a8_linear_fused_ex(x, M, K, ldx, Wq, s_w, bias, N, y, ldy, q_out, s_a_out, workspace,
                         ws_bytes, options, stream) -> int:
    return lib().w8a8_linear_fused_ex(x, M, K, ldx, Wq, s_w, bias, N, y, ldy, q_out, s_a_out,
                                      workspace, ws_bytes, options, stream)


FUSED_ONE_LAUNCH = 1


def w8a8_linear_fused_host(x_host, M, K, Wq, s_w, bias, N, y_host, x_dev, y_dev, workspace,
                           ws_bytes, stream) -> int:
    return lib().w8a8_linear_fused_host(x_host, M, K, Wq, s_w, bias, N, y_host, x_dev, y_dev,
                                        workspace, ws_bytes, stream)


def w8a8_linear_fused_noalloc(x, M, K, ldx, Wq, s_w, bias, N, y, ldy, stream) -> int:
    return lib().w8a8_linear_fused_noalloc(x, M, K, ldx, Wq, s_w, bias, N, y, ldy, stream)


def w8a16_linear_raw(x, M, K, ldx, Wq, s_w, bias, N, y, ldy, stream) -> int:
    return lib().w8a16_linear(x, M, K, ldx, Wq, s_w, bias, N, y, ldy, stream)


def w8a8_input_grad_workspace_size(M, N, K, variant) -> tuple[int, int]:
    out = ctypes.c_size_t(0)
    st = lib().w8a8_input_grad_workspace_size(M, N, K, variant, ctypes.byref(out))
    return st, int(out.value)


def w8a8_linear_input_grad(dy, M, N, lddy, Wq, s_w, K, dx, lddx, variant, workspace, ws_bytes,
                           stream) -> int:
    return lib().w8a8_linear_input_grad(dy, M, N, lddy, Wq, s_w, K, dx, lddx, variant, workspace,
                                        ws_bytes, stream)


def w8a8_rotary(tensors, num_tensors, dtype, batch, tokens, dim, rot, layout, positions,
                position_bits, pos_batch, pos_token, axes, inv_freq, axis, scale, backward,
                stream) -> int:
    return lib().w8a8_rotary(tensors, num_tensors, dtype, batch, tokens, dim, rot, layout,
                             positions, position_bits, pos_batch, pos_token, axes, inv_freq, axis,
                             scale, backward, stream)


def w8a8_group_norm_workspace_size(B, S, C, G, dtype, backward) -> tuple[int, int]:
    out = ctypes.c_size_t(0)
    st = lib().w8a8_group_norm_workspace_size(B, S, C, G, dtype, backward, ctypes.byref(out))
    return st, int(out.value)


def w8a8_group_norm(x, x_batch, x_pixel, dtype, B, S, C, G, weight, bias, param_dtype, eps,
                    activation, y, y_batch, y_pixel, mean, rstd, workspace, ws_bytes,
                    stream) -> int:
    return lib().w8a8_group_norm(x, x_batch, x_pixel, dtype, B, S, C, G, weight, bias, param_dtype,
                                 eps, activation, y, y_batch, y_pixel, mean, rstd, workspace,
                                 ws_bytes, stream)


def w8a8_group_norm_quant(x, x_batch, x_pixel, B, S, C, G, weight, bias, param_dtype, eps,
                          activation, q, s_a, mean, rstd, workspace, ws_bytes, stream) -> int:
    return lib().w8a8_group_norm_quant(x, x_batch, x_pixel, B, S, C, G, weight, bias, param_dtype,
                                       eps, activation, q, s_a, mean, rstd, workspace, ws_bytes,
                                       stream)


def w8a8_group_norm_backward(dy, dy_batch, dy_pixel, x, x_batch, x_pixel, dtype, B, S, C, G, mean,
                             rstd, weight, bias, param_dtype, activation, dx, dx_batch, dx_pixel,
                             dweight, dbias, workspace, ws_bytes, stream) -> int:
    return lib().w8a8_group_norm_backward(dy, dy_batch, dy_pixel, x, x_batch, x_pixel, dtype, B, S,
                                          C, G, mean, rstd, weight, bias, param_dtype, activation,
                                          dx, dx_batch, dx_pixel, dweight, dbias, workspace,
                                          ws_bytes, stream)


def w8a8_select(M, N, K, num_sms=148, variant=VARIANT_AUTO) -> tuple[int, Plan]:
    plan = Plan()
    st = lib().w8a8_select(M, N, K, num_sms, variant, ctypes.byref(plan))
    return st, plan


def w8a8_last_device_error(stream) -> int:
    return lib().w8a8_last_device_error(stream)


def w8a8_selftest_bounded_wait(limit_ns, stream) -> int:
    return lib().w8a8_selftest_bounded_wait(limit_ns, stream)


# ------------------------------------------------------------------ torch helpers

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if isinstance(stream, int):  # a raw handle (see _OnCurrent)
        return ctypes.c_void_p(stream)
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype, ndim):
    """dtype, rank and unit inner stride (checked before the device, so shape
    errors surface the same way on any device)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D")
    if t.numel() > 0 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")


def _shape(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _on_one_device(**tensors):
    """The CUDA device every given tensor lives on (all must share it)."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
    return dev


class _OnCurrent:
    """The common case of _launching: the tensors' device is already current
    and no stream is given, so nothing needs switching; yields that device's
    current stream as a raw handle."""
    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


def _launching(dev, stream=None):
    """Run a call on the tensors' device: the library reads the current device
    (its properties, and the allocation-free scratch), so that device is made
    current.  The call is enqueued on `stream`, or on that device's current
    stream; tensors allocated inside belong to that stream, so the caching
    allocator never hands their memory to other work while the call may still
    use it.  When the device is current already and no stream is given,
    nothing is switched (a few microseconds of host time per call less)."""
    if stream is None and dev.index == torch.cuda.current_device():
        return _OnCurrent(torch._C._cuda_getCurrentRawStream(dev.index))
    return _switching(dev, stream)


@contextlib.contextmanager
def _switching(dev, stream):
    with torch.cuda.device(dev):
        if stream is None:
            yield torch.cuda.current_stream()
        else:
            if stream.device != dev:
                raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
            with torch.cuda.stream(stream):
                yield stream


@functools.lru_cache(maxsize=1024)
def workspace_size(M: int, N: int, K: int, variant: int = VARIANT_AUTO) -> int:
    st, n = w8a8_workspace_size_ex(M, N, K, variant)
    _check(st, "w8a8_workspace_size_ex")
    return n


def select(M: int, N: int, K: int, num_sms: int = 148, variant: int = VARIANT_AUTO) -> dict:
    st, plan = w8a8_select(M, N, K, num_sms, variant)
    _check(st, "w8a8_select")
    d = plan.as_dict()
    d["variant_name"] = VARIANT_NAMES[d["variant"]]
    return d


def quantize_weights(W: torch.Tensor, stream=None):
    """bf16 W [N, K] -> (Wq int8 [N, K], s_w fp32 [N]) on W's device."""
    _need(W, "W", torch.bfloat16, 2)
    dev = _on_one_device(W=W)
    N, K = W.shape
    with _launching(dev, stream) as s:
        Wq = torch.empty((N, K), dtype=torch.int8, device=dev)
        s_w = torch.empty((N,), dtype=torch.float32, device=dev)
        _check(w8a8_quantize_weights(_ptr(W), N, K, W.stride(0), _ptr(Wq), _ptr(s_w), _stream(s)),
               "w8a8_quantize_weights")
    return Wq, s_w


def unpack_int32_weights(packed: torch.Tensor, stream=None) -> torch.Tensor:
    """Packed int32 [N, K/4] weight storage (codes + 128, four per word, first
    code in the low byte) -> Wq int8 [N, K] on packed's device."""
    _need(packed, "packed", torch.int32, 2)
    if not packed.is_contiguous():
        raise ValueError("packed must be dense row-major")
    dev = _on_one_device(packed=packed)
    N, K = packed.shape[0], packed.shape[1] * 4
    with _launching(dev, stream) as s:
        Wq = torch.empty((N, K), dtype=torch.int8, device=dev)
        _check(w8a8_unpack_int32_weights(_ptr(packed), N, K, _ptr(Wq), _stream(s)),
               "w8a8_unpack_int32_weights")
    return Wq


def quant_act(x: torch.Tensor, stream=None):
    """bf16 x [M, K] -> (q int8 [M, K], s_a fp32 [M])."""
    _need(x, "x", torch.bfloat16, 2)
    dev = _on_one_device(x=x)
    M, K = x.shape
    with _launching(dev, stream) as s:
        q = torch.empty((M, K), dtype=torch.int8, device=dev)
        s_a = torch.empty((M,), dtype=torch.float32, device=dev)
        _check(w8a8_quant_act(_ptr(x), M, K, x.stride(0), _ptr(q), _ptr(s_a), _stream(s)),
               "w8a8_quant_act")
    return q, s_a


def _workspace_for(M, N, K, workspace, dev, variant=VARIANT_AUTO):
    """(tensor, pointer, bytes): the caller's workspace, or a fresh one of
    workspace_size(M, N, K, variant) bytes when `workspace` is None (allocated
    on the launching stream, inside _launching).  The caller keeps the returned
    tensor alive until the launch has been enqueued: the device memory must
    not return to the allocator before then, or an output allocated
    afterwards could share it."""
    need = workspace_size(M, N, K, variant)
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    return workspace, _ptr(workspace), workspace.numel() * workspace.element_size()


def _check_layer_args(M, N, K, bias, out):
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, 1)
        _shape(bias, "bias", (N,))
    if out is not None:
        _need(out, "out", torch.bfloat16, 2)
        _shape(out, "out", (M, N))


def linear(q, s_a, Wq, s_w, bias=None, out=None, acc_debug=False, variant=VARIANT_AUTO,
           workspace=None, split=True, stream=None):
    """y = bf16(((float)(q @ Wq^T) * s_a) * s_w + bias); with acc_debug=True the raw
    int32 accumulators [M, N] are returned instead.  split=False runs the pair
    kernel without its K-split tail (no workspace is passed)."""
    _need(q, "q", torch.int8, 2)
    _need(s_a, "s_a", torch.float32, 1)
    _need(Wq, "Wq", torch.int8, 2)
    _need(s_w, "s_w", torch.float32, 1)
    M, K = q.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or s_a.shape[0] != M or s_w.shape[0] != N:
        raise ValueError("shape mismatch between q, s_a, Wq, s_w")
    if not (q.is_contiguous() and Wq.is_contiguous()):
        raise ValueError("q and Wq must be dense row-major")
    _check_layer_args(M, N, K, bias, None if acc_debug else out)
    dev = _on_one_device(q=q, s_a=s_a, Wq=Wq, s_w=s_w, bias=bias,
                         out=None if acc_debug else out, workspace=workspace)
    with _launching(dev, stream) as s:
        ws, ws_ptr, ws_bytes = (_workspace_for(M, N, K, workspace, dev, variant) if split
                                else (None, None, 0))
        if acc_debug:
            acc = torch.empty((M, N), dtype=torch.int32, device=dev)
            _check(w8a8_linear_ex(_ptr(q), _ptr(s_a), M, K, _ptr(Wq), _ptr(s_w), _ptr(bias), N,
                                  None, N, _ptr(acc), variant, ws_ptr, ws_bytes, _stream(s)),
                   "w8a8_linear_ex")
            del ws  # enqueued on s: later allocations on s are ordered after the launch
            return acc
        y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        _check(w8a8_linear_ex(_ptr(q), _ptr(s_a), M, K, _ptr(Wq), _ptr(s_w), _ptr(bias), N,
                              _ptr(y), y.stride(0), None, variant, ws_ptr, ws_bytes, _stream(s)),
               "w8a8_linear_ex")
        del ws
    return y


def linear_fused(x, Wq, s_w, bias=None, out=None, workspace=None, return_intermediates=False,
                 stream=None):
    """Whole layer from bf16 x [M, K]: per-token quantization, int8 GEMM, fused
    epilogue.  Returns y [M, N] (and (q, s_a) with return_intermediates=True)."""
    _need(x, "x", torch.bfloat16, 2)
    _need(Wq, "Wq", torch.int8, 2)
    _need(s_w, "s_w", torch.float32, 1)
    M, K = x.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or s_w.shape[0] != N or not Wq.is_contiguous():
        raise ValueError("shape mismatch between x, Wq, s_w")
    _check_layer_args(M, N, K, bias, out)
    dev = _on_one_device(x=x, Wq=Wq, s_w=s_w, bias=bias, out=out, workspace=workspace)
    with _launching(dev, stream) as s:
        y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        q = s_a = None
        if return_intermediates:
            q = torch.empty((M, K), dtype=torch.int8, device=dev)
            s_a = torch.empty((M,), dtype=torch.float32, device=dev)
        ws, ws_ptr, ws_bytes = _workspace_for(M, N, K, workspace, dev)
        _check(w8a8_linear_fused(_ptr(x), M, K, x.stride(0), _ptr(Wq), _ptr(s_w), _ptr(bias), N,
                                 _ptr(y), y.stride(0), _ptr(q), _ptr(s_a), ws_ptr, ws_bytes,
                                 _stream(s)), "w8a8_linear_fused")
        del ws
    if return_intermediates:
        return y, q, s_a
    return y


def w8a16_linear(x, Wq, s_w, bias=None, out=None, stream=None):
    """Weight-only int8 layer on bf16 x [M, K]: y = bf16((x @ Wq^T) * s_w + bias),
    fp32 accumulation on the tensor cores."""
    _need(x, "x", torch.bfloat16, 2)
    _need(Wq, "Wq", torch.int8, 2)
    _need(s_w, "s_w", torch.float32, 1)
    M, K = x.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or s_w.shape[0] != N or not Wq.is_contiguous():
        raise ValueError("shape mismatch between x, Wq, s_w")
    _check_layer_args(M, N, K, bias, out)
    dev = _on_one_device(x=x, Wq=Wq, s_w=s_w, bias=bias, out=out)
    with _launching(dev, stream) as s:
        y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        _check(w8a16_linear_raw(_ptr(x), M, K, x.stride(0), _ptr(Wq), _ptr(s_w), _ptr(bias), N,
                                _ptr(y), y.stride(0), _stream(s)), "w8a16_linear")
    return y


def linear_fused_host(x_host, Wq, s_w, bias, y_host, x_dev, y_dev, workspace, stream=None):
    """End-to-end call on host buffers: copy x in, run the layer, copy y out
    (all enqueued on the stream; synchronize before reading y_host)."""
    M, K = x_host.shape
    N = Wq.shape[0]
    if tuple(y_host.shape) != (M, N) or tuple(x_dev.shape) != (M, K) or tuple(y_dev.shape) != (M, N):
        raise ValueError("x_host / x_dev must be [M, K] and y_host / y_dev [M, N]")
    dev = _on_one_device(Wq=Wq, s_w=s_w, bias=bias, x_dev=x_dev, y_dev=y_dev, workspace=workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _launching(dev, stream) as s:
        _check(w8a8_linear_fused_host(_ptr(x_host), M, K, _ptr(Wq), _ptr(s_w), _ptr(bias), N,
                                      _ptr(y_host), _ptr(x_dev), _ptr(y_dev), _ptr(workspace),
                                      ws_bytes, _stream(s)), "w8a8_linear_fused_host")
    return y_host


@functools.lru_cache(maxsize=1024)
def input_grad_workspace_size(M: int, N: int, K: int, variant: int = VARIANT_AUTO) -> int:
    st, n = w8a8_input_grad_workspace_size(M, N, K, variant)
    _check(st, "w8a8_input_grad_workspace_size")
    return n


def _launch_handle(x, others, stream):
    """The raw handle of the stream a call on x's device goes to, or None where
    the device or the stream has to be switched first (see _launching).  Every
    tensor of `others` (None allowed) must be on x's device."""
    index = x.get_device()
    if index < 0:
        raise ValueError("the tensors must be CUDA tensors")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"a tensor is on {t.device}, expected cuda:{index} (all must be CUDA "
                             "tensors on one device)")
    if stream is None and index == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(index)
    return None


def _scratch(need, workspace, x):
    """(tensor, pointer, bytes) of the caller's workspace, or of a fresh one of
    `need` bytes on x's device (allocated on the launching stream; kept alive by
    the caller until the launches have been enqueued)."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        return workspace, workspace.data_ptr(), need
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _address(t):
    return None if t is None else t.data_ptr()


def linear_input_grad(dy, Wq, s_w, out=None, workspace=None, variant=VARIANT_AUTO, stream=None):
    """Gradient of the layer with respect to its input, through the frozen int8
    weights: dx [M, K] from dy bf16 [M, N].  The rows dy * s_w are quantized per
    token and multiplied with Wq as it is stored (exact int32 sums)."""
    _need(dy, "dy", torch.bfloat16, 2)
    _need(Wq, "Wq", torch.int8, 2)
    _need(s_w, "s_w", torch.float32, 1)
    M, N = dy.shape
    K = Wq.shape[1]
    if Wq.shape[0] != N or s_w.shape[0] != N or not Wq.is_contiguous():
        raise ValueError("shape mismatch between dy, Wq, s_w")
    if out is not None:
        _need(out, "out", torch.bfloat16, 2)
        _shape(out, "out", (M, K))
    need = input_grad_workspace_size(M, N, K, variant)
    handle = _launch_handle(dy, (Wq, s_w, out, workspace), stream)
    if handle is None:
        with _switching(dy.device, stream):
            return linear_input_grad(dy, Wq, s_w, out, workspace, variant)
    dx = out if out is not None else torch.empty_strided((M, K), (K, 1), dtype=torch.bfloat16,
                                                         device=dy.device)
    ws, ws_ptr, ws_bytes = _scratch(need, workspace, dy)
    st = lib().w8a8_linear_input_grad(dy.data_ptr(), M, N, dy.stride(0), Wq.data_ptr(),
                                      s_w.data_ptr(), K, dx.data_ptr(), dx.stride(0), variant,
                                      ws_ptr, ws_bytes, handle)
    del ws  # enqueued: later allocations on the stream are ordered after the launches
    if st != W8A8_OK:
        raise W8A8Error(st, "w8a8_linear_input_grad")
    return dx


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None,
                       factor: float = 1.0, trained: int = 0, fast: float = 32.0,
                       slow: float = 1.0):
    """(inv_freq, scale) for rotary(): radians per position of the rot / 2 pairs
    (CPU float64), f_i = base^(-2i / rot), and the factor on rotated values.

    scaling, for contexts `factor` times the trained one:
      None       as they are;
      "linear"   every frequency divided by factor;
      "base"     base raised to base * factor^(rot / (rot - 2)), which divides
                 the slowest frequency by factor and keeps the fastest;
      "ramp"     pairs that turn more than `fast` times over the `trained`
                 positions are kept, those that turn less than `slow` times are
                 divided by factor, a linear ramp over the pair index between,
                 from the whole index below the one to the whole index above
                 the other.  These ends lie within [0, rot - 1], so the upper
                 one may be past the last pair, which then is only partly
                 divided.  scale = 0.1 ln(factor) + 1.
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be above 1 and factor at least 1")
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "base":
        if rot == 2:
            raise ValueError("scaling 'base' needs rot of at least 4")
        base = base * factor ** (rot / (rot - 2))
    freq = torch.pow(torch.tensor(base, dtype=torch.float64), -2.0 * i / rot)
    if scaling in (None, "base"):
        return freq, 1.0
    if scaling == "linear":
        return freq / factor, 1.0
    if scaling != "ramp":
        raise ValueError(f"unknown scaling {scaling!r}")
    if trained < 1 or not fast > slow > 0.0:
        raise ValueError("scaling 'ramp' needs trained >= 1 and fast > slow > 0")
    # the pair that turns t times over the trained positions
    low, high = (rot * math.log(trained / (t * 2.0 * math.pi)) / (2.0 * math.log(base))
                 for t in (fast, slow))
    low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
    if high <= 0:  # no pair turns `slow` times
        ramp = torch.ones_like(i)
    else:
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return freq * (1.0 - ramp) + freq / factor * ramp, 0.1 * math.log(factor) + 1.0


def _heads(t, name, dtype):
    """[tokens, heads, dim] or [batch, tokens, heads, dim]."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'bfloat16, float16 or float32'}, got {t.dtype}")


@functools.lru_cache(maxsize=4096)
def _head_strides(shape, strides, name):
    """(batch, tokens, heads, dim) and the strides of the first three."""
    if len(shape) not in (3, 4):
        raise ValueError(f"{name} must be [tokens, heads, dim] or [batch, tokens, heads, dim]")
    if shape[-1] > 1 and strides[-1] != 1 and 0 not in shape:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    four = len(shape) == 4
    return (shape[0] if four else 1, *shape[-3:]), (strides[0] if four else 0, *strides[-3:-1])


def _position_strides(shape, strides, batch, tokens, with_axes):
    """(batch stride, token stride, axes) of positions."""
    lead = len(shape) - with_axes
    if lead not in (1, 2) or shape[lead - 1] != tokens or (lead == 2 and shape[0] != batch):
        raise ValueError(f"positions must be [{tokens}] or [{batch}, {tokens}]"
                         + (" and a last dimension of axes" if with_axes else ""))
    axes = shape[-1] if with_axes else 1
    if axes > 1 and strides[-1] != 1:
        raise ValueError("positions must have unit stride in its last dimension")
    return strides[0] if lead == 2 else 0, strides[lead - 1], axes


@functools.lru_cache(maxsize=4096)
def _rotary_geometry(x_shape, x_strides, k_shape, k_strides, pos_shape, pos_strides, pairs, layout,
                     with_axes):
    """What a call's shapes and strides say, checked once: ((heads, strides) of
    x, of k or None, sizes and codes up to the layout, strides of positions)."""
    (batch, tokens, heads, dim), xs = _head_strides(x_shape, x_strides, "x")
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
    if 2 * pairs > dim:
        raise ValueError(f"inv_freq turns {2 * pairs} values of a head, which has {dim}")
    k = None
    if k_shape is not None:
        (k_batch, k_tokens, k_heads, k_dim), ks = _head_strides(k_shape, k_strides, "k")
        if len(k_shape) != len(x_shape) or (k_batch, k_tokens, k_dim) != (batch, tokens, dim):
            raise ValueError("x and k differ in more than their heads")
        k = (k_heads, *ks)
    return ((heads, *xs), k, (batch, tokens, dim, 2 * pairs, _LAYOUTS[layout]),
            _position_strides(pos_shape, pos_strides, batch, tokens, with_axes))


def _rotary_out(x, heads, out):
    """out, or a new tensor laid out as x, and its strides."""
    if out is None:
        out = torch.empty_like(x)
        if x.is_contiguous():
            return out, heads[1:]
    return out, _head_strides(out.shape, out.stride(), "out")[1]


def rotary(x, positions, inv_freq, k=None, layout="interleaved", axis=None, scale=1.0,
           backward=False, out=None, out_k=None, stream=None):
    """Rotary positions on heads x [tokens, heads, dim] or [batch, tokens, heads,
    dim] (and, in the same launch, on k with its own number of heads); bf16,
    fp16 or fp32, any strides outside a head.  inv_freq: CPU float64 [rot / 2]
    radians per position, at least 0 and below 2^64 (see rotary_frequencies);
    the first rot values of a head turn, the others are copied.  positions:
    int32 or int64 on x's device, [tokens] or [batch, tokens], or with a last
    dimension of axes when `axis` (CPU int32 [rot / 2], the axis of each pair) is
    given.  backward=True: the gradient.  out / out_k: where to write; x / k
    themselves, or memory that does not overlap them, each head a place of its
    own.  Returns y, or (y, y_k) with k, laid out as x and k where those are
    dense."""
    _heads(x, "x", None)
    dtype = x.dtype
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype != torch.float64 or \
            inv_freq.is_cuda or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a dense 1-D CPU float64 tensor")
    if k is not None:
        _heads(k, "k", dtype)
    if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64):
        raise TypeError("positions must be an int32 or int64 tensor")
    if axis is not None and (
            not isinstance(axis, torch.Tensor) or axis.dtype != torch.int32 or axis.is_cuda or
            axis.shape != inv_freq.shape or not axis.is_contiguous()):
        raise TypeError("axis must be a dense CPU int32 tensor of inv_freq's shape")
    geometry = _rotary_geometry(
        x.shape, x.stride(), None if k is None else k.shape, None if k is None else k.stride(),
        positions.shape, positions.stride(), inv_freq.shape[0], layout, axis is not None)
    if out is not None:
        _heads(out, "out", dtype)
        _shape(out, "out", x.shape)
    if out_k is not None:
        if k is None:
            raise ValueError("out_k is given without k")
        _heads(out_k, "out_k", dtype)
        _shape(out_k, "out_k", k.shape)
    handle = _launch_handle(x, (k, positions, out, out_k), stream)
    if handle is None:
        with _switching(x.device, stream):
            return rotary(x, positions, inv_freq, k, layout, axis, scale, backward, out, out_k)
    x_heads, k_heads, sizes, pos = geometry
    y, ys = _rotary_out(x, x_heads, out)
    y_k = None
    if k is None:
        tensors = _ONE_HEADS(x.data_ptr(), y.data_ptr(), *x_heads, *ys)
    else:
        y_k, ks = _rotary_out(k, k_heads, out_k)
        tensors = _TWO_HEADS(x.data_ptr(), y.data_ptr(), *x_heads, *ys, k.data_ptr(),
                             y_k.data_ptr(), *k_heads, *ks)
    st = lib().w8a8_rotary(tensors, 1 if k is None else 2, _DTYPES[dtype], *sizes,
                           positions.data_ptr(), 64 if positions.dtype == torch.int64 else 32, *pos,
                           inv_freq.data_ptr(), _address(axis), scale, 1 if backward else 0, handle)
    if st != W8A8_OK:
        raise W8A8Error(st, "w8a8_rotary")
    return y if k is None else (y, y_k)


@functools.lru_cache(maxsize=1024)
def group_norm_workspace_size(B: int, S: int, C: int, groups: int, dtype=torch.bfloat16,
                              backward: bool = False) -> int:
    st, n = w8a8_group_norm_workspace_size(B, S, C, groups, _DTYPES[dtype], int(backward))
    _check(st, "w8a8_group_norm_workspace_size")
    return n


def _channels_last(t, name, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'bfloat16, float16 or float32'}, got {t.dtype}")
    return t.dtype


@functools.lru_cache(maxsize=4096)
def _pixels(sizes, strides, name):
    """Channels-last [B, ..., C]: (B, pixels, C, sample stride, pixel stride).
    The dimensions between must be evenly strided, as one run of pixels."""
    if len(sizes) < 3:
        raise ValueError(f"{name} must be [B, ..., C] with its channels last")
    if sizes[-1] > 1 and strides[-1] != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    pixels, step = 1, sizes[-1]
    for n, st in zip(reversed(sizes[1:-1]), reversed(strides[1:-1])):
        if n == 1:
            continue
        if pixels == 1:
            step = st
        elif st != step * pixels:
            raise ValueError(f"{name}'s pixels must be evenly strided")
        pixels *= n
    return sizes[0], pixels, sizes[-1], strides[0], step


@functools.lru_cache(maxsize=4096)
def _norm_geometry(sizes, strides, groups, dtype, backward):
    """_pixels of x and the bytes of workspace that a call takes."""
    B, S, C, xb, xs = _pixels(sizes, strides, "x")
    return B, S, C, xb, xs, group_norm_workspace_size(B, S, C, groups, dtype, backward)


def _norm_params(dtype, C, weight, bias):
    """The type code of weight and bias ([C], both in x's type or in fp32)."""
    wt = dtype if weight is None else _norm_param(dtype, C, "weight", weight)
    bt = wt if bias is None else _norm_param(dtype, C, "bias", bias)
    if weight is not None and bt is not wt:
        raise TypeError("weight and bias must have the same type")
    return _DTYPES[bt]


def _norm_param(dtype, C, name, t):
    if not isinstance(t, torch.Tensor) or (t.dtype != dtype and t.dtype != torch.float32):
        raise TypeError(f"{name} must be a {dtype} or float32 tensor")
    if t.shape != (C,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a dense [{C}] tensor")
    return t.dtype


def _activation(activation):
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    return _ACTIVATIONS[activation]


def _norm_out(x, out, S, C):
    """out, or a dense new tensor like x, and its strides of a sample and a pixel."""
    if out is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format), S * C, C
    return (out, *_pixels(out.shape, out.stride(), "out")[3:])


def _norm_stats(wanted, B, groups, x):
    if not wanted:
        return None, None
    mean = torch.empty_strided((B, groups), (groups, 1), dtype=torch.float32, device=x.device)
    return mean, torch.empty_like(mean)


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, activation=None, out=None,
               return_stats=False, workspace=None, stream=None):
    """Group normalization of a channels-last x [B, ..., C] (bf16, fp16, fp32)
    with an optional SiLU: y in x's type and shape (and, with return_stats, the
    mean and 1 / standard deviation, fp32 [B, groups], that the backward pass
    takes).  out may be x itself."""
    dtype = _channels_last(x, "x")
    B, S, C, xb, xs, need = _norm_geometry(x.shape, x.stride(), groups, dtype, False)
    act = _activation(activation)
    pdt = _norm_params(dtype, C, weight, bias)
    if out is not None:
        _channels_last(out, "out", dtype)
        _shape(out, "out", x.shape)
    handle = _launch_handle(x, (weight, bias, out, workspace), stream)
    if handle is None:
        with _switching(x.device, stream):
            return group_norm(x, groups, weight, bias, eps, activation, out, return_stats, workspace)
    y, yb, ys = _norm_out(x, out, S, C)
    mean, rstd = _norm_stats(return_stats, B, groups, x)
    ws, ws_ptr, ws_bytes = _scratch(need, workspace, x)
    st = lib().w8a8_group_norm(x.data_ptr(), xb, xs, _DTYPES[dtype], B, S, C, groups,
                               _address(weight), _address(bias), pdt, eps, act, y.data_ptr(), yb,
                               ys, _address(mean), _address(rstd), ws_ptr, ws_bytes, handle)
    del ws  # enqueued: later allocations on the stream are ordered after the launch
    if st != W8A8_OK:
        raise W8A8Error(st, "w8a8_group_norm")
    return (y, mean, rstd) if return_stats else y


def group_norm_quant(x, groups, weight=None, bias=None, eps=1e-5, activation=None,
                     return_stats=False, workspace=None, stream=None):
    """group_norm of a bf16 x as the operand of linear(): (q int8 [B * pixels,
    C], s_a fp32 [B * pixels]), the rows of the fp32 result quantized per pixel
    (and the statistics, with return_stats)."""
    dtype = _channels_last(x, "x", torch.bfloat16)
    B, S, C, xb, xs, need = _norm_geometry(x.shape, x.stride(), groups, dtype, False)
    act = _activation(activation)
    pdt = _norm_params(dtype, C, weight, bias)
    handle = _launch_handle(x, (weight, bias, workspace), stream)
    if handle is None:
        with _switching(x.device, stream):
            return group_norm_quant(x, groups, weight, bias, eps, activation, return_stats,
                                    workspace)
    q = torch.empty_strided((B * S, C), (C, 1), dtype=torch.int8, device=x.device)
    s_a = torch.empty(B * S, dtype=torch.float32, device=x.device)
    mean, rstd = _norm_stats(return_stats, B, groups, x)
    ws, ws_ptr, ws_bytes = _scratch(need, workspace, x)
    st = lib().w8a8_group_norm_quant(x.data_ptr(), xb, xs, B, S, C, groups, _address(weight),
                                     _address(bias), pdt, eps, act, q.data_ptr(), s_a.data_ptr(),
                                     _address(mean), _address(rstd), ws_ptr, ws_bytes, handle)
    del ws
    if st != W8A8_OK:
        raise W8A8Error(st, "w8a8_group_norm_quant")
    return (q, s_a, mean, rstd) if return_stats else (q, s_a)


def group_norm_backward(dy, x, mean, rstd, weight=None, bias=None, activation=None, out=None,
                        workspace=None, stream=None):
    """Gradients of group_norm (or, straight through the rounding, of
    group_norm_quant): (dx in x's type, dweight, dbias fp32 [C], None where
    there is no such parameter).  mean, rstd: the forward's statistics; out may
    be dy or x itself."""
    dtype = _channels_last(x, "x")
    _channels_last(dy, "dy", dtype)
    _shape(dy, "dy", x.shape)
    act = _activation(activation)
    _need(mean, "mean", torch.float32, 2)
    _need(rstd, "rstd", torch.float32, 2)
    groups = mean.shape[1]
    B, S, C, xb, xs, need = _norm_geometry(x.shape, x.stride(), groups, dtype, True)
    pdt = _norm_params(dtype, C, weight, bias)
    if mean.shape[0] != B:
        raise ValueError(f"mean must have shape ({B}, groups), got {tuple(mean.shape)}")
    _shape(rstd, "rstd", mean.shape)
    if not (mean.is_contiguous() and rstd.is_contiguous()):
        raise ValueError("mean and rstd must be dense")
    if out is not None:
        _channels_last(out, "out", dtype)
        _shape(out, "out", x.shape)
    handle = _launch_handle(x, (dy, mean, rstd, weight, bias, out, workspace), stream)
    if handle is None:
        with _switching(x.device, stream):
            return group_norm_backward(dy, x, mean, rstd, weight, bias, activation, out, workspace)
    _, _, _, gb, gs = _pixels(dy.shape, dy.stride(), "dy")
    dx, ob, os_ = _norm_out(x, out, S, C)
    dweight = dbias = None
    if weight is not None:
        dweight = torch.empty(C, dtype=torch.float32, device=x.device)
    if bias is not None:
        dbias = torch.empty(C, dtype=torch.float32, device=x.device)
    ws, ws_ptr, ws_bytes = _scratch(need, workspace, x)
    st = lib().w8a8_group_norm_backward(
        dy.data_ptr(), gb, gs, x.data_ptr(), xb, xs, _DTYPES[dtype], B, S, C, groups,
        mean.data_ptr(), rstd.data_ptr(), _address(weight), _address(bias), pdt, act, dx.data_ptr(),
        ob, os_, _address(dweight), _address(dbias), ws_ptr, ws_bytes, handle)
    del ws
    if st != W8A8_OK:
        raise W8A8Error(st, "w8a8_group_norm_backward")
    return dx, dweight, dbias


def last_device_error(stream=None) -> int:
    return w8a8_last_device_error(_stream(stream))


def selftest_bounded_wait(limit_ns: int, stream=None) -> int:
    return w8a8_selftest_bounded_wait(int(limit_ns), _stream(stream))


def w8a8_selftest_quant_exhaustive(counts_dev, stream) -> int:
    return lib().w8a8_selftest_quant_exhaustive(counts_dev, stream)


def selftest_quant_exhaustive(stream=None) -> tuple[int, int]:
    """(pairs checked, pairs whose code differs from the IEEE-division path)."""
    counts = torch.zeros(2, dtype=torch.int64, device="cuda")
    _check(w8a8_selftest_quant_exhaustive(_ptr(counts), _stream(stream)),
           "w8a8_selftest_quant_exhaustive")
    torch.cuda.current_stream().synchronize() if stream is None else stream.synchronize()
    c = counts.cpu().tolist()
    return int(c[0]), int(c[1])


PEAK_OPS_PER_PAIR_ITERATION = 4 * 2 * 256 * 256 * 32


def bench_mma_i8_peak(iterations: int, pairs: int, stream=None) -> None:
    """Enqueue the int8 tensor-core peak loop (pairs * iterations *
    PEAK_OPS_PER_PAIR_ITERATION operations); time it with CUDA events."""
    _check(lib().w8a8_bench_mma_i8_peak(int(iterations), int(pairs), _stream(stream)),
           "w8a8_bench_mma_i8_peak")


def debug_peek_tag() -> int:
    """The launch tag the next call using arrival counters will draw."""
    out = ctypes.c_uint64(0)
    _check(lib().w8a8_debug_peek_tag(ctypes.byref(out)), "w8a8_debug_peek_tag")
    return int(out.value)
