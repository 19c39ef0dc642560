"""ctypes binding of libfn.so: the C entry points under the same names.

Argument marshalling only: every step of the operation runs in the
library's HIP kernels.  PyTorch supplies device memory and streams; a
buffer argument may be a torch CUDA tensor (its data pointer is passed) or
a raw device address as an int.  A nonzero return code raises ``FnError``
with the library's message.  Importing this module raises ImportError if
the library has not been built (there is no CPU fallback).
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np
import torch  # loads the HIP runtime the library binds to
from torch.autograd import forward_ad

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; "
                      f"g.build()'` from the repository root")

_lib = ctypes.CDLL(LIB_PATH)

# what every call asks torch for, without the attribute reads on the way
_current_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_any_requires_grad, _increment_version = torch._C._any_requires_grad, torch._C._increment_version

FN_OK, FN_EINVAL, FN_EOVERFLOW, FN_EHIP = 0, -1, -2, -3
FN_OUT_FP32, FN_OUT_FP16, FN_OUT_FP16_PAD4, FN_OUT_BF16 = 0, 1, 2, 3

# fn_sample_params: eight int32 fields, 32 bytes
PARAMS_DTYPE = np.dtype(
    [("flip", "<i4"), ("erase", "<i4"), ("i", "<i4"), ("j", "<i4"),
     ("eh", "<i4"), ("ew", "<i4"), ("attempt", "<i4"), ("words_used", "<i4")]
)

_P = ctypes.c_void_p
_u64, _i64, _i32, _f32 = ctypes.c_uint64, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
_SIGS = {
    "fn_fused_normalize": [_P, _i64, _i32, _i32, _i32, _P, _P, _f32, _f32, _f32, _f32, _f32, _f32,
                           _u64, _i32, _P, _P],
    "fn_fused_normalize_ex": [_P, _i64, _i64, _i64, _i32, _i32, _i32, _P, _P, _f32, _f32, _f32,
                              _f32, _f32, _f32, _u64, _i64, _i32, _P, _P],
    "fn_params": [_u64, _i64, _i32, _i32, _f32, _f32, _f32, _f32, _f32, _f32, _P, _P],
    "fn_params_ex": [_u64, _i64, _i64, _i32, _i32, _f32, _f32, _f32, _f32, _f32, _f32, _P, _P],
    "fn_rms_norm": [_P, _i64, _P, _i64, _P, _i64, _i32, _f32, _i32, _P, _i64, _P, _i64, _P, _P],
    "fn_rms_norm_q8": [_P, _i64, _P, _i64, _P, _i64, _i32, _f32, _i32, _P, _i64, _P, _i64, _P, _P,
                       _P],
    "fn_quantize_rows": [_P, _i64, _i64, _i32, _i32, _P, _i64, _P, _P],
    "fn_rms_norm_backward": [_P, _i64, _P, _i64, _P, _P, _P, _i64, _i64, _i32, _i32, _P, _i64, _P,
                             _P, _i64, _P],
    "fn_rms_norm_backward_workspace": [_i64, _i32, _P],
    "fn_matmul_q8": [_P, _i64, _P, _P, _i64, _P, _P, _i64, _i64, _i32, _i32, _P, _i64, _P],
    "fn_test_erase_dims": [_P, _P, _i64, _i32, _i32, _f32, _f32, _f32, _f32, _P, _P, _P, _P],
    "fn_test_cr_ops": [_i32, _P, _P, _i64, _P, _P],
    "fn_test_stream": [_P, _P, _i64, _i32, _P],
    "fn_test_timeline": [_P, _i64],
}


def _declare(lib) -> None:
    for name, args in _SIGS.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ctypes.c_int
    lib.fn_last_error.argtypes = []
    lib.fn_last_error.restype = ctypes.c_char_p


_declare(_lib)

EXPORTED = ("fn_fused_normalize", "fn_fused_normalize_ex", "fn_params", "fn_params_ex",
            "fn_rms_norm", "fn_rms_norm_q8", "fn_quantize_rows", "fn_rms_norm_backward",
            "fn_rms_norm_backward_workspace", "fn_matmul_q8",
            "fn_last_error", "fn_test_erase_dims", "fn_test_cr_ops", "fn_test_stream",
            "fn_test_timeline")

TIMELINE_LIB_PATH = os.path.join(_HERE, "libfn_timeline.so")


def timeline_library():
    """The instrumented build libfn_timeline.so (same entry points; its
    tiles kernel records per-tile clock stamps, see fn_test_timeline), as a
    ctypes handle.  A measurement tool: the product path is libfn.so."""
    if not os.path.exists(TIMELINE_LIB_PATH):
        raise ImportError(f"{TIMELINE_LIB_PATH} is not built")
    lib = ctypes.CDLL(TIMELINE_LIB_PATH)
    _declare(lib)
    return lib


class FnError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"libfn error {code}: {message}")
        self.code = code


def fn_last_error() -> str:
    return _lib.fn_last_error().decode()


def _addr(x) -> int | None:
    """Device address of a torch tensor or an int (None/0 -> NULL)."""
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        return x.data_ptr()
    return int(x)


def _stream(stream) -> int | None:
    if stream is None:
        # the current stream's handle, without the 2.6 us that building a
        # torch.cuda.Stream object for it takes
        return _current_stream(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor that belongs to the call's stream: its memory was last used
    there.  One of the current stream's could still be in use by that, and be
    written from both."""
    if stream is None or _stream(stream) == _stream(None):
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _check(rc: int) -> int:
    if rc != FN_OK:
        raise FnError(rc, fn_last_error())
    return rc


_FLOATS: dict = {}  # recent constant arrays: the library only reads them during the call


def _host_floats(v, C: int):
    try:
        key = (C, v if isinstance(v, tuple) else tuple(v) if hasattr(v, "__len__") else v)
        a = _FLOATS.get(key)
        if a is not None:
            return a
    except TypeError:  # unhashable values
        key = None
    a = (ctypes.c_float * C)()
    vals = list(v) if hasattr(v, "__len__") else [v] * C
    if len(vals) != C:
        raise ValueError(f"expected {C} values, got {len(vals)}")
    for k, x in enumerate(vals):
        a[k] = float(x)
    if key is not None and len(_FLOATS) < 64:
        _FLOATS[key] = a
    return a


def fn_fused_normalize(in_u8, N, H, W, C, mean, std, flip_p, erase_p, scale_min, scale_max,
                       ratio_min, ratio_max, seed, out_dtype, out, stream=None) -> int:
    return _check(_lib.fn_fused_normalize(
        _addr(in_u8), N, H, W, C, _host_floats(mean, C), _host_floats(std, C), flip_p, erase_p,
        scale_min, scale_max, ratio_min, ratio_max, seed & 0xFFFFFFFFFFFFFFFF, out_dtype,
        _addr(out), _stream(stream)))


def fn_fused_normalize_ex(in_u8, in_row_stride, in_image_stride, N, H, W, C, mean, std, flip_p,
                          erase_p, scale_min, scale_max, ratio_min, ratio_max, seed,
                          first_sample_id, out_dtype, out, stream=None) -> int:
    return _check(_lib.fn_fused_normalize_ex(
        _addr(in_u8), in_row_stride, in_image_stride, N, H, W, C, _host_floats(mean, C),
        _host_floats(std, C), flip_p, erase_p, scale_min, scale_max, ratio_min, ratio_max,
        seed & 0xFFFFFFFFFFFFFFFF, first_sample_id, out_dtype, _addr(out), _stream(stream)))


def fn_params_ex(seed, first_sample_id, N, H, W, flip_p, erase_p, scale_min, scale_max,
                 ratio_min, ratio_max, params_dev, stream=None) -> int:
    return _check(_lib.fn_params_ex(seed & 0xFFFFFFFFFFFFFFFF, first_sample_id, N, H, W, flip_p,
                                    erase_p, scale_min, scale_max, ratio_min, ratio_max,
                                    _addr(params_dev), _stream(stream)))


def fn_params(seed, N, H, W, flip_p, erase_p, scale_min, scale_max, ratio_min, ratio_max,
              params_dev, stream=None) -> int:
    return _check(_lib.fn_params(seed & 0xFFFFFFFFFFFFFFFF, N, H, W, flip_p, erase_p, scale_min,
                                 scale_max, ratio_min, ratio_max, _addr(params_dev),
                                 _stream(stream)))


def fn_rms_norm(x, x_stride, residual, residual_stride, weight, rows, width, eps, dtype, sum_out,
                sum_stride, out, out_stride, rstd, stream=None) -> int:
    return _check(_lib.fn_rms_norm(_addr(x), x_stride, _addr(residual), residual_stride,
                                   _addr(weight), rows, width, eps, dtype, _addr(sum_out),
                                   sum_stride, _addr(out), out_stride, _addr(rstd),
                                   _stream(stream)))


def fn_rms_norm_q8(x, x_stride, residual, residual_stride, weight, rows, width, eps, dtype,
                   sum_out, sum_stride, codes, codes_stride, scales, rstd, stream=None) -> int:
    return _check(_lib.fn_rms_norm_q8(_addr(x), x_stride, _addr(residual), residual_stride,
                                      _addr(weight), rows, width, eps, dtype, _addr(sum_out),
                                      sum_stride, _addr(codes), codes_stride, _addr(scales),
                                      _addr(rstd), _stream(stream)))


def fn_quantize_rows(x, x_stride, rows, width, dtype, codes, codes_stride, scales,
                     stream=None) -> int:
    return _check(_lib.fn_quantize_rows(_addr(x), x_stride, rows, width, dtype, _addr(codes),
                                        codes_stride, _addr(scales), _stream(stream)))


def fn_rms_norm_backward(dout, dout_stride, h, h_stride, weight, rstd, dsum, dsum_stride, rows,
                         width, dtype, dx, dx_stride, dweight, workspace, workspace_bytes,
                         stream=None) -> int:
    return _check(_lib.fn_rms_norm_backward(
        _addr(dout), dout_stride, _addr(h), h_stride, _addr(weight), _addr(rstd), _addr(dsum),
        dsum_stride, rows, width, dtype, _addr(dx), dx_stride, _addr(dweight), _addr(workspace),
        workspace_bytes, _stream(stream)))


def fn_rms_norm_backward_workspace(rows, width) -> int:
    """The workspace's size in bytes."""
    n = _i64()
    _check(_lib.fn_rms_norm_backward_workspace(rows, width, ctypes.byref(n)))
    return n.value


def fn_matmul_q8(a, a_stride, a_scales, b, b_stride, b_scales, bias, M, N, K, out_dtype, out,
                 out_stride, stream=None) -> int:
    return _check(_lib.fn_matmul_q8(_addr(a), a_stride, _addr(a_scales), _addr(b), b_stride,
                                    _addr(b_scales), _addr(bias), M, N, K, out_dtype, _addr(out),
                                    out_stride, _stream(stream)))


def fn_test_erase_dims(w_scale, w_ratio, count, H, W, scale_min, scale_max, ratio_min, ratio_max,
                       eh, ew, accepted, stream=None) -> int:
    return _check(_lib.fn_test_erase_dims(_addr(w_scale), _addr(w_ratio), count, H, W, scale_min,
                                          scale_max, ratio_min, ratio_max, _addr(eh), _addr(ew),
                                          _addr(accepted), _stream(stream)))


def fn_test_cr_ops(op, a, b, count, out, stream=None) -> int:
    return _check(_lib.fn_test_cr_ops(op, _addr(a), _addr(b), count, _addr(out), _stream(stream)))


def fn_test_stream(src, dst, in_bytes, widen, stream=None) -> int:
    return _check(_lib.fn_test_stream(_addr(src), _addr(dst), in_bytes, widen, _stream(stream)))


def fn_test_timeline(stamps, tiles) -> int:
    """libfn.so records no timeline: this raises FnError (FN_EINVAL)."""
    return _check(_lib.fn_test_timeline(_addr(stamps), tiles))


# ------------------------------------------------------------ tensor helpers
#
# `stream`: a torch.cuda.Stream or a handle; the current stream if None.  What a
# helper allocates belongs to that stream, as with torch.cuda.stream(stream).
# As for torch's own work on several streams, the caller sees to it that the
# arguments are ready for the stream and live until it has finished, and waits
# for it before results are used elsewhere.

def fused_normalize(x: torch.Tensor, mean, std, flip_p=0.5, erase_p=0.0, scale=(0.02, 0.33),
                    ratio=(0.3, 3.3), seed=0, out_dtype=FN_OUT_FP32, out=None,
                    stream=None) -> torch.Tensor:
    """fn_fused_normalize on an (N, H, W, C) uint8 CUDA tensor; returns (or
    fills) the (N, H, W, C) float32/float16 output tensor, (N, H, W, 4)
    float16 for FN_OUT_FP16_PAD4."""
    if x.dtype != torch.uint8 or x.dim() != 4 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous (N, H, W, C) uint8 CUDA tensor")
    N, H, W, C = x.shape
    tdt = torch.float32 if out_dtype == FN_OUT_FP32 else torch.float16
    shape = (N, H, W, 4 if out_dtype == FN_OUT_FP16_PAD4 else C)
    if out is None:
        out = _empty(shape, tdt, x.device, stream)
    elif out.dtype != tdt or tuple(out.shape) != shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of shape %s and out_dtype" % (shape,))
    fn_fused_normalize(x, N, H, W, C, mean, std, flip_p, erase_p, scale[0], scale[1], ratio[0],
                       ratio[1], seed, out_dtype, out, stream)
    return out


def sample_params(N, H, W, flip_p=0.5, erase_p=0.0, scale=(0.02, 0.33), ratio=(0.3, 3.3), seed=0,
                  device="cuda", stream=None) -> torch.Tensor:
    """fn_params into a new (N, 8) int32 CUDA tensor (fields in PARAMS_DTYPE order)."""
    out = _empty((max(N, 0), 8), torch.int32, device, stream)
    fn_params(seed, N, H, W, flip_p, erase_p, scale[0], scale[1], ratio[0], ratio[1], out, stream)
    return out


def params_to_numpy(t: torch.Tensor) -> np.ndarray:
    """(N, 8) int32 tensor -> structured array with PARAMS_DTYPE fields."""
    return np.ascontiguousarray(t.cpu().numpy()).view(PARAMS_DTYPE).reshape(-1)


# ------------------------------------- tensor helpers: the 8-bit linear layer
#
# These are called once per layer and token, so they keep to the fewest
# attribute reads that check an argument.
#
# They compute and do not differentiate: no result has a gradient function.  A
# tensor that requires a gradient while gradients are recorded, or that carries
# a forward-mode tangent, is refused, for its derivative would be lost without
# a word.  In training they stand inside a torch.autograd.Function (rms_norm in
# its forward, rms_norm_backward in its backward), where torch records none.
# What a call writes counts a version, as with torch's in-place operations: a
# backward pass that saved such a tensor raises instead of using what has taken
# its place.

_TYPE_CODES = {torch.float32: FN_OUT_FP32, torch.float16: FN_OUT_FP16, torch.bfloat16: FN_OUT_BF16}
_CODE_TYPES = {code: t for t, code in _TYPE_CODES.items()}


def _refuse_gradients(*tensors) -> None:
    if _any_requires_grad(*tensors) and torch.is_grad_enabled():
        raise ValueError("an argument requires a gradient, which this call does not record: call "
                         "it under torch.no_grad() or within a torch.autograd.Function")
    if forward_ad._current_level >= 0 and any(
            t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise ValueError("an argument carries a forward-mode tangent, which this call does not "
                         "carry on")


def _type_code(dtype) -> int:
    code = _TYPE_CODES.get(dtype)
    if code is None:
        raise ValueError(f"dtype {dtype}: float32, float16 or bfloat16 is needed")
    return code


def _row_stride(t: torch.Tensor, name: str) -> int:
    """The row stride of a (..., D) tensor whose leading dimensions step by
    one common stride (any contiguous tensor, a slice of its last dimension,
    one row expanded to many) and whose last dimension is contiguous."""
    if t.is_contiguous():
        return t.shape[-1]
    shape, st = t.shape, t.stride()
    stride = None
    if shape[-1] <= 1 or st[-1] == 1:
        for d in range(t.dim() - 2, -1, -1):
            if shape[d] == 1:
                continue
            if stride is None:
                stride, span = st[d], st[d] * shape[d]
            elif st[d] == span:
                span *= shape[d]
            else:
                break
        else:
            return shape[-1] if stride is None else stride
    raise ValueError(f"{name}: the last dimension must be contiguous and the others one row stride "
                     "(use .contiguous())")


def _want(t, shape, dtype, dev: int, name: str, flat: bool = False, stream=None) -> torch.Tensor:
    """`t` if it has this shape, dtype and device (and is contiguous, if
    `flat`); a new tensor of the stream's if it is None."""
    if t is None:
        return _empty(shape, dtype, dev, stream)
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")
    if flat and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _rows_of(x: torch.Tensor):
    """(shape, rows, width, device index) of a (..., D) CUDA tensor."""
    shape, dev = x.shape, x.get_device()
    if dev < 0 or len(shape) < 1:
        raise ValueError("a CUDA tensor of at least one dimension is needed")
    width = shape[-1]
    return shape, (x.numel() // width if width else 0), width, dev


def _norm(x, weight, eps, residual, sum_out, stream, out_args, q8):
    """What both norms pass before and after their own outputs."""
    _refuse_gradients(x, weight, residual, sum_out, *out_args)
    shape, rows, width, dev = _rows_of(x)
    dtype = x.dtype
    code = _type_code(dtype)
    _want(weight, (width,), dtype, dev, "weight", True)
    res_at = sum_at = None
    res_stride = sum_stride = 0
    if residual is not None:
        _want(residual, shape, dtype, dev, "residual")
        sum_out = _want(sum_out, shape, dtype, dev, "sum_out", False, stream)
        res_at, sum_at = residual.data_ptr(), sum_out.data_ptr()
        res_stride = width if residual.is_contiguous() else _row_stride(residual, "residual")
        sum_stride = width if sum_out.is_contiguous() else _row_stride(sum_out, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out without a residual")
    x_stride = width if x.is_contiguous() else _row_stride(x, "x")
    if q8:
        codes, scales, rstd = out_args
        codes = _want(codes, shape, torch.int8, dev, "codes", False, stream)
        scales = _want(scales, shape[:-1], torch.float32, dev, "scales", True, stream)
        if rstd is not None:
            _want(rstd, shape[:-1], torch.float32, dev, "rstd", True)
        _check(_lib.fn_rms_norm_q8(
            x.data_ptr(), x_stride, res_at, res_stride, weight.data_ptr(), rows, width, eps, code,
            sum_at, sum_stride, codes.data_ptr(),
            width if codes.is_contiguous() else _row_stride(codes, "codes"), scales.data_ptr(),
            None if rstd is None else rstd.data_ptr(), _stream(stream)))
        _increment_version([t for t in (codes, scales, sum_out, rstd) if t is not None])
        return codes, scales, x if residual is None else sum_out
    out, rstd = out_args
    out = _want(out, shape, dtype, dev, "out", False, stream)
    rstd = _want(rstd, shape[:-1], torch.float32, dev, "rstd", True, stream)
    _check(_lib.fn_rms_norm(
        x.data_ptr(), x_stride, res_at, res_stride, weight.data_ptr(), rows, width, eps, code,
        sum_at, sum_stride, out.data_ptr(), width if out.is_contiguous() else _row_stride(out, "out"),
        rstd.data_ptr(), _stream(stream)))
    _increment_version((out, rstd) if residual is None else (out, rstd, sum_out))
    return out, rstd, x if residual is None else sum_out


def rms_norm(x, weight, eps=1e-6, residual=None, out=None, sum_out=None, rstd=None, stream=None):
    """fn_rms_norm on (..., D) CUDA tensors of one dtype.  Returns (out, rstd,
    h): the norm of h = x + residual, each row's 1/rms (fp32), and h itself
    (x when there is no residual).  out and sum_out may be x or residual."""
    return _norm(x, weight, eps, residual, sum_out, stream, (out, rstd), False)


def rms_norm_q8(x, weight, eps=1e-6, residual=None, codes=None, scales=None, sum_out=None,
                rstd=None, stream=None):
    """fn_rms_norm_q8 on (..., D) CUDA tensors of one dtype.  Returns (codes,
    scales, h): int8 codes of the shape of x, an fp32 scale per row, and h = x
    + residual (x when there is no residual).  sum_out may be x or residual;
    rstd, if given, receives each row's 1/rms."""
    return _norm(x, weight, eps, residual, sum_out, stream, (codes, scales, rstd), True)


def quantize_rows(x, codes=None, scales=None, stream=None):
    """fn_quantize_rows on a (..., D) CUDA tensor: (int8 codes of its shape,
    an fp32 scale per row)."""
    _refuse_gradients(x, scales)
    shape, rows, width, dev = _rows_of(x)
    codes = _want(codes, shape, torch.int8, dev, "codes", False, stream)
    scales = _want(scales, shape[:-1], torch.float32, dev, "scales", True, stream)
    _check(_lib.fn_quantize_rows(
        x.data_ptr(), width if x.is_contiguous() else _row_stride(x, "x"), rows, width,
        _type_code(x.dtype), codes.data_ptr(),
        width if codes.is_contiguous() else _row_stride(codes, "codes"), scales.data_ptr(),
        _stream(stream)))
    _increment_version((codes, scales))
    return codes, scales


_workspace_bytes = functools.lru_cache(maxsize=256)(fn_rms_norm_backward_workspace)  # of the sizes


def rms_norm_backward_workspace(rows, width, device="cuda") -> torch.Tensor:
    """A workspace for rms_norm_backward on rows of this size."""
    return torch.empty(_workspace_bytes(rows, width), dtype=torch.uint8, device=device)


def rms_norm_backward(dout, h, weight, rstd, dsum=None, dx=None, dweight=None, workspace=None,
                      stream=None):
    """fn_rms_norm_backward on (..., D) CUDA tensors of one dtype; rstd and h
    as rms_norm returned them.  Returns (dx, dweight): the gradient of x (and
    of the residual) and the fp32 gradient of the weight.  dx may be dout, h
    or dsum.  Without a workspace one is allocated for the call.  The last bit
    of dx in 16-bit rows of odd width beyond 2,560 may depend on whether the
    row's number and dout's row stride are odd."""
    _refuse_gradients(dout, h, weight, rstd, dsum, dx, dweight)
    shape, rows, width, dev = _rows_of(h)
    dtype = h.dtype
    code = _type_code(dtype)
    _want(weight, (width,), dtype, dev, "weight", True)
    _want(dout, shape, dtype, dev, "dout")
    _want(rstd, shape[:-1], torch.float32, dev, "rstd", True)
    dsum_at, dsum_stride = None, 0
    if dsum is not None:
        _want(dsum, shape, dtype, dev, "dsum")
        dsum_at = dsum.data_ptr()
        dsum_stride = width if dsum.is_contiguous() else _row_stride(dsum, "dsum")
    dx = _want(dx, shape, dtype, dev, "dx", False, stream)
    dweight = _want(dweight, (width,), torch.float32, dev, "dweight", True, stream)
    if workspace is None:
        size = _workspace_bytes(rows, width)
        if size:
            workspace = _empty((size,), torch.uint8, dev, stream)
        at = workspace.data_ptr() if size else None
    else:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        at, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(_lib.fn_rms_norm_backward(
        dout.data_ptr(), width if dout.is_contiguous() else _row_stride(dout, "dout"),
        h.data_ptr(), width if h.is_contiguous() else _row_stride(h, "h"), weight.data_ptr(),
        rstd.data_ptr(), dsum_at, dsum_stride, rows, width, code, dx.data_ptr(),
        width if dx.is_contiguous() else _row_stride(dx, "dx"), dweight.data_ptr(), at, size,
        _stream(stream)))
    _increment_version((dx, dweight) if workspace is None else (dx, dweight, workspace))
    return dx, dweight


def matmul_q8(a, a_scales, b, b_scales, bias=None, out_dtype=FN_OUT_BF16, out=None, stream=None):
    """fn_matmul_q8: the (..., N) product of int8 codes a (..., K) with a scale
    per row and b (N, K) with a scale per row, plus an fp32 bias (N,).  Given
    `out`, its dtype counts and not out_dtype."""
    _refuse_gradients(a_scales, b_scales, bias, out)
    shape, b_shape, dev = a.shape, b.shape, a.get_device()
    if a.dtype is not torch.int8 or b.dtype is not torch.int8 or len(shape) < 1 \
            or len(b_shape) != 2 or dev < 0 or b.get_device() != dev or shape[-1] != b_shape[1]:
        raise ValueError("a must be an int8 (..., K) CUDA tensor and b an int8 (N, K) one beside it")
    N, K = b_shape
    lead = shape[:-1]
    M = lead.numel()
    if out is None:
        if out_dtype not in _CODE_TYPES:
            raise ValueError(f"unknown out_dtype {out_dtype}")
        out = _empty((*lead, N), _CODE_TYPES[out_dtype], dev, stream)
    else:
        out_dtype = _type_code(out.dtype)
        _want(out, (*lead, N), out.dtype, dev, "out")
    _want(a_scales, lead, torch.float32, dev, "a_scales", True)
    _want(b_scales, (N,), torch.float32, dev, "b_scales", True)
    if bias is not None:
        _want(bias, (N,), torch.float32, dev, "bias", True)
    _check(_lib.fn_matmul_q8(
        a.data_ptr(), K if a.is_contiguous() else _row_stride(a, "a"), a_scales.data_ptr(),
        b.data_ptr(), K if b.is_contiguous() else _row_stride(b, "b"), b_scales.data_ptr(),
        None if bias is None else bias.data_ptr(), M, N, K, out_dtype, out.data_ptr(),
        N if out.is_contiguous() else _row_stride(out, "out"), _stream(stream)))
    _increment_version((out,))
    return out
