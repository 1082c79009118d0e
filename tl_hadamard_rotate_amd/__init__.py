"""Python binding of libtl (ternary g128 linear layer with a signed
block-Hadamard rotation, MI355X / gfx950).

Argument marshalling only: every function checks dtype, shape, device and
contiguity of torch tensors, then passes raw device pointers and torch's
current HIP stream to the C ABI declared in include/tl.h.  All computation runs
in the library's HIP kernels; there is no fallback path.  A missing library
raises at first use.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtl.so")

FMT_TRIT5 = 0
FMT_SLOT2 = 1
FMT_BIT1 = 2
TL_F32 = 0
TL_F16 = 1
TL_BF16 = 2
TL_I8 = 3
BLOCK = 1024
GROUP = 128

_STATUS = {0: "TL_OK", 1: "TL_ERR_NULL", 2: "TL_ERR_SHAPE", 3: "TL_ERR_FORMAT",
           4: "TL_ERR_ALIGN", 5: "TL_ERR_ALIAS", 6: "TL_ERR_LAUNCH", 7: "TL_ERR_DTYPE",
           8: "TL_ERR_WORKSPACE", 9: "TL_ERR_DATA", 10: "TL_ERR_VALUE"}

_lib = None


class TLError(RuntimeError):
    def __init__(self, call: str, status: int, detail: str = ""):
        self.status = status
        self.status_name = _STATUS.get(status, f"status {status}")
        msg = f"{call} failed: {self.status_name}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


def lib() -> ctypes.CDLL:
    """Load libtl.so (built by ``python -m tl_hadamard_rotate_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m tl_hadamard_rotate_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        p, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        sig = {
            "tl_packed_bytes": (i64, [i64, i64, i32]),
            "tl_pack": (i32, [p, i64, i64, i32, p, p, p]),
            "tl_unpack": (i32, [p, i64, i64, i32, p, p]),
            "tl_hadamard_rotate": (i32, [p, p, i64, i64, p, p]),
            "tl_gemv": (i32, [p, p, i32, p, i64, i64, i64, p, i32, p]),
            "tl_gemm": (i32, [p, p, i32, p, i64, i64, i64, p, i32, p, i64, p]),
            "tl_gemm_noalloc": (i32, [p, p, i32, p, i64, i64, i64, p, i32, p]),
            "tl_gemm_workspace_bytes": (i64, [i64, i64, i64, i32]),
            "tl_gemm_bf16_workspace_bytes": (i64, [i64, i64, i64, i32]),
            "tl_gemm_plan": (i32, [i64, i64, i64, p]),
            "tl_linear": (i32, [p, p, i32, p, p, i64, i64, i64, p, p, i32, p, i64, p]),
            "tl_quantize": (i32, [p, p, i64, i64, p, p, p]),
            "tl_gemm_bf16": (i32, [p, p, i32, p, i64, i64, i64, p, i32, p, i64, p]),
            "tl_chain_plan_bytes": (i64, [i32]),
            "tl_chain_sync_bytes": (i64, [i32]),
            "tl_chain_encode": (i32, [p, i32, p, i64]),
            "tl_linear_chain": (i32, [p, i32, p, p]),
            "tl_rms_norm": (i32, [p, p, p, p, i64, i64, i32, f32, p, p, i32, p, p]),
            "tl_q4_packed_bytes": (i64, [i64, i64]),
            "tl_q4_quantize": (i32, [p, p, i64, i64, i32, i32, p, p, p]),
            "tl_q4_dequantize": (i32, [p, p, i64, i64, i32, p, i32, p]),
            "tl_q4_gemv_workspace_bytes": (i64, [i64, i64, i64]),
            "tl_q4_gemv": (i32, [p, p, i32, p, i32, p, i64, i64, i64, p, i32, p, i64, p]),
            "tl_f8_quantize": (i32, [p, i64, i64, i32, p, p, p]),
            "tl_f8_dequantize": (i32, [p, p, i64, i64, p, i32, p]),
            "tl_f8_gemm_workspace_bytes": (i64, [i64, i64, i64]),
            "tl_f8_gemm": (i32, [p, p, p, p, i64, i64, i64, p, i32, p, i64, p]),
            "tl_f8_gemm_approx": (i32, [p, p, p, p, i64, i64, i64, p, i32, p, i64, p]),
            "tl_q4_rows": (i32, [p, p, i32, p, i64, i64, i64, f32, p, i32, p]),
            "tl_f8_rows": (i32, [p, p, p, i64, i64, i64, f32, p, i32, p]),
            "tl_adjust_logits": (i32, [p, i64, i64, i32, p, i64, p, p, p, p, p, p, p, i64, p, p, i32, p]),
            "tl_status_str": (ctypes.c_char_p, [i32]),
            "tl_last_error": (ctypes.c_char_p, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(call: str, status: int) -> None:
    if status != 0:
        detail = lib().tl_last_error().decode() if status in (6, 9) else ""
        raise TLError(call, status, detail)


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int | None = None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def packed_bytes(n: int, k: int, fmt: int) -> int:
    return int(lib().tl_packed_bytes(n, k, fmt))


def pack(codes: torch.Tensor, fmt: int, bad_count: torch.Tensor | None = None) -> torch.Tensor:
    """int8 codes [N, K] -> uint8 packed [N, row_bytes] (see include/tl.h)."""
    _need(codes, "codes", torch.int8, 2)
    if bad_count is not None:
        _need(bad_count, "bad_count", torch.int32)
    n, k = codes.shape
    nbytes = packed_bytes(n, k, fmt)
    if nbytes < 0:
        raise TLError("tl_pack", 2)
    out = torch.empty((n, nbytes // n), dtype=torch.uint8, device=codes.device)
    _check("tl_pack", lib().tl_pack(_ptr(codes), n, k, fmt, _ptr(out), _ptr(bad_count),
                                    _stream(codes)))
    return out


def unpack(packed: torch.Tensor, k: int, fmt: int) -> torch.Tensor:
    _need(packed, "packed", torch.uint8, 2)
    n = packed.shape[0]
    out = torch.empty((n, k), dtype=torch.int8, device=packed.device)
    if packed.numel() != packed_bytes(n, k, fmt):
        raise ValueError("packed size does not match K and the format")
    _check("tl_unpack", lib().tl_unpack(_ptr(packed), n, k, fmt, _ptr(out), _stream(packed)))
    return out


def hadamard_rotate(x: torch.Tensor, signs: torch.Tensor,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """Signed 1024-block Hadamard rotation of the rows of fp16 x [M, K]."""
    _need(x, "x", torch.float16, 2)
    _need(signs, "signs", torch.int8, 1)
    m, k = x.shape
    if signs.shape[0] != k:
        raise ValueError("signs must have K entries")
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, "out", torch.float16, 2)
        if out.shape != x.shape:
            raise ValueError("out must have the shape of x")
    _check("tl_hadamard_rotate",
           lib().tl_hadamard_rotate(_ptr(x), _ptr(signs), m, k, _ptr(out), _stream(x)))
    return out


def quantize(w: torch.Tensor, signs: torch.Tensor):
    """Rotate fp32 weight rows w [N, K] with the signed transform and round
    them to ternary g128: returns (codes int8 [N, K], scales float16 [N, K/128])."""
    _need(w, "w", torch.float32, 2)
    _need(signs, "signs", torch.int8, 1)
    n, k = w.shape
    if signs.shape[0] != k:
        raise ValueError("signs must have K entries")
    codes = torch.empty((n, k), dtype=torch.int8, device=w.device)
    scales = torch.empty((n, k // 128), dtype=torch.float16, device=w.device)
    _check("tl_quantize", lib().tl_quantize(_ptr(w), _ptr(signs), n, k, _ptr(codes), _ptr(scales),
                                            _stream(w)))
    return codes, scales


def gemm_workspace_bytes(m: int, n: int, k: int, fmt: int) -> int:
    """Device workspace bytes tl_gemm / tl_linear need (0: none)."""
    b = int(lib().tl_gemm_workspace_bytes(m, n, k, fmt))
    if b < 0:
        raise TLError("tl_gemm_workspace_bytes", 2)
    return b


def gemm_bf16_workspace_bytes(m: int, n: int, k: int, fmt: int) -> int:
    """Device workspace bytes tl_gemm_bf16 needs."""
    b = int(lib().tl_gemm_bf16_workspace_bytes(m, n, k, fmt))
    if b < 0:
        raise TLError("tl_gemm_bf16_workspace_bytes", 2)
    return b


def gemm_plan(m: int, n: int, k: int) -> tuple[int, int, int]:
    """tl_gemm's launch plan: (output tiles, tiles computed whole, K parts of
    each remaining tile)."""
    out = (ctypes.c_int64 * 3)()
    _check("tl_gemm_plan", lib().tl_gemm_plan(m, n, k, out))
    return int(out[0]), int(out[1]), int(out[2])


def _workspace(m, n, k, fmt, device, workspace, size=None):
    """(pointer, bytes) of the workspace a prefill call needs: the caller's
    uint8 tensor when given, else one from torch's allocator (None when the
    call needs none)."""
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1)
        return _ptr(workspace), workspace.numel(), workspace
    need = (size or gemm_workspace_bytes)(m, n, k, fmt)
    if need == 0:
        return _ptr(None), 0, None
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    return _ptr(ws), need, ws


def _linear(call: str, packed, scales, fmt, x_rot, out_dtype, out, x_dtype=torch.float16,
            workspace=None):
    _need(packed, "packed", torch.uint8, 2)
    _need(scales, "scales", torch.float16, 2)
    _need(x_rot, "x_rot", x_dtype, 2)
    m, k = x_rot.shape
    n = packed.shape[0]
    if scales.shape != (n, k // GROUP):
        raise ValueError(f"scales must be [N, K/128] = {(n, k // GROUP)}, got {tuple(scales.shape)}")
    if packed.numel() != packed_bytes(n, k, fmt):
        raise ValueError("packed size does not match N, K and the format")
    if out_dtype not in (torch.float32, torch.float16):
        raise TypeError("out_dtype must be float32 or float16")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=x_rot.device)
    else:
        _need(out, "out", out_dtype, 2)
        if out.shape != (m, n):
            raise ValueError("out must be [M, N]")
    yd = TL_F32 if out_dtype == torch.float32 else TL_F16
    fn = getattr(lib(), call)
    if call in ("tl_gemv", "tl_gemm_noalloc"):
        _check(call, fn(_ptr(packed), _ptr(scales), fmt, _ptr(x_rot), m, n, k, _ptr(out), yd,
                        _stream(x_rot)))
    else:
        size = gemm_bf16_workspace_bytes if call == "tl_gemm_bf16" else None
        wp, wb, _keep = _workspace(m, n, k, fmt, x_rot.device, workspace, size)
        _check(call, fn(_ptr(packed), _ptr(scales), fmt, _ptr(x_rot), m, n, k, _ptr(out), yd,
                        wp, wb, _stream(x_rot)))
    return out


def gemv(packed, scales, fmt, x_rot, out_dtype=torch.float32, out=None) -> torch.Tensor:
    """y[M, N] = x_rot . dequant(codes, scales)^T, decode-shaped (M <= 16)."""
    return _linear("tl_gemv", packed, scales, fmt, x_rot, out_dtype, out)


def gemm_noalloc(packed, scales, fmt, x_rot, out_dtype=torch.float32, out=None) -> torch.Tensor:
    """``gemm`` through tl_gemm_noalloc: no workspace argument and no
    allocation by the library (its workspace is a fixed device array of
    TL_GEMM_NOALLOC_MAX_WORKSPACE bytes shared by all calls on a GPU)."""
    return _linear("tl_gemm_noalloc", packed, scales, fmt, x_rot, out_dtype, out)


def gemm_bf16(packed, scales, fmt, x_rot, out_dtype=torch.float32, out=None,
              workspace=None) -> torch.Tensor:
    """The prefill product with bfloat16 rotated activations x_rot [M, K]: each
    row taken exactly to binary16 under a power-of-two factor, then the
    binary16 product (``workspace``: at least ``gemm_bf16_workspace_bytes``)."""
    return _linear("tl_gemm_bf16", packed, scales, fmt, x_rot, out_dtype, out,
                   x_dtype=torch.bfloat16, workspace=workspace)


def gemm(packed, scales, fmt, x_rot, out_dtype=torch.float32, out=None,
         workspace=None) -> torch.Tensor:
    """Same as ``gemv``, prefill-shaped (large M).  ``workspace`` (uint8, at
    least ``gemm_workspace_bytes``) is taken from torch's allocator when not
    given."""
    return _linear("tl_gemm", packed, scales, fmt, x_rot, out_dtype, out, workspace=workspace)


def linear(packed, scales, fmt, x, signs, out_dtype=torch.float32, out=None,
           x_rot=None, workspace=None) -> torch.Tensor:
    """y[M, N] = R(x) . dequant(codes, scales)^T on unrotated fp16 x [M, K];
    x_rot (allocated when None) receives R(x).  One fused launch at M = 1
    with the 2-bit-slot and dense trit packings (within their K limits)."""
    _need(packed, "packed", torch.uint8, 2)
    _need(scales, "scales", torch.float16, 2)
    _need(x, "x", torch.float16, 2)
    _need(signs, "signs", torch.int8, 1)
    m, k = x.shape
    n = packed.shape[0]
    if signs.shape[0] != k:
        raise ValueError("signs must have K entries")
    if scales.shape != (n, k // GROUP):
        raise ValueError(f"scales must be [N, K/128] = {(n, k // GROUP)}, got {tuple(scales.shape)}")
    if packed.numel() != packed_bytes(n, k, fmt):
        raise ValueError("packed size does not match N, K and the format")
    if out_dtype not in (torch.float32, torch.float16):
        raise TypeError("out_dtype must be float32 or float16")
    if x_rot is None:
        x_rot = torch.empty_like(x)
    else:
        _need(x_rot, "x_rot", torch.float16, 2)
        if x_rot.shape != x.shape:
            raise ValueError("x_rot must have the shape of x")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=x.device)
    else:
        _need(out, "out", out_dtype, 2)
        if out.shape != (m, n):
            raise ValueError("out must be [M, N]")
    yd = TL_F32 if out_dtype == torch.float32 else TL_F16
    if m >= 64:
        wp, wb, _keep = _workspace(m, n, k, fmt, x.device, workspace)
    else:
        wp, wb = _ptr(None), 0
    _check("tl_linear", lib().tl_linear(_ptr(packed), _ptr(scales), fmt, _ptr(x), _ptr(signs), m,
                                        n, k, _ptr(x_rot), _ptr(out), yd, wp, wb, _stream(x)))
    return out


_REAL = {torch.float32: TL_F32, torch.float16: TL_F16, torch.bfloat16: TL_BF16}
_I8, _U8, _F16, _F32 = torch.int8, torch.uint8, torch.float16, torch.float32
# (a torch without GPU support has neither; the calls refuse its tensors before they ask)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None)

# The calls below take microseconds, so their checks are written out: each
# tensor's type, shape, device and contiguity in one condition, and only a
# tensor that fails it goes to the function that says why.


def _refuse(t, name: str, dtype: torch.dtype, shape, index: int) -> None:
    """Raise for a tensor that is not a contiguous one of this type and shape
    on this device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    raise ValueError(f"{name} must be contiguous {tuple(shape)}, got {tuple(t.shape)}")


def _rows(t, name: str):
    """(TL_ type, shape, device index) of a contiguous 2-D device tensor of real numbers."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dt = _REAL.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    shape, index = t.shape, t.get_device()
    if index < 0 or len(shape) != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D device tensor")
    return dt, shape, index


def _out_type(dtype: torch.dtype) -> int:
    dt = _REAL.get(dtype)
    if dt is None:
        raise TypeError(f"out_dtype must be float32, float16 or bfloat16, got {dtype}")
    return dt


def _call(name: str, index: int, args: tuple) -> None:
    """One library call on the device's current stream, with that device
    current (a stream and the look-ups of a launch belong to a device)."""
    fn = getattr(_lib or lib(), name)
    if index == _get_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st:
        _check(name, st)


def _rms_norm(x, dt, shape, index, gain, eps, residual, signs, sum_out, out, out_dtype, out_scales):
    dtype = x.dtype
    m, k = shape
    row = (k,)
    if not (isinstance(gain, torch.Tensor) and gain.dtype is dtype and gain.shape == row and
            gain.get_device() == index and gain.is_contiguous()):
        _refuse(gain, "gain", dtype, row, index)
    rp = sp = gp = None
    if residual is not None:
        if not (isinstance(residual, torch.Tensor) and residual.dtype is dtype and
                residual.shape == shape and residual.get_device() == index and
                residual.is_contiguous()):
            _refuse(residual, "residual", dtype, shape, index)
        if sum_out is None:
            sum_out = torch.empty_like(x)
        elif not (isinstance(sum_out, torch.Tensor) and sum_out.dtype is dtype and
                  sum_out.shape == shape and sum_out.get_device() == index and
                  sum_out.is_contiguous()):
            _refuse(sum_out, "sum_out", dtype, shape, index)
        rp, sp = residual.data_ptr(), sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    if signs is not None:
        if not (isinstance(signs, torch.Tensor) and signs.dtype is _I8 and signs.shape == row and
                signs.get_device() == index and signs.is_contiguous()):
            _refuse(signs, "signs", _I8, row, index)
        gp = signs.data_ptr()
    _call("tl_rms_norm", index, (x.data_ptr(), rp, gain.data_ptr(), gp, m, k, dt, eps, sp,
                                 out.data_ptr(), out_dtype, out_scales))
    return sum_out


def rms_norm(x, gain, eps, residual=None, signs=None, out_dtype=torch.float16, sum_out=None,
             out=None):
    """Root-mean-square norm of the rows of x [M, K] (float32, float16 or
    bfloat16), with the addition of ``residual`` in front and, with ``signs``,
    the signed rotation of the ternary linear behind it: ``out`` is then its
    x_rot (see tl_rms_norm).  Returns out, or (out, sum) with a residual; the
    sum x + residual goes to ``sum_out``, which may be x or residual itself."""
    yd = _out_type(out_dtype)
    dt, shape, index = _rows(x, "x")
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=x.device)
    elif not (isinstance(out, torch.Tensor) and out.dtype is out_dtype and out.shape == shape and
              out.get_device() == index and out.is_contiguous()):
        _refuse(out, "out", out_dtype, shape, index)
    s = _rms_norm(x, dt, shape, index, gain, eps, residual, signs, sum_out, out, yd, None)
    return out if s is None else (out, s)


def rms_norm_i8(x, gain, eps, residual=None, signs=None, sum_out=None, out=None, scales=None):
    """``rms_norm`` with 8-bit outputs for ``q4_gemv``: returns (codes int8
    [M, K], scales float32 [M, K/128]), and the sum behind them with a
    residual; value = code * scale of its 128."""
    dt, shape, index = _rows(x, "x")
    m, k = shape
    if k % GROUP:
        raise ValueError("K must be a multiple of 128")
    groups = (m, k // GROUP)
    if out is None:
        out = torch.empty(shape, dtype=_I8, device=x.device)
    elif not (isinstance(out, torch.Tensor) and out.dtype is _I8 and out.shape == shape and
              out.get_device() == index and out.is_contiguous()):
        _refuse(out, "out", _I8, shape, index)
    if scales is None:
        scales = torch.empty(groups, dtype=_F32, device=x.device)
    elif not (isinstance(scales, torch.Tensor) and scales.dtype is _F32 and
              scales.shape == groups and scales.get_device() == index and scales.is_contiguous()):
        _refuse(scales, "scales", _F32, groups, index)
    s = _rms_norm(x, dt, shape, index, gain, eps, residual, signs, sum_out, out, TL_I8,
                  scales.data_ptr())
    return (out, scales) if s is None else (out, scales, s)


def q4_packed_bytes(n: int, k: int) -> int:
    return int(lib().tl_q4_packed_bytes(n, k))


def q4_quantize(w, group=GROUP, signs=None, packed=None, scales=None):
    """Weight rows w [N, K] to 4-bit codes with a binary16 scale per ``group``
    (32, 64 or 128) weights, after the signed rotation of the rows when
    ``signs`` is given: returns (packed uint8 [N, K/2], scales float16
    [N, K/group]); the layout is in include/tl.h."""
    dt, (n, k), index = _rows(w, "w")
    if group not in (32, 64, 128) or k % GROUP:
        raise ValueError("group must be 32, 64 or 128 and K a multiple of 128")
    gp = None
    if signs is not None:
        if not (isinstance(signs, torch.Tensor) and signs.dtype is _I8 and signs.shape == (k,) and
                signs.get_device() == index and signs.is_contiguous()):
            _refuse(signs, "signs", _I8, (k,), index)
        gp = signs.data_ptr()
    halves, groups = (n, k // 2), (n, k // group)
    if packed is None:
        packed = torch.empty(halves, dtype=_U8, device=w.device)
    elif not (isinstance(packed, torch.Tensor) and packed.dtype is _U8 and
              packed.shape == halves and packed.get_device() == index and packed.is_contiguous()):
        _refuse(packed, "packed", _U8, halves, index)
    if scales is None:
        scales = torch.empty(groups, dtype=_F16, device=w.device)
    elif not (isinstance(scales, torch.Tensor) and scales.dtype is _F16 and
              scales.shape == groups and scales.get_device() == index and scales.is_contiguous()):
        _refuse(scales, "scales", _F16, groups, index)
    _call("tl_q4_quantize", index, (w.data_ptr(), gp, n, k, dt, group, packed.data_ptr(),
                                    scales.data_ptr()))
    return packed, scales


def _q4_shape(packed, scales):
    """(N, K, group, device index) of packed 4-bit weights and their scales."""
    if not (isinstance(packed, torch.Tensor) and isinstance(scales, torch.Tensor)):
        raise TypeError("packed and scales must be torch.Tensors")
    if packed.dtype is not _U8 or scales.dtype is not _F16:
        raise TypeError("packed must be uint8 and scales float16")
    index = packed.get_device()
    if index < 0 or scales.get_device() != index:
        raise ValueError("packed and scales must be device tensors, on the same device")
    ps, ss = packed.shape, scales.shape
    if len(ps) != 2 or len(ss) != 2 or not packed.is_contiguous() or not scales.is_contiguous():
        raise ValueError("packed and scales must be contiguous with 2 dims")
    n, half = ps
    groups = ss[1]
    k = 2 * half
    group = k // groups if groups else 0
    if ss[0] != n or k % GROUP or group not in (32, 64, 128) or group * groups != k:
        raise ValueError(f"packed {tuple(ps)} and scales {tuple(ss)} must be "
                         "[N, K/2] and [N, K/group], group 32, 64 or 128, K a multiple of 128")
    return n, k, group, index


def q4_dequantize(packed, scales, out_dtype=torch.float16, out=None) -> torch.Tensor:
    """The weights [N, K] that 4-bit codes and scales stand for."""
    n, k, group, index = _q4_shape(packed, scales)
    dt = _out_type(out_dtype)
    if out is None:
        out = torch.empty((n, k), dtype=out_dtype, device=packed.device)
    elif not (isinstance(out, torch.Tensor) and out.dtype is out_dtype and out.shape == (n, k) and
              out.get_device() == index and out.is_contiguous()):
        _refuse(out, "out", out_dtype, (n, k), index)
    _call("tl_q4_dequantize", index, (packed.data_ptr(), scales.data_ptr(), n, k, group,
                                      out.data_ptr(), dt))
    return out


def q4_gemv_workspace_bytes(m: int, n: int, k: int) -> int:
    """Device workspace bytes tl_q4_gemv needs (0 while m * k <= 16384)."""
    b = int(lib().tl_q4_gemv_workspace_bytes(m, n, k))
    if b < 0:
        raise TLError("tl_q4_gemv_workspace_bytes", 2)
    return b


@functools.lru_cache(maxsize=4096)
def _q4_workspace(index: int, m: int, n: int, k: int) -> int:
    """q4_gemv_workspace_bytes of a shape, asked once a device."""
    with torch.cuda.device(index):
        return q4_gemv_workspace_bytes(m, n, k)


def q4_gemv(packed, scales, x, x_scales=None, out_dtype=torch.float32, out=None,
            workspace=None) -> torch.Tensor:
    """y[M, N] = x . dequant4(packed, scales)^T for few tokens (M <= 64): x
    [M, K] float16 or bfloat16, or int8 with ``x_scales`` float32 [M, K/128]
    (``rms_norm_i8``).  ``workspace`` (uint8, at least
    ``q4_gemv_workspace_bytes``) is taken from torch's allocator when not given."""
    n, k, group, index = _q4_shape(packed, scales)
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    xs = x.shape
    if len(xs) != 2 or xs[1] != k or x.get_device() != index or not x.is_contiguous():
        raise ValueError(f"x must be a contiguous [M, {k}] tensor on {packed.device}")
    m = xs[0]
    sp = None
    if x.dtype is _I8:
        xd = TL_I8
        if x_scales is None:
            raise ValueError("int8 activations need x_scales")
        groups = (m, k // GROUP)
        if not (isinstance(x_scales, torch.Tensor) and x_scales.dtype is _F32 and
                x_scales.shape == groups and x_scales.get_device() == index and
                x_scales.is_contiguous()):
            _refuse(x_scales, "x_scales", _F32, groups, index)
        sp = x_scales.data_ptr()
    else:
        xd = _REAL.get(x.dtype)
        if xd is None or xd == TL_F32:
            raise TypeError(f"x must be float16, bfloat16 or int8, got {x.dtype}")
        if x_scales is not None:
            raise ValueError("x_scales go with int8 activations")
    yd = _out_type(out_dtype)
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=packed.device)
    elif not (isinstance(out, torch.Tensor) and out.dtype is out_dtype and out.shape == (m, n) and
              out.get_device() == index and out.is_contiguous()):
        _refuse(out, "out", out_dtype, (m, n), index)
    wp, wb = None, 0
    if workspace is not None:
        if not (isinstance(workspace, torch.Tensor) and workspace.dtype is _U8 and
                workspace.dim() == 1 and workspace.get_device() == index and
                workspace.is_contiguous()):
            _refuse(workspace, "workspace", _U8, ("bytes",), index)
        wp, wb = workspace.data_ptr(), workspace.numel()
    elif m * k > 16384:
        wb = _q4_workspace(index, m, n, k)
        if wb:
            workspace = torch.empty(wb, dtype=_U8, device=packed.device)
            wp = workspace.data_ptr()
    _call("tl_q4_gemv", index, (packed.data_ptr(), scales.data_ptr(), group, x.data_ptr(), xd, sp, m,
                                n, k, out.data_ptr(), yd, wp, wb))
    return out


class Q4Linear:
    """A linear layer with 4-bit weights and group scales, for the matrices
    beside the ternary ones.  With ``signs`` the weights carry the folded
    rotation (``q4_quantize`` with the same signs) and ``forward`` rotates its
    float16 input first, as ``TernaryLinear`` does; int8 input with scales
    (``rms_norm_i8``) has been rotated there."""

    def __init__(self, packed, scales, signs=None):
        self.packed, self.scales, self.signs = packed, scales, signs

    def forward(self, x: torch.Tensor, x_scales=None, out_dtype=torch.float32) -> torch.Tensor:
        if self.signs is not None and x.dtype != torch.int8:
            x = hadamard_rotate(x, self.signs)
        return q4_gemv(self.packed, self.scales, x, x_scales, out_dtype)

    __call__ = forward


# (torch has the scales' type from 2.7 on; the other calls do without)
_F8, _E8 = getattr(torch, "float8_e4m3fn", None), getattr(torch, "float8_e8m0fnu", None)
_I32 = torch.int32


def _no_f8_types():
    raise RuntimeError(f"torch {torch.__version__} lacks float8_e4m3fn or float8_e8m0fnu, the types of 8-bit rows")


def f8_quantize(x, codes=None, scales=None):
    """Rows x [M, K] (float32, float16 or bfloat16; weights or activations) to
    8-bit floating point with a power-of-two scale per 128: returns (codes
    float8_e4m3fn [M, K], scales float8_e8m0fnu [M, K/128]); value = code * scale."""
    if _E8 is None or _F8 is None:
        _no_f8_types()
    dt, shape, index = _rows(x, "x")
    m, k = shape
    if k % GROUP:
        raise ValueError("K must be a multiple of 128")
    groups = (m, k // GROUP)
    if codes is None:
        codes = torch.empty(shape, dtype=_F8, device=x.device)
    elif not (isinstance(codes, torch.Tensor) and codes.dtype is _F8 and codes.shape == shape and
              codes.get_device() == index and codes.is_contiguous()):
        _refuse(codes, "codes", _F8, shape, index)
    if scales is None:
        scales = torch.empty(groups, dtype=_E8, device=x.device)
    elif not (isinstance(scales, torch.Tensor) and scales.dtype is _E8 and scales.shape == groups and
              scales.get_device() == index and scales.is_contiguous()):
        _refuse(scales, "scales", _E8, groups, index)
    _call("tl_f8_quantize", index, (x.data_ptr(), m, k, dt, codes.data_ptr(), scales.data_ptr()))
    return codes, scales


def _f8_shape(codes, scales, what="codes"):
    """(rows, K, device index) of 8-bit floating point rows and their scales."""
    if not (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor)):
        raise TypeError(f"{what} and their scales must be torch.Tensors")
    if codes.dtype is not _F8 or scales.dtype is not _E8:
        if _E8 is None or _F8 is None:
            _no_f8_types()
        raise TypeError(f"{what} must be float8_e4m3fn and their scales float8_e8m0fnu")
    index = codes.get_device()
    if index < 0 or scales.get_device() != index:
        raise ValueError(f"{what} and their scales must be device tensors, on the same device")
    cs, ss = codes.shape, scales.shape
    if len(cs) != 2 or len(ss) != 2 or not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError(f"{what} and their scales must be contiguous with 2 dims")
    n, k = cs
    if ss[0] != n or k % GROUP or ss[1] * GROUP != k:
        raise ValueError(f"{what} {tuple(cs)} and their scales {tuple(ss)} must be "
                         "[rows, K] and [rows, K/128], K a multiple of 128")
    return n, k, index


def f8_dequantize(codes, scales, out_dtype=torch.float16, out=None) -> torch.Tensor:
    """The values [M, K] that 8-bit floating point rows stand for."""
    m, k, index = _f8_shape(codes, scales)
    dt = _out_type(out_dtype)
    if out is None:
        out = torch.empty((m, k), dtype=out_dtype, device=codes.device)
    elif not (isinstance(out, torch.Tensor) and out.dtype is out_dtype and out.shape == (m, k) and
              out.get_device() == index and out.is_contiguous()):
        _refuse(out, "out", out_dtype, (m, k), index)
    _call("tl_f8_dequantize", index, (codes.data_ptr(), scales.data_ptr(), m, k, out.data_ptr(), dt))
    return out


def f8_gemm_workspace_bytes(m: int, n: int, k: int) -> int:
    """Device workspace bytes tl_f8_gemm and tl_f8_gemm_approx need (0: none)."""
    b = int(lib().tl_f8_gemm_workspace_bytes(m, n, k))
    if b < 0:
        raise TLError("tl_f8_gemm_workspace_bytes", 2)
    return b


@functools.lru_cache(maxsize=4096)
def _f8_workspace(index: int, m: int, n: int, k: int) -> int:
    """f8_gemm_workspace_bytes of a shape, asked once a device."""
    with torch.cuda.device(index):
        return f8_gemm_workspace_bytes(m, n, k)


def f8_gemm(codes, scales, x, x_scales, out_dtype=torch.float32, out=None, workspace=None,
            approx=False) -> torch.Tensor:
    """y[M, N] = x . w^T with both in 8-bit floating point (``f8_quantize``):
    weights codes [N, K] and scales, activations x [M, K] and x_scales, one
    token or a prompt.  Products are exact and their sums fp32; ``approx``
    allows float16 and bfloat16 outputs sums of 14 bits in every 8 products,
    in about half the time for a prompt (tl_f8_gemm_approx).  ``workspace``
    (uint8, at least ``f8_gemm_workspace_bytes``) is taken from torch's
    allocator when not given."""
    n, k, index = _f8_shape(codes, scales)
    m, kx, at = _f8_shape(x, x_scales, "x")
    if kx != k or at != index:
        raise ValueError(f"x must be [M, {k}] on {codes.device}, got {tuple(x.shape)} on {x.device}")
    yd = _out_type(out_dtype)
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=codes.device)
    elif not (isinstance(out, torch.Tensor) and out.dtype is out_dtype and out.shape == (m, n) and
              out.get_device() == index and out.is_contiguous()):
        _refuse(out, "out", out_dtype, (m, n), index)
    wp, wb = None, 0
    if workspace is not None:
        if not (isinstance(workspace, torch.Tensor) and workspace.dtype is _U8 and workspace.dim() == 1 and
                workspace.get_device() == index and workspace.is_contiguous()):
            _refuse(workspace, "workspace", _U8, ("bytes",), index)
        wp, wb = workspace.data_ptr(), workspace.numel()
    else:
        wb = _f8_workspace(index, m, n, k)
        if wb:
            workspace = torch.empty(wb, dtype=_U8, device=codes.device)
            wp = workspace.data_ptr()
    _call("tl_f8_gemm_approx" if approx else "tl_f8_gemm", index,
          (codes.data_ptr(), scales.data_ptr(), x.data_ptr(), x_scales.data_ptr(), m, n, k, out.data_ptr(), yd, wp, wb))
    return out


class F8Linear:
    """A linear layer with weights in 8-bit floating point, for the matrices
    beside the ternary ones; ``forward`` rounds its input rows to the same form.
    ``approx`` as for ``f8_gemm``."""

    def __init__(self, codes, scales, approx=False):
        self.codes, self.scales, self.approx = codes, scales, approx

    def forward(self, x: torch.Tensor, out_dtype=torch.float32) -> torch.Tensor:
        return f8_gemm(self.codes, self.scales, *f8_quantize(x), out_dtype, approx=self.approx)

    __call__ = forward


def _lookup(call, n, k, index, head, ids, factor, out_dtype, out, device):
    dt = _out_type(out_dtype)
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    m = ids.numel()
    if ids.dtype is not _I32 or ids.dim() != 1 or ids.get_device() != index or not ids.is_contiguous():
        _refuse(ids, "ids", _I32, ("M",), index)
    if out is None:
        out = torch.empty((m, k), dtype=out_dtype, device=device)
    elif not (isinstance(out, torch.Tensor) and out.dtype is out_dtype and out.shape == (m, k) and
              out.get_device() == index and out.is_contiguous()):
        _refuse(out, "out", out_dtype, (m, k), index)
    _call(call, index, (*head, ids.data_ptr(), m, n, k, factor, out.data_ptr(), dt))
    return out


def q4_rows(packed, scales, ids, factor=1.0, out_dtype=torch.float16, out=None) -> torch.Tensor:
    """Embedding lookup in a table of 4-bit weights (``q4_quantize`` without
    signs): row ids[m] times ``factor`` for each of ids (int32 [M]), zeros for an
    id outside the table."""
    n, k, group, index = _q4_shape(packed, scales)
    return _lookup("tl_q4_rows", n, k, index, (packed.data_ptr(), scales.data_ptr(), group), ids, factor, out_dtype,
                   out, packed.device)


def f8_rows(codes, scales, ids, factor=1.0, out_dtype=torch.float16, out=None) -> torch.Tensor:
    """``q4_rows`` in a table of 8-bit floating point (``f8_quantize``)."""
    n, k, index = _f8_shape(codes, scales)
    return _lookup("tl_f8_rows", n, k, index, (codes.data_ptr(), scales.data_ptr()), ids, factor, out_dtype, out,
                   codes.device)


def adjust_logits(logits, history=None, history_lens=None, prompt_lens=None, repetition=None, presence=None,
                  frequency=None, bias_ids=None, bias_values=None, mask=None, out_dtype=None, out=None):
    """Penalties for repeated tokens, biases and a grammar's mask on logits [M, V]
    (float32, float16 or bfloat16), in this order (see tl_adjust_logits):
    history int32 [M, H], of which a row's first ``history_lens`` ids count and
    its first ``prompt_lens`` are the prompt's (int32 [M]); repetition, presence
    and frequency float32 [M]; bias_ids int32 and bias_values float32 [M, B], the
    last entry of a token counts; mask int32 [M, ceil(V/32)], bit 1 = allowed.
    Ids outside the vocabulary are padding.  ``out`` may be logits itself."""
    dt, shape, index = _rows(logits, "logits")
    m, v = shape
    if out_dtype is None:
        out_dtype, od = logits.dtype, dt
    else:
        od = _out_type(out_dtype)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=logits.device)
    elif not (isinstance(out, torch.Tensor) and out.dtype is out_dtype and out.shape == shape and
              out.get_device() == index and out.is_contiguous()):
        _refuse(out, "out", out_dtype, shape, index)
    h = b = 0
    hp = lp = pp = rp = ep = fp = ip = vp = mp = None
    if history is not None:
        if not (isinstance(history, torch.Tensor) and history.dtype is _I32 and history.dim() == 2 and
                history.shape[0] == m and history.get_device() == index and history.is_contiguous()):
            _refuse(history, "history", _I32, (m, "H"), index)
        h = history.shape[1]
        row = (m,)
        if history_lens is not None:
            if not (isinstance(history_lens, torch.Tensor) and history_lens.dtype is _I32 and
                    history_lens.shape == row and history_lens.get_device() == index and
                    history_lens.is_contiguous()):
                _refuse(history_lens, "history_lens", _I32, row, index)
            lp = history_lens.data_ptr()
        if prompt_lens is not None:
            if not (isinstance(prompt_lens, torch.Tensor) and prompt_lens.dtype is _I32 and
                    prompt_lens.shape == row and prompt_lens.get_device() == index and
                    prompt_lens.is_contiguous()):
                _refuse(prompt_lens, "prompt_lens", _I32, row, index)
            pp = prompt_lens.data_ptr()
        if repetition is not None:
            if not (isinstance(repetition, torch.Tensor) and repetition.dtype is _F32 and
                    repetition.shape == row and repetition.get_device() == index and
                    repetition.is_contiguous()):
                _refuse(repetition, "repetition", _F32, row, index)
            rp = repetition.data_ptr()
        if presence is not None:
            if not (isinstance(presence, torch.Tensor) and presence.dtype is _F32 and presence.shape == row and
                    presence.get_device() == index and presence.is_contiguous()):
                _refuse(presence, "presence", _F32, row, index)
            ep = presence.data_ptr()
        if frequency is not None:
            if not (isinstance(frequency, torch.Tensor) and frequency.dtype is _F32 and frequency.shape == row and
                    frequency.get_device() == index and frequency.is_contiguous()):
                _refuse(frequency, "frequency", _F32, row, index)
            fp = frequency.data_ptr()
        if h:
            hp = history.data_ptr()
        else:       # (an empty history has no address, and nothing to penalise)
            lp = pp = rp = ep = fp = None
    elif not (history_lens is prompt_lens is repetition is presence is frequency is None):
        raise ValueError("history_lens, prompt_lens and penalties need a history")
    if bias_ids is not None or bias_values is not None:
        if not (isinstance(bias_ids, torch.Tensor) and bias_ids.dtype is _I32 and bias_ids.dim() == 2 and
                bias_ids.shape[0] == m and bias_ids.get_device() == index and bias_ids.is_contiguous()):
            _refuse(bias_ids, "bias_ids", _I32, (m, "B"), index)
        if not (isinstance(bias_values, torch.Tensor) and bias_values.dtype is _F32 and
                bias_values.shape == bias_ids.shape and bias_values.get_device() == index and
                bias_values.is_contiguous()):
            _refuse(bias_values, "bias_values", _F32, bias_ids.shape, index)
        b = bias_ids.shape[1]
        if b:
            ip, vp = bias_ids.data_ptr(), bias_values.data_ptr()
    if mask is not None:
        words = (m, (v + 31) // 32)
        if not (isinstance(mask, torch.Tensor) and mask.dtype is _I32 and mask.shape == words and
                mask.get_device() == index and mask.is_contiguous()):
            _refuse(mask, "mask", _I32, words, index)
        mp = mask.data_ptr()
    _call("tl_adjust_logits", index, (logits.data_ptr(), m, v, dt, hp, h, lp, pp, rp, ep, fp, ip, vp, b, mp,
                                      out.data_ptr(), od))
    return out


class TernaryLinear:
    """A ternary g128 linear layer whose weights carry the folded rotation.

    ``forward`` always rotates its input first: skipping the runtime rotation
    gives wrong output without any error (page "A 27-billion model that fits
    in 8.6 GB", paragraph 3), so it is not optional here."""

    def __init__(self, packed, scales, fmt, signs, prefill_threshold: int = 64):
        self.packed, self.scales, self.fmt, self.signs = packed, scales, fmt, signs
        self.prefill_threshold = prefill_threshold

    def forward(self, x: torch.Tensor, out_dtype=torch.float32) -> torch.Tensor:
        if x.shape[0] >= self.prefill_threshold:
            return gemm(self.packed, self.scales, self.fmt, hadamard_rotate(x, self.signs),
                        out_dtype)
        return linear(self.packed, self.scales, self.fmt, x, self.signs, out_dtype)

    __call__ = forward


class ChainOp(ctypes.Structure):
    """tl_chain_op of include/tl.h."""
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("signs", ctypes.c_void_p), ("x_rot", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("fmt", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32)]


class Chain:
    """A decode chain (tl_linear_chain): linears at M = 1 run in order in one
    launch, each the rotation of its input and the ternary product, with the
    next linear's weights requested before the current one ends.  ``ops``:
    dicts with packed, scales, fmt, x, signs, y and optionally x_rot (device
    tensors; x [1, K] or [K] binary16, y [1, N] or [N] float32/float16).  An
    x that is a view into the binary16 y of an earlier op makes that op wait
    for it.  The plan is encoded once (on the host, by the library) and kept
    on the device with the sync buffer; the tensors must stay alive."""

    def __init__(self, ops):
        if not ops:
            raise ValueError("a chain needs at least one linear")
        count = len(ops)
        arr = (ChainOp * count)()
        for i, o in enumerate(ops):
            _need(o["packed"], "packed", torch.uint8, 2)
            _need(o["scales"], "scales", torch.float16, 2)
            _need(o["x"], "x", torch.float16)
            _need(o["signs"], "signs", torch.int8, 1)
            n, k = o["packed"].shape[0], o["x"].numel()
            y = o["y"]
            if y.dtype not in (torch.float32, torch.float16) or y.numel() != n or not y.is_contiguous():
                raise ValueError("y must be a contiguous float32/float16 tensor of N elements")
            if o["signs"].numel() != k or o["scales"].shape != (n, k // GROUP):
                raise ValueError("signs must have K entries and scales be [N, K/128]")
            if o["packed"].numel() != packed_bytes(n, k, o["fmt"]):
                raise ValueError("packed size does not match N, K and the format")
            xr = o.get("x_rot")
            if xr is not None:
                _need(xr, "x_rot", torch.float16)
            arr[i] = ChainOp(o["packed"].data_ptr(), o["scales"].data_ptr(), o["x"].data_ptr(),
                             o["signs"].data_ptr(), 0 if xr is None else xr.data_ptr(),
                             y.data_ptr(), n, k, o["fmt"],
                             TL_F32 if y.dtype == torch.float32 else TL_F16)
        L = lib()
        nbytes = int(L.tl_chain_plan_bytes(count))
        host = (ctypes.c_uint8 * nbytes)()
        _check("tl_chain_encode", L.tl_chain_encode(arr, count, host, nbytes))
        device = ops[0]["x"].device
        self.count = count
        self.plan = torch.frombuffer(bytearray(host), dtype=torch.uint8).to(device)
        self.sync = torch.zeros(int(L.tl_chain_sync_bytes(count)) // 4, dtype=torch.int32,
                                device=device)
        self._ops = ops

    def __call__(self) -> None:
        _check("tl_linear_chain", lib().tl_linear_chain(_ptr(self.plan), self.count,
                                                        _ptr(self.sync), _stream(self.sync)))

    def error(self) -> int:
        """The chain's error word (0: none; see tl_linear_chain)."""
        return int(self.sync[self.count + 1].item())

    def clear_error(self) -> None:
        self.sync[self.count + 1].zero_()
