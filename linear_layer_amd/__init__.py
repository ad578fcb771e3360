"""Python binding of the MI355X GEMM / fully-connected C-ABI library.

Argument marshalling only: shape, dtype and layout checks, then the tensors'
device pointers and the current HIP stream go to ``liblinear_layer.so``,
whose HIP kernels do all of the arithmetic. There is no fallback: if the
library is missing, importing the functions raises.

Entry points (same names as the C ABI in ``include/linear_layer.h``):

* ``gemm_f32(A, B, C, alpha=1.0, beta=0.0)`` — C = alpha*A*B + beta*C, fp32.
* ``gemm_f16f32(A, B, C, alpha=1.0, beta=0.0)`` — fp16 A, B; fp32 C.
* ``gemm_bf16f32(A, B, C, alpha=1.0, beta=0.0)`` — bf16 A, B; fp32 C.
* ``linear_bias_act(X, W, bias, act, Y)`` — Y = act(X*W + bias), fp32.
* ``gemm_f32_nt``, ``gemm_f16f32_nt``, ``gemm_bf16f32_nt``, ``linear_bias_act_nt``
  — the same with B (W) given N-by-K: C = alpha*A*B^T + beta*C, Y = act(X*W^T + b)
  (W in the [out_features, in_features] layout of ``torch.nn.Linear.weight``).
* ``linear_bias_act_ws(X, W, bias, act, Y, workspace, w_trans=False)`` — the fused
  layer with a caller workspace (``linear_workspace_size``): stream-K shapes in one
  launch with bias and ReLU in every tile's write-back.
* ``linear_bias_act_noalloc(X, W, bias, act, Y, w_trans=False)`` — the same on the
  library's static per-GPU workspace, for callers that cannot allocate.
* ``gemm_f32_batched``, ``gemm_f16f32_batched``, ``gemm_bf16f32_batched``
  ``(A, B, C, alpha=1.0, beta=0.0, trans_b=False)`` — C[i] = alpha*A[i]*op(B[i])
  + beta*C[i] over 3-D tensors whose first axis is the batch; its stride is the
  batch stride (0, e.g. from ``expand``, shares one matrix among all items).
* ``mx4_quantize(X, codes, scales, trans=False)``, ``mx4_dequantize(codes, scales, Y)``
  — microscaled 4-bit floating point (blocks of 32 values along a row, two 4-bit
  codes a byte, one scale byte a block; ``mx4_shapes`` gives the tensors' shapes).
* ``gemm_mx4f32_nt(A, SA, B, SB, C, alpha=1.0, beta=0.0, K=None)`` — C = alpha*A*B^T
  + beta*C, both operands in that format; ``gemm_f16mx4f32_nt`` and
  ``gemm_bf16mx4f32_nt(A, B, SB, C, alpha=1.0, beta=0.0)`` — the same with 16-bit A.
  On the current stream, a product whose K is worth sharing out over workgroups takes
  its workspace from torch's allocator; with ``stream`` given it runs without one.
  ``mx4_chosen_kernel`` names the kernel that such a product takes.
* ``rmsnorm_residual(Y, w_post, gate, alpha, X, w_pre, XO, H, eps=1e-5)`` — the residual
  step between two blocks: XO = X + alpha*gate*rms(Y)*w_post, H = rms(XO)*w_pre;
  ``rmsnorm_residual_grad`` — its gradient (``rmsnorm_grad_workspace_size`` bytes of
  workspace).
* ``linear16_nt(X, W, bias, act, R, Y, Z=None, offsets=None)`` — Y = act(X*W^T + bias) + R
  in float16 or bfloat16 with fp32 sums (Y and R in that type or fp32); Z keeps the
  activation's input for the way back, in 16 bits or as (codes, scales) in 8.
  With ``offsets`` (int32, groups + 1 row numbers on the device) the rows are those of
  experts and W, bias are stacks, one for each.
* ``linear16_grad_act(DY, Z, act, DZ, dbias=None, offsets=None)``,
  ``linear16_grad_input(DZ, W, DX, offsets=None)``,
  ``linear16_grad_weight(DZ, X, DW, beta=0.0, offsets=None)`` — its gradients: DZ = DY *
  act'(Z) and its sums, DX = DZ*W, DW = DZ^T*X + beta*DW, Z and X in 16 or in 8 bits.
* ``mx8_quantize(X, codes, scales)``, ``mx8_dequantize(codes, scales, Y)`` — microscaled
  8-bit floating point (a byte a value, a scale byte a block of 32; ``mx8_shapes``).

Matrices are 2-D, row-major with unit column stride (a row stride larger than
the width is a leading dimension), on the current CUDA/HIP device. The calls
are asynchronous on ``torch.cuda.current_stream()`` unless ``stream`` is given.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "LinearLayerError", "gemm_f32", "gemm_f16f32", "gemm_bf16f32", "linear_bias_act", "status_string",
    "gemm_f32_nt", "gemm_f16f32_nt", "gemm_bf16f32_nt", "linear_bias_act_nt",
    "gemm_f32_batched", "gemm_f16f32_batched", "gemm_bf16f32_batched",
    "linear_bias_act_ws", "linear_workspace_size", "linear_bias_act_noalloc", "NOALLOC_SCRATCH_BYTES",
    "set_noalloc_limit",
    "mx4_quantize", "mx4_dequantize", "mx4_shapes", "gemm_mx4f32_nt", "gemm_f16mx4f32_nt", "gemm_bf16mx4f32_nt",
    "mx4_chosen_kernel", "A_MX4", "A_F16", "A_BF16", "rmsnorm_residual", "rmsnorm_residual_grad", "rmsnorm_grad_workspace_size",
    "TYPE_F32", "TYPE_F16", "TYPE_BF16",
    "mx8_quantize", "mx8_dequantize", "mx8_shapes", "linear16_nt", "linear16_grad_act", "linear16_grad_input",
    "linear16_grad_weight", "linear16_grad_act_workspace_size", "linear16_workspace_size",
    "linear16_chosen_kernel", "L16_FORWARD", "L16_GRAD_INPUT", "L16_GRAD_WEIGHT", "ACT_GELU", "ACT_GELU_TANH", "ACT_SILU", "MAX_GROUPS",
    "library_path", "load", "set_tile", "num_tiles", "tile_name", "chosen_tile",
    "set_split_k", "chosen_split_k", "set_stream_k", "chosen_stream_k",
    "ACT_NONE", "ACT_RELU", "DTYPE_F32", "DTYPE_F16", "PLAN_RELU", "PLAN_B_NK", "PLAN_UNALIGNED",
    "OK", "ERR_INVALID_VALUE", "ERR_NO_DEVICE", "ERR_UNSUPPORTED_ARCH", "ERR_LAUNCH",
]

OK, ERR_INVALID_VALUE, ERR_NO_DEVICE, ERR_UNSUPPORTED_ARCH, ERR_LAUNCH = 0, 1, 2, 3, 4
ACT_NONE, ACT_RELU = 0, 1
ACT_GELU, ACT_GELU_TANH, ACT_SILU = 2, 3, 4   # of linear16_nt and linear16_grad_act
MAX_GROUPS = 1 << 20   # of rows, in the linear16 calls
L16_FORWARD, L16_GRAD_INPUT, L16_GRAD_WEIGHT = 0, 1, 2   # products of linear16_chosen_kernel
DTYPE_F32, DTYPE_F16 = 0, 1
TYPE_F32, TYPE_F16, TYPE_BF16 = 0, 1, 2   # element types of the microscaled formats, the norms and the 16-bit layer
A_MX4, A_F16, A_BF16 = 0, 1, 2   # the forms of A of the 4-bit products
PLAN_RELU, PLAN_B_NK, PLAN_UNALIGNED = 0x100, 0x200, 0x400   # flags OR-ed into dtype for chosen_*
NOALLOC_SCRATCH_BYTES = 65 << 20   # the static workspace of linear_bias_act_noalloc

_HERE = os.path.dirname(os.path.abspath(__file__))
# The in-package library, or another build of it named by LINEAR_LAYER_LIBRARY
# (the CPU sanitizer test loads an AddressSanitizer build of the host code
# that way). Either way the file must exist: there is no fallback.
_DEFAULT_LIB_PATH = os.path.join(_HERE, "liblinear_layer.so")
_LIB_PATH = os.environ.get("LINEAR_LAYER_LIBRARY") or _DEFAULT_LIB_PATH
_lib = None

# Every symbol the C header declares.
EXPORTED = ("gemm_f32", "gemm_f16f32", "gemm_bf16f32", "linear_bias_act", "ll_status_string",
            "gemm_f32_nt", "gemm_f16f32_nt", "gemm_bf16f32_nt", "linear_bias_act_nt",
            "gemm_f32_batched", "gemm_f16f32_batched", "gemm_bf16f32_batched",
            "ll_num_tiles", "ll_tile_name", "ll_set_tile", "ll_chosen_tile",
            "ll_set_split_k", "ll_chosen_split_k", "ll_set_stream_k", "ll_chosen_stream_k",
            "linear_bias_act_ws", "ll_linear_workspace_size", "linear_bias_act_noalloc",
            "ll_set_noalloc_limit",
            "mx4_quantize", "mx4_dequantize", "gemm_mx4f32_nt", "gemm_f16mx4f32_nt", "gemm_bf16mx4f32_nt",
            "gemm_mx4f32_nt_ws", "gemm_f16mx4f32_nt_ws", "gemm_bf16mx4f32_nt_ws", "ll_mx4_workspace_size",
            "ll_mx4_chosen_kernel",
            "rmsnorm_residual", "rmsnorm_residual_grad", "ll_rmsnorm_grad_workspace_size",
            "mx8_quantize", "mx8_dequantize", "linear16_nt", "linear16_grad_act", "linear16_grad_input",
            "linear16_grad_weight", "ll_linear16_grad_act_workspace_size", "ll_linear16_workspace_size",
            "ll_linear16_chosen_kernel")


class LinearLayerError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load liblinear_layer.so (built in-tree by ``python -m linear_layer_amd._build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with `python -m linear_layer_amd._build`")
    lib = ctypes.CDLL(_LIB_PATH)
    i32, f32, vp = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
    lib.gemm_f32.argtypes = [i32, i32, i32, f32, vp, i32, vp, i32, f32, vp, i32, vp]
    lib.gemm_f16f32.argtypes = lib.gemm_f32.argtypes
    lib.gemm_bf16f32.argtypes = lib.gemm_f32.argtypes
    lib.linear_bias_act.argtypes = [i32, i32, i32, vp, i32, vp, i32, vp, i32, vp, i32, vp]
    lib.linear_bias_act_ws.argtypes = [i32, i32, i32, vp, i32, vp, i32, i32, vp, i32, vp, i32, vp,
                                       ctypes.c_int64, vp]
    lib.linear_bias_act_ws.restype = i32
    lib.linear_bias_act_noalloc.argtypes = [i32, i32, i32, vp, i32, vp, i32, i32, vp, i32, vp, i32, vp]
    lib.linear_bias_act_noalloc.restype = i32
    lib.ll_set_noalloc_limit.argtypes = [ctypes.c_int64]
    lib.ll_set_noalloc_limit.restype = i32
    lib.ll_linear_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.ll_linear_workspace_size.restype = ctypes.c_int64
    for nt in ("gemm_f32_nt", "gemm_f16f32_nt", "gemm_bf16f32_nt"):
        getattr(lib, nt).argtypes = lib.gemm_f32.argtypes
    lib.linear_bias_act_nt.argtypes = lib.linear_bias_act.argtypes
    i64 = ctypes.c_int64
    for b in ("gemm_f32_batched", "gemm_f16f32_batched", "gemm_bf16f32_batched"):
        getattr(lib, b).argtypes = [i32, i32, i32, i32, f32, vp, i32, i64, vp, i32, i64,
                                    f32, vp, i32, i64, i32, vp]
    for f in (lib.gemm_f32, lib.gemm_f16f32, lib.gemm_bf16f32, lib.linear_bias_act,
              lib.gemm_f32_nt, lib.gemm_f16f32_nt, lib.gemm_bf16f32_nt, lib.linear_bias_act_nt,
              lib.gemm_f32_batched, lib.gemm_f16f32_batched, lib.gemm_bf16f32_batched):
        f.restype = i32
    lib.mx4_quantize.argtypes = [i32, i32, i32, vp, i32, i32, vp, i32, vp, i32, vp]
    lib.mx4_dequantize.argtypes = [i32, i32, vp, i32, vp, i32, i32, vp, i32, vp]
    lib.gemm_mx4f32_nt.argtypes = [i32, i32, i32, f32, vp, i32, vp, i32, vp, i32, vp, i32, f32, vp, i32, vp]
    lib.gemm_f16mx4f32_nt.argtypes = [i32, i32, i32, f32, vp, i32, vp, i32, vp, i32, f32, vp, i32, vp]
    lib.gemm_bf16mx4f32_nt.argtypes = lib.gemm_f16mx4f32_nt.argtypes
    lib.gemm_mx4f32_nt_ws.argtypes = lib.gemm_mx4f32_nt.argtypes[:-1] + [vp, i64, vp]
    lib.gemm_f16mx4f32_nt_ws.argtypes = lib.gemm_f16mx4f32_nt.argtypes[:-1] + [vp, i64, vp]
    lib.gemm_bf16mx4f32_nt_ws.argtypes = lib.gemm_f16mx4f32_nt_ws.argtypes
    lib.ll_mx4_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.ll_mx4_workspace_size.restype = i64
    lib.ll_mx4_chosen_kernel.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.ll_mx4_chosen_kernel.restype = ctypes.c_char_p
    lib.rmsnorm_residual.argtypes = [i32, i32, i32, vp, i32, vp, vp, f32, vp, i32, vp, f32, vp, i32, vp, i32, vp]
    lib.rmsnorm_residual_grad.argtypes = [i32, i32, i32, vp, i32, vp, i32, vp, i32, vp, vp, f32, vp, i32, vp, f32,
                                          vp, i32, vp, i32, vp, vp, vp, vp, i64, vp]
    lib.rmsnorm_residual.restype = lib.rmsnorm_residual_grad.restype = i32
    lib.mx8_quantize.argtypes = [i32, i32, i32, vp, i32, vp, i32, vp, i32, vp]
    lib.mx8_dequantize.argtypes = [i32, i32, vp, i32, vp, i32, i32, vp, i32, vp]
    lib.linear16_nt.argtypes = [i32, i32, i32, i32, vp, i32, i32, vp, vp, i32, i64, vp, i32, i32, vp, i32, vp, i32,
                                vp, i32, vp, i32, vp, i32, vp, i64, vp]
    lib.ll_linear16_chosen_kernel.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.ll_linear16_chosen_kernel.restype = ctypes.c_char_p
    lib.ll_linear16_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.ll_linear16_workspace_size.restype = i64
    lib.linear16_grad_act.argtypes = [i32, i32, i32, i32, i32, vp, i32, i32, vp, vp, i32, vp, i32, vp, i32, vp, i32, vp,
                                      vp, i64, vp]
    lib.linear16_grad_input.argtypes = [i32, i32, i32, i32, vp, i32, i32, vp, vp, i32, i64, i32, vp, i32, vp, i64, vp]
    lib.linear16_grad_weight.argtypes = [i32, i32, i32, i32, vp, i32, i32, vp, vp, i32, vp, i32, vp, i32, i32, f32, vp,
                                         i32, i64, vp]
    for f in (lib.mx8_quantize, lib.mx8_dequantize, lib.linear16_nt, lib.linear16_grad_act, lib.linear16_grad_input,
              lib.linear16_grad_weight):
        f.restype = i32
    lib.ll_linear16_grad_act_workspace_size.argtypes = [i32, i32, i32]
    lib.ll_linear16_grad_act_workspace_size.restype = i64
    lib.ll_rmsnorm_grad_workspace_size.argtypes = [i32, i32]
    lib.ll_rmsnorm_grad_workspace_size.restype = i64
    for f in (lib.mx4_quantize, lib.mx4_dequantize, lib.gemm_mx4f32_nt, lib.gemm_f16mx4f32_nt,
              lib.gemm_bf16mx4f32_nt, lib.gemm_mx4f32_nt_ws, lib.gemm_f16mx4f32_nt_ws, lib.gemm_bf16mx4f32_nt_ws):
        f.restype = i32
    lib.ll_status_string.argtypes = [i32]
    lib.ll_status_string.restype = ctypes.c_char_p
    lib.ll_num_tiles.argtypes = [i32]
    lib.ll_num_tiles.restype = i32
    lib.ll_tile_name.argtypes = [i32, i32]
    lib.ll_tile_name.restype = ctypes.c_char_p
    lib.ll_set_tile.argtypes = [i32, i32]
    lib.ll_set_tile.restype = i32
    lib.ll_chosen_tile.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.ll_chosen_tile.restype = i32
    lib.ll_chosen_split_k.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.ll_chosen_split_k.restype = i32
    lib.ll_set_split_k.argtypes = [i32]
    lib.ll_set_split_k.restype = i32
    lib.ll_set_stream_k.argtypes = [i32]
    lib.ll_set_stream_k.restype = i32
    lib.ll_chosen_stream_k.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.ll_chosen_stream_k.restype = i32
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().ll_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != OK:
        raise LinearLayerError(status, where)


def set_tile(dtype: int, tile: int) -> None:
    """Force a tile shape for later calls of that dtype; -1 = automatic.

    Like set_split_k and set_stream_k, a process-wide override for benchmarks
    and tests (include/linear_layer_tuning.h): it steers every later call from
    every thread and on every stream until reset."""
    _check(load().ll_set_tile(int(dtype), int(tile)), "ll_set_tile")


def num_tiles(dtype: int) -> int:
    return load().ll_num_tiles(int(dtype))


def tile_name(dtype: int, tile: int) -> str:
    return load().ll_tile_name(int(dtype), int(tile)).decode()


def chosen_tile(dtype: int, M: int, N: int, K: int, num_cus: int = 0, batch: int = 1) -> int:
    return load().ll_chosen_tile(int(dtype), int(M), int(N), int(K), int(batch), int(num_cus))


def set_split_k(splits: int) -> None:
    """Force the number of K-splits (1..16) for later calls; -1 = automatic.
    Process-wide, like set_tile."""
    _check(load().ll_set_split_k(int(splits)), "ll_set_split_k")


def chosen_split_k(dtype: int, M: int, N: int, K: int, num_cus: int = 0, batch: int = 1) -> int:
    return load().ll_chosen_split_k(int(dtype), int(M), int(N), int(K), int(batch), int(num_cus))


def set_stream_k(mode: int) -> None:
    """Stream-K for leftover tiles: -1 automatic, 0 never, 1 whenever possible.
    Process-wide, like set_tile."""
    _check(load().ll_set_stream_k(int(mode)), "ll_set_stream_k")


def chosen_stream_k(dtype: int, M: int, N: int, K: int, num_cus: int = 0, batch: int = 1) -> int:
    """Number of tiles the plan shares out with stream-K (0: none)."""
    return load().ll_chosen_stream_k(int(dtype), int(M), int(N), int(K), int(batch), int(num_cus))


# ---- tensor marshalling ---------------------------------------------------

_torch_module = None
_INT_MAX = 2 ** 31 - 1   # of the C calls' sizes and leading dimensions


def _torch():
    global _torch_module
    if _torch_module is None:   # (an import statement costs a few tenths of a microsecond a call)
        import torch
        _torch_module = torch
    return _torch_module


def _mat(t, dtype, name):
    """(pointer, rows, cols, ld) of a 2-D row-major device tensor."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    rows, cols = shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"{name}: row stride {ld} smaller than width {cols}")
    if ld > _INT_MAX or rows > _INT_MAX:   # (ctypes would pass on the lower 32 bits)
        raise ValueError(f"{name}: {rows} rows of {cols} values, {ld} apart: the calls take sizes up to {_INT_MAX}")
    return t.data_ptr(), rows, cols, ld if ld > 1 else 1


def _bmat(t, dtype, name):
    """(pointer, batch, rows, cols, ld, batch stride) of a 3-D tensor of row-major matrices."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D (batch, rows, cols), got shape {tuple(t.shape)}")
    nb = t.shape[0]
    if nb == 0:
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        return 0, 0, t.shape[1], t.shape[2], max(t.shape[2], 1), 0
    if nb > _INT_MAX:
        raise ValueError(f"{name}: the calls take sizes up to {_INT_MAX}")
    ptr, rows, cols, ld = _mat(t[0], dtype, name)
    bstride = t.stride(0) if nb > 1 else 0
    if bstride < 0:
        raise ValueError(f"{name}: negative batch stride")
    return t.data_ptr(), nb, rows, cols, ld, bstride


def _gemm_batched(fn_name, in_dtype, A, B, C, alpha, beta, trans_b, stream):
    torch = _torch()
    pa, nb, M, K, lda, sa = _bmat(A, in_dtype, "A")
    if trans_b:
        pb, nb2, N, K2, ldb, sb = _bmat(B, in_dtype, "B")
    else:
        pb, nb2, K2, N, ldb, sb = _bmat(B, in_dtype, "B")
    pc, nb3, M2, N2, ldc, sc = _bmat(C, torch.float32, "C")
    if nb2 != nb or nb3 != nb or K2 != K or M2 != M or N2 != N:
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)}")
    if nb == 0:
        return C
    st = getattr(load(), fn_name)(int(bool(trans_b)), M, N, K, float(alpha), pa, lda, sa, pb, ldb, sb,
                                  float(beta), pc, ldc, sc, nb, _stream(stream, A, B, C))
    _check(st, fn_name)
    return C


def gemm_f32_batched(A, B, C, alpha: float = 1.0, beta: float = 0.0, trans_b: bool = False,
                     stream=None):
    """C[i] = alpha*A[i]*op(B[i]) + beta*C[i], fp32; op(B) = B^T when trans_b."""
    return _gemm_batched("gemm_f32_batched", _torch().float32, A, B, C, alpha, beta, trans_b, stream)


def gemm_f16f32_batched(A, B, C, alpha: float = 1.0, beta: float = 0.0, trans_b: bool = False,
                        stream=None):
    """Batched product with fp16 A, B and fp32 C."""
    return _gemm_batched("gemm_f16f32_batched", _torch().float16, A, B, C, alpha, beta, trans_b, stream)


def gemm_bf16f32_batched(A, B, C, alpha: float = 1.0, beta: float = 0.0, trans_b: bool = False,
                         stream=None):
    """Batched product with bf16 A, B and fp32 C."""
    return _gemm_batched("gemm_bf16f32_batched", _torch().bfloat16, A, B, C, alpha, beta, trans_b,
                         stream)


_RAW = None


def _raw_getters():
    """(current device index, raw current stream of a device): torch's direct
    getters when it has them (no Stream object per call), else the public API."""
    global _RAW
    if _RAW is None:
        torch = _torch()
        get_dev = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        get_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if get_raw is None:
            def get_raw(index):
                return torch.cuda.current_stream(index).cuda_stream
        _RAW = (get_dev, get_raw)
    return _RAW


def _stream(stream, *tensors):
    if stream is None:
        dev = tensors[0].get_device()
        for t in tensors:
            if t is not None and t.get_device() != dev:
                raise ValueError("all tensors must be on the same device")
        get_dev, get_raw = _raw_getters()
        if get_dev() != dev:
            raise ValueError(f"tensors are on {tensors[0].device}, but the current device is cuda:{get_dev()}")
        return get_raw(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _gemm(fn_name, in_dtype, A, B, C, alpha, beta, stream, bt=False):
    torch = _torch()
    pa, M, K, lda = _mat(A, in_dtype, "A")
    if bt:
        pb, N, K2, ldb = _mat(B, in_dtype, "B")
    else:
        pb, K2, N, ldb = _mat(B, in_dtype, "B")
    pc, M2, N2, ldc = _mat(C, torch.float32, "C")
    if K2 != K or M2 != M or N2 != N:
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)}")
    st = getattr(load(), fn_name)(M, N, K, float(alpha), pa, lda, pb, ldb, float(beta), pc, ldc,
                                  _stream(stream, A, B, C))
    _check(st, fn_name)
    return C


def gemm_f32(A, B, C, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """C = alpha*A*B + beta*C (fp32); C is written in place and returned."""
    return _gemm("gemm_f32", _torch().float32, A, B, C, alpha, beta, stream)


def gemm_f16f32(A, B, C, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """C = alpha*A*B + beta*C with fp16 A, B and fp32 C; C returned."""
    return _gemm("gemm_f16f32", _torch().float16, A, B, C, alpha, beta, stream)


def gemm_bf16f32(A, B, C, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """C = alpha*A*B + beta*C with bf16 A, B and fp32 C; C returned."""
    return _gemm("gemm_bf16f32", _torch().bfloat16, A, B, C, alpha, beta, stream)


def gemm_f32_nt(A, B, C, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """C = alpha*A*B^T + beta*C (fp32) with B given N-by-K; C returned."""
    return _gemm("gemm_f32_nt", _torch().float32, A, B, C, alpha, beta, stream, bt=True)


def gemm_f16f32_nt(A, B, C, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """C = alpha*A*B^T + beta*C with fp16 A, B (B N-by-K) and fp32 C."""
    return _gemm("gemm_f16f32_nt", _torch().float16, A, B, C, alpha, beta, stream, bt=True)


def gemm_bf16f32_nt(A, B, C, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """C = alpha*A*B^T + beta*C with bf16 A, B (B N-by-K) and fp32 C."""
    return _gemm("gemm_bf16f32_nt", _torch().bfloat16, A, B, C, alpha, beta, stream, bt=True)


def linear_bias_act_nt(X, W, bias, act: int, Y, stream=None):
    """Y = act(X*W^T + bias) (fp32; W is N-by-K, e.g. a torch Linear weight)."""
    return _linear("linear_bias_act_nt", X, W, bias, act, Y, stream, wt=True)


def linear_bias_act(X, W, bias, act: int, Y, stream=None):
    """Y = act(X*W + bias) (fp32; W is K-by-N row-major; bias may be None)."""
    return _linear("linear_bias_act", X, W, bias, act, Y, stream)


def linear_workspace_size(M: int, N: int, K: int, w_trans: bool = False, act: int = ACT_RELU,
                          num_cus: int = 0) -> int:
    """Bytes of workspace linear_bias_act_ws uses for this shape (0: none)."""
    n = load().ll_linear_workspace_size(int(M), int(N), int(K), int(bool(w_trans)), int(act),
                                        int(num_cus))
    if n < 0:
        raise ValueError("invalid shape, layout or activation")
    return n


def linear_bias_act_ws(X, W, bias, act: int, Y, workspace, w_trans: bool = False, stream=None):
    """Y = act(X*W + bias) (or X*W^T with w_trans) with a workspace tensor (zero-filled
    before its first use; the call leaves it zero-filled), so the epilogue stays
    fused into every tile of a stream-K plan. ``workspace`` may be None."""
    torch = _torch()
    pws, nws = None, 0
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous device tensor")
        pws, nws = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    return _linear("linear_bias_act_ws", X, W, bias, act, Y, stream, wt=w_trans, ws=(pws, nws))


def set_noalloc_limit(nbytes: int) -> None:
    """Lower the workspace linear_bias_act_noalloc may use (process-wide;
    -1 restores the full static array). For tests of its refusal."""
    _check(load().ll_set_noalloc_limit(int(nbytes)), "ll_set_noalloc_limit")


def linear_bias_act_noalloc(X, W, bias, act: int, Y, w_trans: bool = False, stream=None):
    """linear_bias_act_ws on the library's own static workspace (nothing is
    allocated); calls that overlap in time on one GPU race."""
    return _linear("linear_bias_act_noalloc", X, W, bias, act, Y, stream, wt=w_trans, ws="static")


def _linear(fn_name, X, W, bias, act, Y, stream, wt=False, ws=None):
    torch = _torch()
    px, M, K, ldx = _mat(X, torch.float32, "X")
    if wt:
        pw, N, K2, ldw = _mat(W, torch.float32, "W")
    else:
        pw, K2, N, ldw = _mat(W, torch.float32, "W")
    py, M2, N2, ldy = _mat(Y, torch.float32, "Y")
    if K2 != K or M2 != M or N2 != N:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, Y {tuple(Y.shape)}")
    pbias = None
    if bias is not None:
        if bias.dtype != torch.float32 or bias.dim() != 1 or bias.shape[0] != N or not bias.is_cuda:
            raise ValueError("bias must be a 1-D fp32 device tensor of length N")
        if N > 1 and bias.stride(0) != 1:
            raise ValueError("bias must be contiguous")
        pbias = bias.data_ptr()
    if ws == "static":
        st = getattr(load(), fn_name)(M, N, K, px, ldx, pw, ldw, int(bool(wt)), pbias, int(act), py,
                                      ldy, _stream(stream, X, W, Y, bias))
    elif ws is not None:
        st = getattr(load(), fn_name)(M, N, K, px, ldx, pw, ldw, int(bool(wt)), pbias, int(act), py,
                                      ldy, ws[0], ws[1], _stream(stream, X, W, Y, bias))
    else:
        st = getattr(load(), fn_name)(M, N, K, px, ldx, pw, ldw, pbias, int(act), py, ldy,
                                      _stream(stream, X, W, Y, bias))
    _check(st, fn_name)
    return Y


_call_module = None


class _NoShortCalls:
    """Every call takes the Python code: another build of the library is in use."""

    def __getattr__(self, name):
        return lambda *args: None


def _short_calls():
    """The module that takes tensors apart for the short calls below. Its functions
    return a status, or None where an argument is not what the call takes; what is
    wrong with it, if anything is, the Python code after the call finds."""
    global _call_module
    if _call_module is None:
        load()
        _torch()
        if os.path.realpath(_LIB_PATH) != os.path.realpath(_DEFAULT_LIB_PATH):
            _call_module = _NoShortCalls()   # (the module is linked with the library beside it)
            return _call_module
        try:
            from . import _call as module
        except ImportError as e:
            raise ImportError("linear_layer_amd/_call.so is missing or does not load: build it with "
                              "`python -m linear_layer_amd._build`") from e
        module.setup(*_raw_getters())
        _call_module = module
    return _call_module


# ---- microscaled 4-bit floating point ---------------------------------------

def mx4_shapes(rows: int, K: int):
    """The shapes of the codes and of the scales of a rows x K matrix (both uint8)."""
    return (rows, (K + 1) // 2), (rows, (K + 31) // 32)


_TYPES = None


def _type_of(t, name):
    """The LL_TYPE_* value of a tensor's dtype."""
    global _TYPES
    torch = _torch()
    if _TYPES is None:
        _TYPES = {torch.float32: TYPE_F32, torch.float16: TYPE_F16, torch.bfloat16: TYPE_BF16}
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _TYPES:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return _TYPES[t.dtype]


def _packed(codes, scales, K, what):
    """(rows, codes pointer, ld, scales pointer, ld) of a packed matrix of K values a row."""
    torch = _torch()
    pq, rows, nq, ldq = _mat(codes, torch.uint8, f"{what} codes")
    ps, rows2, ns, lds = _mat(scales, torch.uint8, f"{what} scales")
    want, want_s = mx4_shapes(rows, K)
    if (rows, nq) != want or (rows2, ns) != want_s:
        raise ValueError(f"{what}: {K} values a row need codes {want} and scales {want_s}, got "
                         f"{tuple(codes.shape)} and {tuple(scales.shape)}")
    return rows, pq, ldq, ps, lds


def mx4_quantize(X, codes, scales, trans: bool = False, stream=None):
    """Quantise X (float32, float16 or bfloat16; M x K) into uint8 codes and scales,
    along its rows, or with ``trans`` along its columns into the packed transposed
    matrix (K rows of M values). Returns (codes, scales)."""
    if stream is None:
        st = _short_calls().mx4_quantize(X, codes, scales, trans)
        if st is not None:
            _check(st, "mx4_quantize")
            return codes, scales
    t = _type_of(X, "X")
    px, M, K, ldx = _mat(X, X.dtype, "X")
    rows, pq, ldq, ps, lds = _packed(codes, scales, M if trans else K, "X")
    if rows != (K if trans else M):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, codes {tuple(codes.shape)}")
    _check(load().mx4_quantize(M, K, t, px, ldx, int(bool(trans)), pq, ldq, ps, lds,
                               _stream(stream, X, codes, scales)), "mx4_quantize")
    return codes, scales


def mx4_dequantize(codes, scales, Y, stream=None):
    """Y (float32, float16 or bfloat16; M x K) = the values codes and scales stand for."""
    if stream is None:
        st = _short_calls().mx4_dequantize(codes, scales, Y)
        if st is not None:
            _check(st, "mx4_dequantize")
            return Y
    t = _type_of(Y, "Y")
    py, M, K, ldy = _mat(Y, Y.dtype, "Y")
    rows, pq, ldq, ps, lds = _packed(codes, scales, K, "Y")
    if rows != M:
        raise ValueError(f"shape mismatch: Y {tuple(Y.shape)}, codes {tuple(codes.shape)}")
    _check(load().mx4_dequantize(M, K, pq, ldq, ps, lds, t, py, ldy, _stream(stream, Y, codes, scales)),
           "mx4_dequantize")
    return Y


def gemm_mx4f32_nt(A, SA, B, SB, C, alpha: float = 1.0, beta: float = 0.0, K: int | None = None, stream=None):
    """C = alpha*A*B^T + beta*C with A (M x K) and B (N x K) as uint8 codes and scales;
    K is twice the codes' width unless given (an odd K has to be)."""
    if stream is None:
        st = _short_calls().gemm_mx4f32_nt(A, SA, B, SB, C, alpha, beta, K)
        if st is not None:
            _check(st, "gemm_mx4f32_nt")
            return C
    torch = _torch()
    if K is None:
        K = 2 * A.shape[1] if getattr(A, "ndim", 0) == 2 else 0
    K = int(K)
    M, pa, lda, psa, ldsa = _packed(A, SA, K, "A")
    N, pb, ldb, psb, ldsb = _packed(B, SB, K, "B")
    pc, M2, N2, ldc = _mat(C, torch.float32, "C")
    if M2 != M or N2 != N:
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)}")
    _check(load().gemm_mx4f32_nt(M, N, K, float(alpha), pa, lda, psa, ldsa, pb, ldb, psb, ldsb, float(beta), pc,
                                 ldc, _stream(stream, A, SA, B, SB, C)), "gemm_mx4f32_nt")
    return C


def _gemm_16mx4(fn_name, in_dtype, A, B, SB, C, alpha, beta, stream):
    if stream is None:
        st = getattr(_short_calls(), fn_name)(A, B, SB, C, alpha, beta)
        if st is not None:
            _check(st, fn_name)
            return C
    in_dtype = getattr(_torch(), in_dtype)
    torch = _torch()
    pa, M, K, lda = _mat(A, in_dtype, "A")
    N, pb, ldb, psb, ldsb = _packed(B, SB, K, "B")
    pc, M2, N2, ldc = _mat(C, torch.float32, "C")
    if M2 != M or N2 != N:
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)}")
    _check(getattr(load(), fn_name)(M, N, K, float(alpha), pa, lda, pb, ldb, psb, ldsb, float(beta), pc, ldc,
                                    _stream(stream, A, B, SB, C)), fn_name)
    return C


def gemm_f16mx4f32_nt(A, B, SB, C, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """C = alpha*A*B^T + beta*C with fp16 A and B (N x K) as uint8 codes and scales."""
    return _gemm_16mx4("gemm_f16mx4f32_nt", "float16", A, B, SB, C, alpha, beta, stream)


def gemm_bf16mx4f32_nt(A, B, SB, C, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """C = alpha*A*B^T + beta*C with bf16 A and B (N x K) as uint8 codes and scales."""
    return _gemm_16mx4("gemm_bf16mx4f32_nt", "bfloat16", A, B, SB, C, alpha, beta, stream)


def mx4_chosen_kernel(M: int, N: int, K: int, a: int, aligned: bool = True, workspace: bool = True,
                      num_cus: int = 0) -> str:
    """Name of the kernel that a product with A in the form ``a`` (A_*) takes, with rows
    on 16 bytes or not; "" for one without work."""
    return load().ll_mx4_chosen_kernel(int(M), int(N), int(K), int(a), int(bool(aligned)), int(bool(workspace)),
                                       int(num_cus)).decode()


# ---- residual norms ------------------------------------------------------------

def _opt_mat(t, dtype, name, M, N):
    """(pointer, ld) of an M x N matrix, or (None, 0) for None."""
    if t is None:
        return None, max(N, 1)
    p, rows, cols, ld = _mat(t, dtype, name)
    if (rows, cols) != (M, N):
        raise ValueError(f"{name} must be {(M, N)}, got {tuple(t.shape)}")
    return p, ld


def _opt_vec(t, name, N):
    """Pointer of a contiguous fp32 vector of N values, or None."""
    torch = _torch()
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != N or not t.is_cuda:
        raise ValueError(f"{name} must be a 1-D fp32 device tensor of length {N}")
    if N > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def rmsnorm_residual(Y, w_post, gate, alpha, X, w_pre, XO, H, eps: float = 1e-5, stream=None):
    """XO = X + alpha*gate*rms(Y)*w_post and H = rms(XO)*w_pre over the rows, rms(v) =
    v / sqrt(mean(v^2) + eps). Y is fp32, X, XO and H of one type; Y, the vectors and
    one of XO and H may be None. XO may be X. Returns (XO, H)."""
    if stream is None:
        st = _short_calls().rmsnorm_residual(Y, w_post, gate, alpha, X, w_pre, XO, H, eps)
        if st is not None:
            _check(st, "rmsnorm_residual")
            return XO, H
    torch = _torch()
    t = _type_of(X, "X")
    px, M, N, ldx = _mat(X, X.dtype, "X")
    py, ldy = _opt_mat(Y, torch.float32, "Y", M, N)
    pxo, ldxo = _opt_mat(XO, X.dtype, "XO", M, N)
    ph, ldh = _opt_mat(H, X.dtype, "H", M, N)
    _check(load().rmsnorm_residual(M, N, t, py, ldy, _opt_vec(w_post, "w_post", N), _opt_vec(gate, "gate", N),
                                   float(alpha), px, ldx, _opt_vec(w_pre, "w_pre", N), float(eps), pxo, ldxo, ph, ldh,
                                   _stream(stream, X, Y, XO, H, w_post, gate, w_pre)), "rmsnorm_residual")
    return XO, H


def rmsnorm_grad_workspace_size(M: int, N: int) -> int:
    """Bytes of workspace rmsnorm_residual_grad needs for M x N."""
    if M > _INT_MAX or N > _INT_MAX:
        raise ValueError(f"the calls take sizes up to {_INT_MAX}")
    n = load().ll_rmsnorm_grad_workspace_size(int(M), int(N))
    if n < 0:
        raise ValueError("negative size")
    return n


def rmsnorm_residual_grad(DXO, DH, Y, w_post, gate, alpha, X, w_pre, DY, DX, dgate, dw_post, dw_pre, workspace,
                          eps: float = 1e-5, stream=None):
    """The gradient of rmsnorm_residual: DXO and DH (either may be None) are those of XO
    and H; DY, DX, dgate, dw_post and dw_pre are written (each may be None). workspace:
    a contiguous device tensor of rmsnorm_grad_workspace_size(M, N) bytes or more.
    Returns (DY, DX, dgate, dw_post, dw_pre)."""
    if stream is None:
        st = _short_calls().rmsnorm_residual_grad(DXO, DH, Y, w_post, gate, alpha, X, w_pre, DY, DX, dgate, dw_post, dw_pre,
                                           workspace, eps)
        if st is not None:
            _check(st, "rmsnorm_residual_grad")
            return DY, DX, dgate, dw_post, dw_pre
    torch = _torch()
    t = _type_of(X, "X")
    px, M, N, ldx = _mat(X, X.dtype, "X")
    pdxo, lddxo = _opt_mat(DXO, X.dtype, "DXO", M, N)
    pdh, lddh = _opt_mat(DH, X.dtype, "DH", M, N)
    py, ldy = _opt_mat(Y, torch.float32, "Y", M, N)
    pdy, lddy = _opt_mat(DY, torch.float32, "DY", M, N)
    pdx, lddx = _opt_mat(DX, X.dtype, "DX", M, N)
    pws, nws = None, 0
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous device tensor")
        pws, nws = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(load().rmsnorm_residual_grad(
        M, N, t, pdxo, lddxo, pdh, lddh, py, ldy, _opt_vec(w_post, "w_post", N), _opt_vec(gate, "gate", N), float(alpha),
        px, ldx, _opt_vec(w_pre, "w_pre", N), float(eps), pdy, lddy, pdx, lddx, _opt_vec(dgate, "dgate", N),
        _opt_vec(dw_post, "dw_post", N), _opt_vec(dw_pre, "dw_pre", N), pws, nws,
        _stream(stream, X, DXO, DH, Y, w_post, gate, w_pre, DY, DX, dgate, dw_post, dw_pre, workspace)),
        "rmsnorm_residual_grad")
    return DY, DX, dgate, dw_post, dw_pre


# ---- microscaled 8-bit floating point ---------------------------------------

def mx8_shapes(rows: int, K: int):
    """The shapes of the codes and of the scales of a rows x K matrix (both uint8)."""
    return (rows, K), (rows, (K + 31) // 32)


def _packed8(q, M, K, what):
    """(codes pointer, ld, scales pointer, ld) of an M x K matrix in 8 bits."""
    torch = _torch()
    codes, scales = q
    pq, rows, nq, ldq = _mat(codes, torch.uint8, f"{what} codes")
    ps, rows2, ns, lds = _mat(scales, torch.uint8, f"{what} scales")
    want, want_s = mx8_shapes(M, K)
    if (rows, nq) != want or (rows2, ns) != want_s:
        raise ValueError(f"{what}: {M} rows of {K} values need codes {want} and scales {want_s}, got "
                         f"{tuple(codes.shape)} and {tuple(scales.shape)}")
    return pq, ldq, ps, lds


def mx8_quantize(X, codes, scales, stream=None):
    """Quantise X (float32, float16 or bfloat16; M x K) along its rows into uint8 codes
    and scales. Returns (codes, scales)."""
    if stream is None:
        st = _short_calls().mx8_quantize(X, codes, scales)
        if st is not None:
            _check(st, "mx8_quantize")
            return codes, scales
    t = _type_of(X, "X")
    px, M, K, ldx = _mat(X, X.dtype, "X")
    packed = _packed8((codes, scales), M, K, "X")
    _check(load().mx8_quantize(M, K, t, px, ldx, *packed, _stream(stream, X, codes, scales)), "mx8_quantize")
    return codes, scales


def mx8_dequantize(codes, scales, Y, stream=None):
    """Y (float32, float16 or bfloat16; M x K) = the values codes and scales stand for."""
    if stream is None:
        st = _short_calls().mx8_dequantize(codes, scales, Y)
        if st is not None:
            _check(st, "mx8_dequantize")
            return Y
    t = _type_of(Y, "Y")
    py, M, K, ldy = _mat(Y, Y.dtype, "Y")
    packed = _packed8((codes, scales), M, K, "Y")
    _check(load().mx8_dequantize(M, K, *packed, t, py, ldy, _stream(stream, Y, codes, scales)), "mx8_dequantize")
    return Y


# ---- the 16-bit layer and its gradients ----------------------------------------

def _type16_of(t, name):
    kind = _type_of(t, name)
    if kind == TYPE_F32:
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    return kind


def _same_or_f32(t, dtype, name):
    """The LL_TYPE_* of a tensor that may be of the call's 16-bit dtype or float32."""
    kind = _type_of(t, name)
    if kind != TYPE_F32 and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} or float32, got {t.dtype}")
    return kind


def _offsets(offsets):
    """(groups, pointer) of the groups' row numbers."""
    torch = _torch()
    if offsets is None:
        return 1, None
    if (not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_cuda
            or offsets.shape[0] < 1 or (offsets.shape[0] > 1 and offsets.stride(0) != 1)):
        raise ValueError("offsets must be a contiguous 1-D int32 device tensor of groups + 1 row numbers")
    if offsets.shape[0] - 1 > MAX_GROUPS:
        raise ValueError(f"at most {MAX_GROUPS} groups")
    return offsets.shape[0] - 1, offsets.data_ptr()


def _weights(W, dtype, groups, grouped, name):
    """(pointer, N, K, ld, stride) of one weight, or of a stack of them."""
    if not grouped:
        return _mat(W, dtype, name) + (0,)
    p, n, N, K, ld, stride = _bmat(W, dtype, name)
    if n != groups:
        raise ValueError(f"{name}: {groups} groups need as many weights, got {n}")
    return p, N, K, ld, stride


def _group_vec(t, groups, grouped, N, name):
    """Pointer of contiguous fp32 values, N or groups x N, or None."""
    torch = _torch()
    if t is None:
        return None
    shape = (groups, N) if grouped else (N,)
    if (not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_cuda
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous fp32 device tensor of shape {shape}")
    return t.data_ptr()


def _held(v, dtype, M, N, name):
    """(pointer, ld, codes, ld, scales, ld) of an M x N tensor of dtype or a pair (codes,
    scales) in 8 bits, or of None; and the tensors."""
    one = max(N, 1)
    if v is None:
        return (None, one, None, one, None, one), ()
    if isinstance(v, (tuple, list)):
        if len(v) != 2:
            raise ValueError(f"{name} must be a tensor or a pair (codes, scales)")
        return (None, one) + _packed8(v, M, N, name), tuple(v)
    p, ld = _opt_mat(v, dtype, name, M, N)
    return (p, ld, None, one, None, one), (v,)


def _workspace(t):
    """(pointer, bytes) of a workspace tensor."""
    if not isinstance(t, _torch().Tensor) or not t.is_cuda or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    return t.data_ptr(), t.numel() * t.element_size()


def _c_ints(*numbers):
    """Numbers as the calls take them. (ctypes would pass on the lower 32 bits of others.)"""
    got = tuple(int(n) for n in numbers)
    if any(not -_INT_MAX <= n <= _INT_MAX for n in got):
        raise ValueError(f"the calls take numbers up to {_INT_MAX}, got {got}")
    return got


def linear16_workspace_size(product: int, M: int, N: int, K: int, groups: int = 1) -> int:
    """Bytes of workspace that linear16_nt (L16_FORWARD) or linear16_grad_input
    (L16_GRAD_INPUT) gains from on the current device (0: none)."""
    if groups > MAX_GROUPS:
        raise ValueError(f"the calls take up to {MAX_GROUPS} groups")
    n = load().ll_linear16_workspace_size(*_c_ints(product, M, N, K, groups))
    if n < 0:
        raise ValueError("negative size, or a product that takes no workspace")
    return n


def _shares_workspace(product, M, N, K, groups, workspace, stream, like):
    """(pointer, bytes, tensor) of the workspace given, or on the current stream of one that
    the product gains from."""
    if workspace is None and stream is None:
        need = load().ll_linear16_workspace_size(product, M, N, K, groups)
        if need > 0:
            workspace = _torch().empty(need, dtype=_torch().uint8, device=like.device)
    return (None, 0, None) if workspace is None else (*_workspace(workspace), workspace)


def linear16_chosen_kernel(product: int, M: int, N: int, K: int, groups: int = 1, aligned: bool = True,
                           num_cus: int = 0) -> str:
    """Name of the kernel that a product (L16_*) of the layer takes, with rows on 16 bytes
    or not; "" for one without work."""
    return load().ll_linear16_chosen_kernel(*_c_ints(product, M, N, K, groups, bool(aligned), num_cus)).decode()


def linear16_nt(X, W, bias, act: int, R, Y, Z=None, offsets=None, workspace=None, stream=None):
    """Y = act(X*W^T + bias) + R with X (M x K) and W (N x K) in float16 or bfloat16, fp32
    sums, bias fp32 or None, R and Y (M x N) both of X's dtype or both float32; R may be
    None or Y. Z, if given, receives X*W^T + bias: a tensor of X's dtype, or a pair (codes,
    scales) of uint8 tensors (``mx8_shapes``). With ``offsets`` (groups + 1 ascending row
    numbers, int32, on the device) W is groups x N x K, bias groups x N, and rows outside
    all groups stay as they are. A product that does not fill the GPU gains from a workspace of
    linear16_workspace_size bytes: on the current stream it comes from torch's allocator, with
    ``stream`` given the call runs without one unless it is given too, which for few rows takes
    longer and adds in another order. ACT_RELU maps NaN to 0, as it does z <= 0. Returns Y."""
    if stream is None:
        st = _short_calls().linear16_nt(X, W, bias, act, R, Y, Z, offsets, workspace)
        if st is not None:
            _check(st, "linear16_nt")
            return Y
    t = _type16_of(X, "X")
    px, M, K, ldx = _mat(X, X.dtype, "X")
    groups, poff = _offsets(offsets)
    pw, N, K2, ldw, stride = _weights(W, X.dtype, groups, poff is not None, "W")
    ty = _same_or_f32(Y, X.dtype, "Y")
    py, M2, N2, ldy = _mat(Y, Y.dtype, "Y")
    if groups and (K2 != K or M2 != M or N2 != N):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, Y {tuple(Y.shape)}")
    pr, ldr = _opt_mat(R, Y.dtype, "R", M, N)
    held, zs = _held(Z, X.dtype, M, N, "Z")
    pb = _group_vec(bias, groups, poff is not None, N, "bias")
    s = _stream(stream, X, W, Y, R, bias, offsets, workspace, *zs)
    pws, nws, workspace = _shares_workspace(L16_FORWARD, M, N, K, groups, workspace, stream, X)
    _check(load().linear16_nt(M, N, K, t, px, ldx, groups, poff, pw, ldw, stride, pb, *_c_ints(act), ty, pr, ldr, py, ldy,
                              *held, pws, nws, s), "linear16_nt")
    return Y


def linear16_grad_act_workspace_size(M: int, N: int, groups: int = 1) -> int:
    """Bytes of workspace linear16_grad_act needs for dbias."""
    if groups > MAX_GROUPS:
        raise ValueError(f"the calls take up to {MAX_GROUPS} groups")
    n = load().ll_linear16_grad_act_workspace_size(*_c_ints(M, N, groups))
    if n < 0:
        raise ValueError("negative size")
    return n


def linear16_grad_act(DY, Z, act: int, DZ, dbias=None, offsets=None, workspace=None, stream=None):
    """DZ = DY * act'(Z) and dbias = DZ's sums over the rows (of each group): DY (M x N) of
    DZ's dtype or float32, Z a tensor of DZ's dtype or a pair (codes, scales) in 8 bits (None
    for ACT_NONE). DZ may be DY or Z. dbias takes a workspace (a contiguous device tensor of
    linear16_grad_act_workspace_size bytes); without one it comes from torch's allocator, on
    the current stream only. Returns DZ."""
    if stream is None:
        st = _short_calls().linear16_grad_act(DY, Z, act, DZ, dbias, offsets, workspace)
        if st is not None:
            _check(st, "linear16_grad_act")
            return DZ
    torch = _torch()
    t = _type16_of(DZ, "DZ")
    pdz, M, N, lddz = _mat(DZ, DZ.dtype, "DZ")
    groups, poff = _offsets(offsets)
    ty = _same_or_f32(DY, DZ.dtype, "DY")
    pdy, lddy = _opt_mat(DY, DY.dtype, "DY", M, N)
    held, zs = _held(Z, DZ.dtype, M, N, "Z")
    pb = _group_vec(dbias, groups, poff is not None, N, "dbias")
    s = _stream(stream, DZ, DY, dbias, offsets, workspace, *zs)
    pws, nws = None, 0
    if pb is not None:
        if workspace is None:
            if stream is not None:
                raise ValueError("dbias on a stream that is given needs a workspace")
            workspace = torch.empty(linear16_grad_act_workspace_size(M, N, groups), dtype=torch.uint8, device=DZ.device)
        pws, nws = _workspace(workspace)
    _check(load().linear16_grad_act(M, N, t, *_c_ints(act), ty, pdy, lddy, groups, poff, *held, pdz, lddz, pb, pws, nws, s),
           "linear16_grad_act")
    return DZ


def linear16_grad_input(DZ, W, DX, offsets=None, workspace=None, stream=None):
    """DX = DZ*W: DZ (M x N) and W (N x K, or groups x N x K) in float16 or bfloat16, DX
    (M x K) of that dtype or float32. workspace: as linear16_nt's. Returns DX."""
    t = _type16_of(DZ, "DZ")
    pdz, M, N, lddz = _mat(DZ, DZ.dtype, "DZ")
    groups, poff = _offsets(offsets)
    pw, N2, K, ldw, stride = _weights(W, DZ.dtype, groups, poff is not None, "W")
    tx = _same_or_f32(DX, DZ.dtype, "DX")
    pdx, M2, K2, lddx = _mat(DX, DX.dtype, "DX")
    if groups and (N2 != N or M2 != M or K2 != K):
        raise ValueError(f"shape mismatch: DZ {tuple(DZ.shape)}, W {tuple(W.shape)}, DX {tuple(DX.shape)}")
    s = _stream(stream, DZ, W, DX, offsets, workspace)
    pws, nws, workspace = _shares_workspace(L16_GRAD_INPUT, M, N, K, groups, workspace, stream, DZ)
    _check(load().linear16_grad_input(M, N, K, t, pdz, lddz, groups, poff, pw, ldw, stride, tx, pdx, lddx, pws, nws, s),
           "linear16_grad_input")
    return DX


def linear16_grad_weight(DZ, X, DW, beta: float = 0.0, offsets=None, stream=None):
    """DW = DZ^T*X + beta*DW: DZ (M x N) in float16 or bfloat16, X (M x K) of that dtype or a
    pair (codes, scales) in 8 bits, DW (N x K, or groups x N x K) of that dtype or float32.
    Returns DW."""
    t = _type16_of(DZ, "DZ")
    pdz, M, N, lddz = _mat(DZ, DZ.dtype, "DZ")
    groups, poff = _offsets(offsets)
    tw = _same_or_f32(DW, DZ.dtype, "DW")
    pdw, N2, K, lddw, stride = _weights(DW, DW.dtype, groups, poff is not None, "DW")
    held, xs = _held(X, DZ.dtype, M, K, "X")
    if not xs:
        raise TypeError("X must be a tensor or a pair (codes, scales)")
    if groups and N2 != N:
        raise ValueError(f"shape mismatch: DZ {tuple(DZ.shape)}, DW {tuple(DW.shape)}")
    _check(load().linear16_grad_weight(M, N, K, t, pdz, lddz, groups, poff, *held, tw, float(beta), pdw, lddw, stride,
                                       _stream(stream, DZ, DW, offsets, *xs)), "linear16_grad_weight")
    return DW
