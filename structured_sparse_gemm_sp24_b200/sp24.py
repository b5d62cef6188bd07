"""Python binding of libsp24 (the C ABI declared in include/sp24.h).

Argument marshalling only: every function takes torch tensors that already
live on the device, checks that they are dense and on CUDA, and passes their
pointers, sizes and the current CUDA stream to the C function of the same
name.  The e4m3 and norm functions, which matter at single tokens, are checked
and called by a native module (csrc/binding.cpp, _binding.so); it also checks
types, sizes and the device.  All computation happens in the library's CUDA kernels; there is no
fallback path.  A non-OK status raises :class:`Sp24Error`.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsp24.so")

# enums of include/sp24.h
SP24_OK = 0
SP24_ERR_ARG = 1
SP24_ERR_ALIGN = 2
SP24_ERR_PATTERN = 3
SP24_ERR_CUDA = 4
SP24_ERR_TIMEOUT = 5
SP24_ERR_UNSUPPORTED = 6
SP24_ERR_INDEX = 7
SP24_MAGNITUDE = 0
SP24_WANDA = 1
SP24_BF16 = 0
SP24_INT8 = 1
SP24_FP8 = 2
SP24_F32 = 3
SP24_OUT_BF16 = 0
SP24_OUT_INT32 = 1
SP24_OUT_INT8 = 2
SP24_OUT_F32 = 3
SP24_NORM_MAX_K = 16384
SP24_NOALLOC_MAX_K = 65536
SP24_PERMUTE_MAX_K = 65536

_c_i64 = ctypes.c_int64
_c_p = ctypes.c_void_p
_c_int = ctypes.c_int
_c_dbl = ctypes.c_double
_c_size = ctypes.c_size_t
_c_flt = ctypes.c_float

# name -> (restype, argtypes)
SIGNATURES = {
    "sp24_mask_bytes": (_c_size, [_c_i64, _c_i64]),
    "sp24_vals_bytes": (_c_size, [_c_i64, _c_i64, _c_int]),
    "sp24_meta_bytes": (_c_size, [_c_i64, _c_i64]),
    "sp24_prune_workspace_bytes": (_c_size, [_c_i64, _c_int]),
    "sp24_colnorm": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p]),
    "sp24_prune": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_i64, _c_int, _c_int, _c_p, _c_p,
                            _c_p, _c_p]),
    "sp24_wscale": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_dbl, _c_p, _c_p]),
    "sp24_act_scale_workspace_bytes": (_c_size, []),
    "sp24_act_scale": (_c_int, [_c_p, _c_i64, _c_dbl, _c_p, _c_p, _c_p]),
    "sp24_quantize": (_c_int, [_c_p, _c_i64, _c_p, _c_p, _c_p]),
    "sp24_compress": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p, _c_p]),
    "sp24_prune_compress": (_c_int, [_c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p, _c_int,
                                     _c_p, _c_p, _c_p, _c_p]),
    "sp24_prune_compress_int8": (_c_int, [_c_p, _c_i64, _c_i64, _c_dbl, _c_p, _c_p, _c_p, _c_p,
                                          _c_p]),
    "sp24_prune_progressive": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_i64, _c_int, _c_p, _c_p,
                                        _c_p, _c_p, _c_p, _c_p]),
    "sp24_conv3x3": (_c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_int,
                              _c_p, _c_p, _c_int, _c_p, _c_p, _c_p]),
    "sp24_gemm": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_int, _c_p, _c_p, _c_int,
                           _c_p, _c_p, _c_p]),
    "sp24_device_status": (_c_int, [_c_p]),
    "sp24_strerror": (ctypes.c_char_p, [_c_int]),
    "sp24_version": (_c_int, []),
    "sp24_last_cuda_error": (ctypes.c_char_p, []),
    "sp24_prune_wanda_noalloc": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_i64, _c_int, _c_p, _c_p,
                                          _c_p]),
    "sp24_gemm_plan": (_c_int, [_c_i64, _c_i64, _c_i64, _c_int, _c_p]),
    "sp24_selftest_wait_timeout": (_c_int, [_c_i64, _c_p]),
    "sp24_fake_quant": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p]),
    "sp24_permute_workspace_bytes": (_c_size, [_c_i64, _c_i64]),
    "sp24_permute_search": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_int, _c_i64, _c_p, _c_p,
                                     _c_size, _c_p, _c_p]),
    "sp24_permute_columns": (_c_int, [_c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p]),
    "sp24_scale_bytes": (_c_size, [_c_i64, _c_i64]),
    "sp24_quantize_fp8": (_c_int, [_c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p]),
    "sp24_prune_compress_fp8": (_c_int, [_c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p, _c_p,
                                         _c_p, _c_p, _c_p]),
    "sp24_compress_fp8": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p]),
    "sp24_gemm_fp8": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_int,
                               _c_p, _c_p]),
    "sp24_rmsnorm_quant": (_c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_int, _c_flt, _c_int,
                                    _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "sp24_rmsnorm_backward_workspace_bytes": (_c_size, [_c_i64, _c_i64]),
    "sp24_rmsnorm_backward": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_int, _c_p,
                                       _c_p, _c_p, _c_size, _c_p]),
    "sp24_im2col3x3": (_c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_int, _c_p, _c_p]),
}


class GemmPlan(ctypes.Structure):
    """sp24_gemm_plan_t: the launch sp24_gemm makes for a problem."""
    _fields_ = [("kernel", ctypes.c_char * 16), ("tile_tokens", ctypes.c_int32),
                ("tile_channels", ctypes.c_int32), ("split_k", ctypes.c_int32),
                ("cluster", ctypes.c_int32), ("ctas", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {"kernel": self.kernel.decode(), "tile_tokens": self.tile_tokens,
                "tile_channels": self.tile_channels, "split_k": self.split_k,
                "cluster": self.cluster, "ctas": self.ctas}


class PermuteResult(ctypes.Structure):
    """sp24_permute_result_t."""
    _fields_ = [("swaps", ctypes.c_int64), ("kept_before", ctypes.c_int64),
                ("kept_after", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {"swaps": self.swaps, "kept_before": self.kept_before,
                "kept_after": self.kept_after}


_LIB: Optional[ctypes.CDLL] = None


class Sp24Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        detail = ""
        if self.status == SP24_ERR_CUDA:
            detail = " [" + lib().sp24_last_cuda_error().decode() + "]"
        super().__init__(f"{where}: {strerror(status)} (status {status}){detail}")


def lib() -> ctypes.CDLL:
    """The loaded library.  Raises if libsp24.so has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m structured_sparse_gemm_sp24_b200.build` (needs nvcc)")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = h
    return _LIB


_NATIVE = None
_NATIVE_FUNCTIONS = ("sp24_quantize_fp8", "sp24_prune_compress_fp8", "sp24_compress_fp8",
                     "sp24_gemm_fp8", "sp24_rmsnorm_quant", "sp24_rmsnorm_backward",
                     "sp24_meta_bytes", "sp24_rmsnorm_backward_workspace_bytes")


def native():
    """The native half of the binding, bound to the loaded library.  Raises if
    _binding.so has not been built for this Python and torch."""
    global _NATIVE
    if _NATIVE is None:
        h = lib()
        how = "build it with `python -m structured_sparse_gemm_sp24_b200.build`"
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError(f"_binding.so is missing or does not load: {how}") from e
        from .build import binding_tag
        if _binding.built_for != binding_tag():
            raise RuntimeError(f"_binding.so is a {_binding.built_for}, this is {binding_tag()}: {how}")
        _binding.bind(*(ctypes.cast(getattr(h, f), _c_p).value for f in _NATIVE_FUNCTIONS))
        _NATIVE = _binding
    return _NATIVE


def _raw(stream) -> Optional[int]:
    """A raw stream for the native functions (None: torch's current stream)."""
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


def strerror(status: int) -> str:
    return lib().sp24_strerror(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != SP24_OK:
        raise Sp24Error(status, where)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("sp24: tensors must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("sp24: tensors must be contiguous")
    return t.data_ptr()


def _f32(t: Optional[torch.Tensor], name: str) -> None:
    """Refuses a tensor that the library would read as float32 and that is not (a
    shorter type would be read past its end)."""
    if t is not None and t.dtype != torch.float32:
        raise ValueError(f"sp24: {name} must be float32, not {t.dtype}")


def _operands(X: torch.Tensor, vals: torch.Tensor, dtype: int) -> None:
    """Refuses product operands that are not bf16 or int8 as `dtype` says (one-byte
    codes taken for bf16 would be read past their end).  Whole numbers of the same
    size, the values' bits, pass."""
    want = {SP24_BF16: torch.bfloat16, SP24_INT8: torch.int8}.get(dtype)
    for t, name in ((X, "X"), (vals, "vals")):
        if want is not None and t.dtype != want and (t.is_floating_point()
                                                     or t.element_size() != want.itemsize):
            raise ValueError(f"sp24: {name} must be {want} for this product, not {t.dtype}")


def _stream(stream) -> Optional[int]:
    if stream is None:   # (current_stream() builds a Python object: 3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# ------------------------------------------------------------------- sizes
def sp24_mask_bytes(N: int, K: int) -> int:
    return lib().sp24_mask_bytes(N, K)


def sp24_vals_bytes(N: int, K: int, dtype: int) -> int:
    return lib().sp24_vals_bytes(N, K, dtype)


def sp24_meta_bytes(N: int, K: int) -> int:
    return lib().sp24_meta_bytes(N, K)


def sp24_prune_workspace_bytes(K: int, mode: int) -> int:
    return lib().sp24_prune_workspace_bytes(K, mode)


def sp24_scale_bytes(rows: int, K: int) -> int:
    return lib().sp24_scale_bytes(rows, K)


def sp24_rmsnorm_backward_workspace_bytes(M: int, K: int) -> int:
    return lib().sp24_rmsnorm_backward_workspace_bytes(M, K)


def sp24_act_scale_workspace_bytes() -> int:
    return lib().sp24_act_scale_workspace_bytes()


def sp24_version() -> int:
    return lib().sp24_version()


# ---------------------------------------------------------------- compute
def sp24_colnorm(Xc: torch.Tensor, norms: torch.Tensor, stream=None) -> None:
    Mc, K = Xc.shape
    _check(lib().sp24_colnorm(_ptr(Xc), Mc, K, _ptr(norms), _stream(stream)), "sp24_colnorm")


def sp24_prune(W: torch.Tensor, Xc: Optional[torch.Tensor], mode: int, n_keep: int,
               mask_in: Optional[torch.Tensor], mask_out: torch.Tensor,
               workspace: Optional[torch.Tensor], stream=None) -> None:
    N, K = W.shape
    Mc = 0 if Xc is None else Xc.shape[0]
    _check(lib().sp24_prune(_ptr(W), N, K, _ptr(Xc), Mc, mode, n_keep, _ptr(mask_in),
                            _ptr(mask_out), _ptr(workspace), _stream(stream)), "sp24_prune")


def sp24_prune_wanda_noalloc(W: torch.Tensor, Xc: torch.Tensor, n_keep: int,
                             mask_in: Optional[torch.Tensor], mask_out: torch.Tensor,
                             stream=None) -> None:
    N, K = W.shape
    _check(lib().sp24_prune_wanda_noalloc(_ptr(W), N, K, _ptr(Xc), Xc.shape[0], n_keep,
                                          _ptr(mask_in), _ptr(mask_out), _stream(stream)),
           "sp24_prune_wanda_noalloc")


def sp24_wscale(W: torch.Tensor, mask: torch.Tensor, coverage: float, s_w: torch.Tensor,
                stream=None) -> None:
    N, K = W.shape
    _check(lib().sp24_wscale(_ptr(W), _ptr(mask), N, K, float(coverage), _ptr(s_w),
                             _stream(stream)), "sp24_wscale")


def sp24_act_scale(X: torch.Tensor, coverage: float, s_x: torch.Tensor,
                   workspace: torch.Tensor, stream=None) -> None:
    _f32(X, "X")
    _check(lib().sp24_act_scale(_ptr(X), X.numel(), float(coverage), _ptr(s_x),
                                _ptr(workspace), _stream(stream)), "sp24_act_scale")


def sp24_quantize(X: torch.Tensor, s_x: torch.Tensor, Xq: torch.Tensor, stream=None) -> None:
    _f32(X, "X")
    _f32(s_x, "s_x")
    _check(lib().sp24_quantize(_ptr(X), X.numel(), _ptr(s_x), _ptr(Xq), _stream(stream)),
           "sp24_quantize")


def sp24_compress(W: torch.Tensor, mask: torch.Tensor, dtype: int, s_w: Optional[torch.Tensor],
                  vals: torch.Tensor, meta: torch.Tensor, stream=None) -> None:
    N, K = W.shape
    _check(lib().sp24_compress(_ptr(W), _ptr(mask), N, K, dtype, _ptr(s_w), _ptr(vals),
                               _ptr(meta), _stream(stream)), "sp24_compress")


def sp24_prune_compress(W: torch.Tensor, mode: int, norms: Optional[torch.Tensor],
                        mask_in: Optional[torch.Tensor], mask_out: Optional[torch.Tensor],
                        dtype: int, s_w: Optional[torch.Tensor], vals: torch.Tensor,
                        meta: torch.Tensor, stream=None) -> None:
    N, K = W.shape
    _check(lib().sp24_prune_compress(_ptr(W), N, K, mode, _ptr(norms), _ptr(mask_in),
                                     _ptr(mask_out), dtype, _ptr(s_w), _ptr(vals), _ptr(meta),
                                     _stream(stream)), "sp24_prune_compress")


def sp24_prune_progressive(W: torch.Tensor, Xc: Optional[torch.Tensor], mode: int,
                           mask1_out: Optional[torch.Tensor], mask2_out: Optional[torch.Tensor],
                           vals: Optional[torch.Tensor], meta: Optional[torch.Tensor],
                           workspace: Optional[torch.Tensor], stream=None) -> None:
    N, K = W.shape
    Mc = Xc.shape[0] if Xc is not None else 0
    _check(lib().sp24_prune_progressive(_ptr(W), N, K, _ptr(Xc), Mc, mode, _ptr(mask1_out),
                                        _ptr(mask2_out), _ptr(vals), _ptr(meta), _ptr(workspace),
                                        _stream(stream)), "sp24_prune_progressive")


def sp24_prune_compress_int8(W: torch.Tensor, coverage: float, mask_out: Optional[torch.Tensor],
                             s_w: torch.Tensor, vals: torch.Tensor, meta: torch.Tensor,
                             stream=None) -> None:
    N, K = W.shape
    _check(lib().sp24_prune_compress_int8(_ptr(W), N, K, coverage, _ptr(mask_out), _ptr(s_w),
                                          _ptr(vals), _ptr(meta), _stream(stream)),
           "sp24_prune_compress_int8")


def sp24_conv3x3(X: torch.Tensor, vals: torch.Tensor, meta: torch.Tensor, Cout: int, dtype: int,
                 s_x: Optional[torch.Tensor], s_w: Optional[torch.Tensor], out_kind: int,
                 s_y: Optional[torch.Tensor], Y: torch.Tensor, stream=None) -> None:
    Bn, H, W, C = X.shape
    _operands(X, vals, dtype)
    _check(lib().sp24_conv3x3(_ptr(X), Bn, H, W, C, _ptr(vals), _ptr(meta), Cout, dtype,
                              _ptr(s_x), _ptr(s_w), out_kind, _ptr(s_y), _ptr(Y),
                              _stream(stream)), "sp24_conv3x3")


def sp24_gemm(X: torch.Tensor, vals: torch.Tensor, meta: torch.Tensor, N: int, dtype: int,
              s_x: Optional[torch.Tensor], s_w: Optional[torch.Tensor], out_kind: int,
              s_y: Optional[torch.Tensor], Y: torch.Tensor, stream=None) -> None:
    M, K = X.shape
    _operands(X, vals, dtype)
    _check(lib().sp24_gemm(_ptr(X), M, K, _ptr(vals), _ptr(meta), N, dtype, _ptr(s_x),
                           _ptr(s_w), out_kind, _ptr(s_y), _ptr(Y), _stream(stream)),
           "sp24_gemm")


def sp24_gemm_plan(M: int, N: int, K: int, dtype: int) -> dict:
    """The kernel, tile and grid sp24_gemm uses for an M x N x K problem."""
    plan = GemmPlan()
    _check(lib().sp24_gemm_plan(M, N, K, dtype, ctypes.byref(plan)), "sp24_gemm_plan")
    return plan.as_dict()


def sp24_fake_quant(W: torch.Tensor, mask: torch.Tensor, s_w: torch.Tensor,
                    W_fq: torch.Tensor, stream=None) -> None:
    N, K = W.shape
    _check(lib().sp24_fake_quant(_ptr(W), _ptr(mask), N, K, _ptr(s_w), _ptr(W_fq),
                                 _stream(stream)), "sp24_fake_quant")


def sp24_permute_workspace_bytes(N: int, K: int) -> int:
    return lib().sp24_permute_workspace_bytes(N, K)


def sp24_permute_search(W: torch.Tensor, norms: Optional[torch.Tensor], n_keep: int,
                        max_swaps: int, perm: torch.Tensor, workspace: torch.Tensor,
                        stream=None) -> dict:
    """Greedy channel permutation search; blocks until it has finished."""
    N, K = W.shape
    res = PermuteResult()
    _check(lib().sp24_permute_search(_ptr(W), N, K, _ptr(norms), n_keep, max_swaps, _ptr(perm),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     ctypes.byref(res), _stream(stream)), "sp24_permute_search")
    return res.as_dict()


def sp24_permute_columns(A: torch.Tensor, perm: torch.Tensor, A_out: torch.Tensor,
                         stream=None) -> None:
    rows, K = A.shape
    _check(lib().sp24_permute_columns(_ptr(A), rows, K, A.element_size(), _ptr(perm),
                                      _ptr(A_out), _stream(stream)), "sp24_permute_columns")


def sp24_im2col3x3(X: torch.Tensor, A: torch.Tensor, stream=None) -> None:
    """X NHWC [B][H][W][C] -> A [B*H*W][9*C] (3x3, stride 1, zero padding 1)."""
    Bn, H, W, C = X.shape
    _check(lib().sp24_im2col3x3(_ptr(X), Bn, H, W, C, X.element_size(), _ptr(A),
                                _stream(stream)), "sp24_im2col3x3")


def sp24_quantize_fp8(X: torch.Tensor, Xq: torch.Tensor, e_x: torch.Tensor, stream=None) -> None:
    """X bf16 or float32 [M, K] -> e4m3 codes [M, K] and e8m0 scales."""
    _check(native().quantize_fp8(X, Xq, e_x, _raw(stream)), "sp24_quantize_fp8")


def sp24_prune_compress_fp8(W: torch.Tensor, mode: int, norms: Optional[torch.Tensor],
                            mask_in: Optional[torch.Tensor], mask_out: Optional[torch.Tensor],
                            vals: torch.Tensor, meta: torch.Tensor, e_w: torch.Tensor,
                            stream=None) -> None:
    """e4m3 weight conversion of bf16 W [N, K] in one pass."""
    _check(native().prune_compress_fp8(W, mode, norms, mask_in, mask_out, vals, meta, e_w,
                                       _raw(stream)), "sp24_prune_compress_fp8")


def sp24_compress_fp8(W: torch.Tensor, mask: torch.Tensor, vals: torch.Tensor,
                      meta: torch.Tensor, e_w: torch.Tensor, stream=None) -> None:
    """The same conversion under a given mask."""
    _check(native().compress_fp8(W, mask, vals, meta, e_w, _raw(stream)), "sp24_compress_fp8")


def sp24_gemm_fp8(X: torch.Tensor, e_x: torch.Tensor, vals: torch.Tensor, meta: torch.Tensor,
                  e_w: torch.Tensor, N: int, out_kind: int, Y: torch.Tensor, stream=None) -> None:
    """Y [M, N] = X W'^T of e4m3 X [M, K] and a compressed e4m3 weight."""
    _check(native().gemm_fp8(X, e_x, vals, meta, e_w, N, out_kind, Y, _raw(stream)),
           "sp24_gemm_fp8")


def sp24_rmsnorm_quant(X: torch.Tensor, R: Optional[torch.Tensor], gamma: torch.Tensor, eps: float,
                       out_dtype: int, s_x: Optional[torch.Tensor], H: Optional[torch.Tensor],
                       Y: torch.Tensor, e_y: Optional[torch.Tensor],
                       rstd: Optional[torch.Tensor], stream=None) -> None:
    """RMS norm of X (+ R) with an e4m3, int8 or bf16 output."""
    _check(native().rmsnorm_quant(X, R, gamma, eps, out_dtype, s_x, H, Y, e_y, rstd, _raw(stream)),
           "sp24_rmsnorm_quant")


def sp24_rmsnorm_backward(dY: torch.Tensor, dH: Optional[torch.Tensor], H: torch.Tensor,
                          gamma: torch.Tensor, rstd: torch.Tensor, dX: torch.Tensor,
                          dgamma: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """Gradients of sp24_rmsnorm_quant to X (and R) and gamma."""
    _check(native().rmsnorm_backward(dY, dH, H, gamma, rstd, dX, dgamma, workspace, _raw(stream)),
           "sp24_rmsnorm_backward")


def sp24_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Launches the bounded-wait self-test (reports SP24_ERR_TIMEOUT through
    sp24_device_status)."""
    _check(lib().sp24_selftest_wait_timeout(limit_ns, _stream(stream)),
           "sp24_selftest_wait_timeout")


def sp24_device_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status."""
    return lib().sp24_device_status(_stream(stream))
