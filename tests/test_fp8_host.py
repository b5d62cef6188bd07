"""CPU checks of the e4m3 and norm entry points: argument validation before any
CUDA call, sizes, and pins of their oracle functions."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import sp24_oracle as O
from structured_sparse_gemm_sp24_b200 import artifact as A
from structured_sparse_gemm_sp24_b200 import build as sp24_build
from structured_sparse_gemm_sp24_b200 import sp24 as B

FAKE = 0x10000   # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    sp24_build.build()
    return B.lib()


def caller(f, names, ok):
    def call(**kw):
        a = dict(zip(names, ok))
        assert set(kw) <= set(a)
        a.update(kw)
        return f(*[ctypes.c_float(v) if n == "eps" else v for n, v in a.items()])
    return call


def test_sizes(lib):
    assert B.sp24_scale_bytes(3, 1) == 12 and B.sp24_scale_bytes(3, 512) == 12
    assert B.sp24_scale_bytes(3, 513) == 24 and B.sp24_scale_bytes(86, 4096) == 86 * 32
    assert B.sp24_scale_bytes(0, 128) == 0 and B.sp24_scale_bytes(-1, 128) == 0
    assert lib.sp24_vals_bytes(64, 128, B.SP24_FP8) == 64 * 64
    ws = B.sp24_rmsnorm_backward_workspace_bytes
    assert ws(1, 16) == 64 and ws(0, 16) == 64 and ws(5, 4096) == 5 * 4096 * 4
    assert ws(1 << 40, 4096) == ws(100000, 4096) <= 4096 * 4 * 1024
    assert ws(5, B.SP24_NORM_MAX_K + 16) == 0 and ws(5, 0) == 0 and ws(-1, 16) == 0


def test_quantize_validation(lib):
    call = caller(lib.sp24_quantize_fp8, ["X", "M", "K", "x_dtype", "Xq", "e", "stream"],
                  (FAKE, 4, 128, B.SP24_BF16, FAKE, FAKE, None))
    assert call(M=-1) == B.SP24_ERR_ARG and call(K=0) == B.SP24_ERR_ARG
    assert call(x_dtype=B.SP24_INT8) == B.SP24_ERR_ARG and call(x_dtype=-1) == B.SP24_ERR_ARG
    for p in ("X", "Xq", "e"):
        assert call(**{p: None}) == B.SP24_ERR_ARG
        assert call(**{p: FAKE + 4}) == B.SP24_ERR_ALIGN
    assert call(K=120) == B.SP24_ERR_ALIGN
    assert call(M=0, X=None) == B.SP24_OK


def test_convert_validation(lib):
    call = caller(lib.sp24_prune_compress_fp8,
                  ["W", "N", "K", "mode", "norms", "mask_in", "mask_out", "vals", "meta", "e", "s"],
                  (FAKE, 8, 64, B.SP24_MAGNITUDE, None, None, None, FAKE, FAKE, FAKE, None))
    assert call(mode=3) == B.SP24_ERR_ARG and call(N=-1) == B.SP24_ERR_ARG
    assert call(mode=B.SP24_WANDA) == B.SP24_ERR_ARG           # no norms
    assert call(K=48) == B.SP24_ERR_ALIGN
    for p in ("W", "vals", "meta", "e"):
        assert call(**{p: None}) == B.SP24_ERR_ARG
        assert call(**{p: FAKE + 8}) == B.SP24_ERR_ALIGN
    for p in ("mask_in", "mask_out", "norms"):
        assert call(**{p: FAKE + 4}) == B.SP24_ERR_ALIGN
    assert call(N=0, W=None) == B.SP24_OK
    call = caller(lib.sp24_compress_fp8, ["W", "mask", "N", "K", "vals", "meta", "e", "s"],
                  (FAKE, FAKE, 8, 64, FAKE, FAKE, FAKE, None))
    assert call(mask=None) == B.SP24_ERR_ARG and call(K=40) == B.SP24_ERR_ALIGN
    assert call(mask=FAKE + 1) == B.SP24_ERR_ALIGN and call(N=0) == B.SP24_OK


def test_gemm_validation(lib):
    call = caller(lib.sp24_gemm_fp8,
                  ["X", "e_x", "M", "K", "vals", "meta", "e_w", "N", "out", "Y", "s"],
                  (FAKE, FAKE, 4, 128, FAKE, FAKE, FAKE, 64, B.SP24_OUT_BF16, FAKE, None))
    for out in (B.SP24_OUT_INT8, B.SP24_OUT_INT32, 9, -1):
        assert call(out=out) == B.SP24_ERR_ARG
    for p in ("X", "e_x", "vals", "meta", "e_w", "Y"):
        assert call(**{p: None}) == B.SP24_ERR_ARG
        assert call(**{p: FAKE + 8}) == B.SP24_ERR_ALIGN
    assert call(K=16) == B.SP24_ERR_ALIGN and call(K=144) == B.SP24_ERR_ALIGN
    assert call(N=60) == B.SP24_ERR_ALIGN
    assert call(M=1 << 31) == B.SP24_ERR_UNSUPPORTED
    assert call(N=1 << 32) == B.SP24_ERR_UNSUPPORTED
    assert call(M=0, X=None) == B.SP24_OK and call(N=0, vals=None) == B.SP24_OK
    # the other product still refuses the e4m3 type
    assert lib.sp24_gemm(FAKE, 16, 128, FAKE, FAKE, 16, B.SP24_FP8, None, None, B.SP24_OUT_BF16,
                         None, FAKE, None) == B.SP24_ERR_ARG


def test_norm_validation(lib):
    call = caller(lib.sp24_rmsnorm_quant,
                  ["X", "R", "gamma", "M", "K", "x_dtype", "eps", "out", "s_x", "H", "Y", "e",
                   "rstd", "s"],
                  (FAKE, None, FAKE, 4, 128, B.SP24_BF16, 1e-6, B.SP24_FP8, None, None, FAKE, FAKE,
                   None, None))
    assert call(M=-1) == B.SP24_ERR_ARG and call(K=0) == B.SP24_ERR_ARG
    assert call(x_dtype=B.SP24_FP8) == B.SP24_ERR_ARG and call(out=B.SP24_F32) == B.SP24_ERR_ARG
    assert call(eps=-1.0) == B.SP24_ERR_ARG and call(eps=float("nan")) == B.SP24_ERR_ARG
    assert call(e=None) == B.SP24_ERR_ARG                        # e4m3 needs its scales
    assert call(out=B.SP24_INT8) == B.SP24_ERR_ARG               # int8 its scale
    assert call(K=136) == B.SP24_ERR_ALIGN
    assert call(K=B.SP24_NORM_MAX_K + 16) == B.SP24_ERR_UNSUPPORTED
    for p in ("X", "gamma", "Y"):
        assert call(**{p: None}) == B.SP24_ERR_ARG
    for p in ("X", "R", "gamma", "H", "Y", "e"):
        assert call(**{p: FAKE + 8}) == B.SP24_ERR_ALIGN
    assert call(M=0, X=None) == B.SP24_OK


def test_norm_backward_validation(lib):
    big = 1 << 40
    call = caller(lib.sp24_rmsnorm_backward,
                  ["dY", "dH", "H", "gamma", "rstd", "M", "K", "x_dtype", "dX", "dgamma", "ws",
                   "bytes", "s"],
                  (FAKE, None, FAKE, FAKE, FAKE, 4, 128, B.SP24_BF16, FAKE, FAKE, FAKE, big, None))
    assert call(x_dtype=B.SP24_INT8) == B.SP24_ERR_ARG and call(M=-1) == B.SP24_ERR_ARG
    for p in ("dY", "H", "gamma", "rstd", "dX", "dgamma", "ws"):
        assert call(**{p: None}) == B.SP24_ERR_ARG
    assert call(bytes=4 * 128 * 4 - 1) == B.SP24_ERR_ARG
    assert call(K=136) == B.SP24_ERR_ALIGN and call(dH=FAKE + 2) == B.SP24_ERR_ALIGN
    assert call(dgamma=FAKE + 4) == B.SP24_ERR_ALIGN and call(ws=FAKE + 8) == B.SP24_ERR_ALIGN
    assert call(K=B.SP24_NORM_MAX_K + 16) == B.SP24_ERR_UNSUPPORTED


# ------------------------------------------------------ compressed-weight files
def test_fp8_weight_file_round_trip(tmp_path, lib):
    n, k = 130, 544
    g = torch.Generator().manual_seed(1)
    u8 = lambda *shape: torch.randint(0, 256, shape, dtype=torch.uint8, generator=g)  # noqa: E731
    vals = u8(n, k // 2).view(torch.float8_e4m3fn)
    meta = u8(B.sp24_meta_bytes(n, k))
    e_w = u8(2, 8).view(torch.float8_e8m0fnu)
    p = tmp_path / "w.sp24"
    A.save_compressed(str(p), vals, meta, n, k, B.SP24_FP8, e_w)
    assert p.stat().st_size == 64 + n * k // 2 + B.sp24_meta_bytes(n, k) + 16
    w = A.load_compressed(str(p))
    assert (w.n, w.k, w.dtype) == (n, k, B.SP24_FP8)
    assert w.vals.dtype == torch.float8_e4m3fn and w.vals.shape == (n, k // 2)
    assert w.s_w.dtype == torch.float8_e8m0fnu and w.s_w.shape == (2, 8)
    assert torch.equal(w.vals.view(torch.uint8), vals.view(torch.uint8))
    assert torch.equal(w.meta, meta)
    assert torch.equal(w.s_w.view(torch.uint8), e_w.view(torch.uint8))
    A.save_compressed(str(p), vals, meta, n, k, B.SP24_FP8, e_w.view(torch.uint8))   # bytes as well
    assert torch.equal(A.load_compressed(str(p)).s_w.view(torch.uint8), e_w.view(torch.uint8))
    with pytest.raises(ValueError):
        A.save_compressed(str(p), vals, meta, n, k, B.SP24_FP8)                       # no scales
    with pytest.raises(ValueError):
        A.save_compressed(str(p), vals, meta, n, k, B.SP24_FP8, torch.ones(16))       # float scales
    with pytest.raises(ValueError):
        A.save_compressed(str(p), vals, meta, n, k, B.SP24_FP8, e_w[:1])
    p.write_bytes(p.read_bytes()[:-1])
    with pytest.raises(ValueError):
        A.load_compressed(str(p))


# ------------------------------------------------------------- oracle pins
def test_e4m3_round_is_the_nearest_code():
    """Against every finite code (torch's decoding), halfway points to the even
    code."""
    codes = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert codes[-1] == 448 and codes[1] == 2.0 ** -9
    np.testing.assert_array_equal(O.e4m3_round(codes), codes)
    mid = (codes[:-1] + codes[1:]) / 2
    even = np.where(np.arange(len(mid)) % 2 == 0, codes[:-1], codes[1:])
    np.testing.assert_array_equal(O.e4m3_round(mid), even)
    np.testing.assert_array_equal(O.e4m3_round(-mid), -even)
    np.testing.assert_array_equal(O.e4m3_round(mid * (1 - 1e-12)), codes[:-1])
    np.testing.assert_array_equal(O.e4m3_round(mid * (1 + 1e-12)), codes[1:])


def test_block_exponent_by_hand():
    assert list(O.block_exponent(np.array([0.0, 448, 448.5, 1.75, 1.0, 2.0, 224.0, 2.0 ** -149]))) == \
        [0, 0, 1, -8, -8, -7, -1, -126]
    e = O.block_exponent(np.array([3e38]))[0]
    assert 448 * 2.0 ** e >= 3e38 > 448 * 2.0 ** (e - 1)


def test_fp8_gemm_and_norm_oracles_by_brute_force():
    rng = np.random.default_rng(0)
    m, n, k = 3, 130, 160
    xq, wq = rng.integers(-3, 4, (m, k)) * 1.0, rng.integers(-3, 4, (n, k)) * 1.0
    ex, ew = rng.integers(-3, 4, (m, 2)), rng.integers(-3, 4, (2, 2))
    y, a = O.fp8_gemm(xq, ex, wq, ew)
    for i, j in [(0, 0), (2, 127), (1, 128), (2, 129)]:
        t = [xq[i, c] * wq[j, c] * 2.0 ** (ex[i, c // 128] + ew[j // 128, c // 128]) for c in range(k)]
        assert y[i, j] == sum(t) and a[i, j] == sum(abs(v) for v in t)
    h, g = rng.standard_normal((2, 8)), rng.standard_normal(8)
    yy, s = O.rmsnorm(h, g, 0.5)
    assert np.isclose(yy[1, 3], h[1, 3] * g[3] / np.sqrt(sum(v * v for v in h[1]) / 8 + 0.5), rtol=1e-14)
    dy = rng.standard_normal((2, 8))
    dx, dg = O.rmsnorm_backward(dy, h, g, s)
    for i, j in [(0, 0), (1, 7)]:
        p, q = h.copy(), h.copy()
        p[i, j] += 1e-6
        q[i, j] -= 1e-6
        d = ((O.rmsnorm(p, g, 0.5)[0] - O.rmsnorm(q, g, 0.5)[0]) * dy).sum() / 2e-6
        assert abs(d - dx[i, j]) < 1e-8
    p, q = g.copy(), g.copy()
    p[2] += 1e-6
    q[2] -= 1e-6
    assert abs(((O.rmsnorm(h, p, 0.5)[0] - O.rmsnorm(h, q, 0.5)[0]) * dy).sum() / 2e-6 - dg[2]) < 1e-8


def test_binding_refuses_before_any_cuda_call(lib):
    n = B.native()
    cpu = torch.zeros(4, 128)
    with pytest.raises(ValueError, match="X must be a CUDA tensor"):
        n.quantize_fp8(cpu, cpu, cpu, None)
    with pytest.raises(ValueError, match="X must be a matrix"):
        n.quantize_fp8(torch.zeros(4), cpu, cpu, None)
    with pytest.raises(ValueError, match="H must be a tensor"):
        n.rmsnorm_backward(cpu, None, None, cpu, cpu, cpu, cpu, cpu, None)
    with pytest.raises(ValueError, match="W must be a CUDA tensor"):
        B.sp24_prune_compress_fp8(cpu, B.SP24_MAGNITUDE, None, None, None, cpu, cpu, cpu)
    with pytest.raises(ValueError, match="unknown type code"):
        n.new_empty(cpu, 7, 1)
    with pytest.raises(RuntimeError, match="wrong number of arguments"):
        n.gemm_fp8(cpu)
    with pytest.raises(TypeError):
        n.new_empty(cpu, 1, 2.5)


def test_binding_allocations(lib):
    n = B.native()
    like = torch.zeros(2, 3, dtype=torch.bfloat16, requires_grad=True)
    types = [torch.bfloat16, torch.int8, torch.bfloat16, torch.float32, torch.float8_e4m3fn,
             torch.float8_e8m0fnu, torch.uint8]
    for code, t in enumerate(types):
        e = n.new_empty(like, code, 3, 5)
        assert e.dtype == t and e.shape == (3, 5) and e.is_contiguous() and not e.requires_grad
    assert n.new_empty(like, 3, 0).shape == (0,)
    assert n.new_meta(like, 65, 192).numel() == B.sp24_meta_bytes(65, 192)
    assert n.new_workspace(like, 7, 4096).numel() == B.sp24_rmsnorm_backward_workspace_bytes(7, 4096)


def test_binding_missing_is_an_error(lib, monkeypatch):
    import sys
    import structured_sparse_gemm_sp24_b200 as pkg
    monkeypatch.setattr(B, "_NATIVE", None)
    monkeypatch.setitem(sys.modules, pkg.__name__ + "._binding", None)
    monkeypatch.delattr(pkg, "_binding", raising=False)
    with pytest.raises(RuntimeError, match="_binding.so"):
        B.native()
