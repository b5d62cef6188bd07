"""GPU tests of the e4m3 and norm entry points at the far ends of their ranges."""
import numpy as np
import pytest
import torch

from oracle import sp24_oracle as O
from structured_sparse_gemm_sp24_b200 import pipeline as P
from structured_sparse_gemm_sp24_b200 import sp24 as B
from tests.test_gpu_fp8 import (BF, F32, assert_product, exps, f64, product_case,  # noqa: F401
                                rand, _device)

pytestmark = pytest.mark.gpu


# ------------------------------------------------ more tiles than 16 bits number
MANY = 65535 * 128                             # rows whose 128-tiles a launch still numbers


@pytest.mark.parametrize("m,n", [(MANY + 1, 64), (MANY + 1, 200), (MANY + 1, 256), (128, MANY + 8),
                                 (255, MANY + 8), (1, MANY + 8), (256, MANY + 8)])
def test_plan_of_more_tiles_than_a_grid_numbers(m, n):
    p = B.sp24_gemm_plan(m, n, 128, B.SP24_FP8)
    assert p["kernel"] in ("pair256", "pair240", "pair224") and p["split_k"] == 1


@pytest.mark.parametrize("m,n", [(MANY, 64), (MANY, 248), (128, MANY), (255, MANY), (1, MANY)])
def test_plan_of_the_last_tiles_a_grid_numbers(m, n):
    assert B.sp24_gemm_plan(m, n, 128, B.SP24_FP8)["kernel"] == "splitk"


def test_gemm_of_more_token_tiles_than_a_grid_numbers():
    m, n, k, t = MANY + 1, 64, 32, 300
    w = rand((n, k), BF, 1, 0.02, 0.5)
    vals, meta, e_w = P.prune_compress_fp8(w.cuda())
    x = torch.zeros((m, k), dtype=BF, device="cuda")
    tail = rand((t, k), BF, 2)
    x[-t:] = tail.cuda()
    xq, e_x = P.quantize_fp8(x)
    del x
    out = P.gemm_fp8(xq, e_x, vals, meta, e_w, n)
    assert B.sp24_device_status() == B.SP24_OK
    wq, we = O.fp8_weight(f64(w), O.prune(f64(w), O.MAGNITUDE, 2))
    y, a = O.fp8_gemm(f64(xq[-t:]), exps(e_x[-t:])[:, :1], wq, we)
    assert_product(out[-t:], y, a, k, True)
    assert not out[:-t].any()


@pytest.mark.parametrize("m", [1, 130])
def test_gemm_of_more_row_tiles_than_a_grid_numbers(m):
    n, k, t = MANY + 8, 32, 520                # the last rows of W in whole blocks and a part
    w = torch.zeros((n, k), dtype=BF, device="cuda")
    tail = rand((t, k), BF, 1, 0.02, 0.5)
    w[-t:] = tail.cuda()
    vals, meta, e_w = P.prune_compress_fp8(w)
    del w
    xq, e_x = P.quantize_fp8(rand((m, k), F32, 2).cuda())
    out = P.gemm_fp8(xq, e_x, vals, meta, e_w, n)
    assert B.sp24_device_status() == B.SP24_OK
    dense = np.zeros((t, k))                   # n is 8 past whole blocks: so is the tail
    dense[:] = f64(tail)
    wq, we = O.fp8_weight(dense, O.prune(dense, O.MAGNITUDE, 2))
    y, a = O.fp8_gemm(f64(xq), exps(e_x)[:, :1], wq, we)
    assert_product(out[:, -t:], y, a, k, True)
    assert not out[:, :-t].any()
