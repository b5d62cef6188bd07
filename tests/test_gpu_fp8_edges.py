"""GPU tests of the e4m3 and norm entry points at the far ends of their ranges."""
import numpy as np
import pytest
import torch

from oracle import sp24_oracle as O
from structured_sparse_gemm_sp24_b200 import pipeline as P
from structured_sparse_gemm_sp24_b200 import sp24 as B
from tests.test_gpu_fp8 import (BF, EPS, F32, HALF_BF16, NORM_REL, _device,  # noqa: F401
                                assert_back, assert_codes_near, assert_product, back_inputs, exps,
                                f64, product_case, rand, stored_sum)

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


# ----------------------------------------------------- columns past 32 bits
def test_quantize_of_rows_longer_than_32_bits():
    """The last block ends inside its 128 columns: what lies behind the row is
    neither read into its scale nor written."""
    k = 2 ** 32 + 16
    x = torch.zeros(k + 256, dtype=BF, device="cuda")
    x[k:] = 300.0                               # behind the row: would raise the scale
    tail = rand((1, 144), BF, 1)
    x[k - 144:k] = tail[0].cuda()
    codes = torch.full((k + 256,), 0x55, dtype=torch.uint8, device="cuda")
    q, e = P.quantize_fp8(x[:k].view(1, k), out=codes[:k].view(torch.float8_e4m3fn).view(1, k))
    assert B.sp24_device_status() == B.SP24_OK
    want_q, want_e = O.fp8_rows(f64(tail))       # k - 144 = 2^32 - 128: whole blocks before
    np.testing.assert_array_equal(f64(q[:, -144:]), want_q)
    ex = exps(e)[0]
    blocks = (k + 127) // 128
    np.testing.assert_array_equal(ex[blocks - 2:blocks], want_e[0])
    assert (ex[:blocks - 2] == 0).all() and (ex[blocks:] == 0).all()
    assert not codes[:k - 144].any() and (codes[k:] == 0x55).all()


# -------------------------------------------- rows whose 1 / rms is exact
def exact_root_rows(m, k, rng):
    """Whole numbers up to 255 of both signs whose squares sum to k * 64^2: every
    partial sum is exact in fp32 and 1 / rms = 2^-6."""
    h = np.zeros((m, k), dtype=np.int64)
    for i in range(m):
        while True:
            a = rng.integers(1, 110, k)
            rest = k * 4096 - int((a[:-4] ** 2).sum())
            p = np.arange(256) ** 2
            two = (p[:, None] + p[None, :]).ravel()
            first = np.full(2 * 255 ** 2 + 1, -1)
            first[two] = np.arange(two.size)
            for t in range(max(rest - 2 * 255 ** 2, 0), min(rest, 2 * 255 ** 2) + 1):
                if first[t] >= 0 and first[rest - t] >= 0:
                    a[-4:] = [first[t] // 256, first[t] % 256, first[rest - t] // 256,
                              first[rest - t] % 256]
                    break
            else:
                continue
            break
        h[i] = a * rng.choice([-1, 1], k)
        assert (h[i] ** 2).sum() == k * 4096
    return h


@pytest.mark.parametrize("m,k", [(3, 256), (2, 512), (3, 2048), (2, 4096), (2, 16384)])
def test_norm_rounds_products_of_an_exact_root_once(m, k):
    """Float32 products a little above a tie of the code or above 448 * 2^e, with
    an s that has no remainder: the part that fp32 cannot hold still decides."""
    rng = np.random.default_rng(k)
    h = exact_root_rows(m, k, rng)
    h[1:] = h[0]                               # (one gamma aims at every row)
    h[1:, :k // 2] *= -1
    top = np.where(np.arange(k) % 128 == 5, 448.0 * 2.0 ** (np.arange(k) // 128 % 3), 0.0)
    tie = np.array([17.0, 19.0, 21.0, 23.0, 25.0, 27.0, 29.0, 31.0])[rng.integers(0, 8, k)]
    want = np.where(top > 0, top, tie * 2.0 ** rng.integers(-3, 3, k))
    mag = np.maximum(np.abs(h[0]), 1)
    gamma = (want * 64 / mag).astype(np.float32)
    low = gamma.astype(np.float64) * mag < want * 64
    gamma = np.where(low, np.nextafter(gamma, np.float32(np.inf)), gamma).astype(np.float32)
    y = h * gamma.astype(np.float64) / 64
    inexact = y.astype(np.float32).astype(np.float64) != y
    assert inexact.mean() > 0.3
    x = torch.from_numpy(h.astype(np.float32)).cuda()
    o = P.rmsnorm_quant(x, torch.from_numpy(gamma).cuda(), eps=0.0, want_rstd=True)
    assert o.rstd.cpu().tolist() == [2.0 ** -6] * m
    want_q, want_e = O.fp8_rows(y)
    np.testing.assert_array_equal(exps(o.e_y)[:, :k // 128], want_e)
    np.testing.assert_array_equal(f64(o.y), want_q)
    # the same sum of two streams: stored over either, apart, and not at all
    g = torch.from_numpy(gamma).cuda()
    r = torch.from_numpy(rng.integers(-64, 65, (m, k)).astype(np.float32)).cuda()
    for target in ("x", "r", "new", "none"):
        a, b = x - r, r.clone()
        q, e = torch.empty_like(o.y), torch.empty_like(o.e_y)
        h = {"x": a, "r": b, "new": torch.empty_like(a), "none": None}[target]
        B.sp24_rmsnorm_quant(a, b, g, 0.0, B.SP24_FP8, None, h, q, e, None)
        assert torch.equal(q.view(torch.uint8), o.y.view(torch.uint8))
        assert torch.equal(e.view(torch.uint8), o.e_y.view(torch.uint8))
        assert h is None or torch.equal(h, x)


# ------------------------------------------------ the range that sp24.h states
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("k", [512, 2048])
def test_norm_range_of_products_and_squares(k, dt):
    """A product h * gamma past float32 makes its block NaN and no other; squares
    past it, a row of zeros."""
    x = torch.ones((3, k), dtype=dt)
    x[1] = 2.0 ** 30
    x[2] = 2.0 ** 70                           # squares past 2^128
    gamma = torch.ones(k, dtype=dt)
    gamma[3] = 2.0 ** 99                       # y of 2^99; times 2^30 past 2^128
    o = P.rmsnorm_quant(x.cuda(), gamma.cuda(), eps=0.0, want_rstd=True)
    assert o.rstd.cpu().tolist() == [1.0, 2.0 ** -30, 0.0]
    by, q = o.e_y.view(torch.uint8).cpu(), o.y.view(torch.uint8).cpu()
    assert exps(o.e_y)[0, 0] == 99 - 8 and f64(o.y)[0, 3] == 256
    # (2^30 and 2^70 times 2^99 both pass 2^128: rows 1 and 2)
    assert (by[1:, 0] == 255).all() and (q[1:, :128] == 0x7F).all()
    assert (exps(o.e_y)[:2, 1:k // 128] == -8).all() and (f64(o.y)[:2, 128:] == 256).all()
    assert (f64(o.y)[2, 128:] == 0).all()


# ------------------------------------------------------------------- errors
def test_an_allocation_that_fails_raises_as_torch_does():
    vals, meta, e_w = P.prune_compress_fp8(torch.zeros((64, 256), dtype=BF, device="cuda"))
    xq, e_x = P.quantize_fp8(torch.zeros((1, 256), dtype=BF, device="cuda"))
    with pytest.raises(torch.OutOfMemoryError, match="out of memory") as e:
        P.gemm_fp8(xq, e_x, vals, meta, e_w, 1 << 48)         # an output of 2^49 bytes
    assert "frame #" not in str(e.value)
    assert B.sp24_device_status() == B.SP24_OK
    assert P.gemm_fp8(xq, e_x, vals, meta, e_w, 64).shape == (1, 64)


def test_a_forced_split_keeps_one_cta_an_sm(monkeypatch):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for m in (1, 20, 40, 100):
        for tiles in (3, 40, 80, sms + 2):
            n = 128 * tiles
            for split in range(1, 9):
                monkeypatch.setenv("SP24_SPLITK", str(split))
                p = B.sp24_gemm_plan(m, n, 4096, B.SP24_FP8)
                assert p["kernel"] == "splitk" and p["split_k"] in (1, 2, 4, 8)
                assert p["split_k"] <= split and (p["ctas"] <= sms or p["split_k"] == 1)
    # a split that would share SMs is lowered, and the product is right
    xq, e_x, vals, meta, e_w, y, a = product_case(20, 128 * 40, 1312, 3)
    for split in (1, 2, 4, 8):
        monkeypatch.setenv("SP24_SPLITK", str(split))
        out = P.gemm_fp8(xq, e_x, vals, meta, e_w, 128 * 40)
        assert B.sp24_device_status() == B.SP24_OK
        assert_product(out, y, a, 1312, True)


# -------------------------------- several rows a warp, and a group, one by one
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("k", [128, 256, 512])
def test_norm_of_more_short_rows_than_warps(k, res, dt):
    """Rows of one warp each, so many that every warp takes several (the next one
    loaded ahead while this one's h is stored over x or over r)."""
    m = 20003
    x = rand((m, k), dt, k)
    r = rand((m, k), dt, k + 1) if res else None
    gamma = (1 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(k))).to(dt)
    h = stored_sum(x, r)
    y, s = O.rmsnorm(f64(h), f64(gamma), EPS)
    for target in (("x", "r", None) if res else (None,)):
        a, b = x.cuda(), None if r is None else r.cuda()
        o = P.rmsnorm_quant(a, gamma.cuda(), b, EPS, want_rstd=True,
                            out_sum={"x": a, "r": b, None: None}[target])
        assert torch.equal(o.h.cpu(), h)
        np.testing.assert_allclose(f64(o.rstd), s, rtol=NORM_REL)
        assert_codes_near(o.y, o.e_y, y, NORM_REL, k)
    rc = None if r is None else r.cuda()
    o = P.rmsnorm_quant(x.cuda(), gamma.cuda(), rc, EPS, B.SP24_BF16)
    assert (np.abs(f64(o.y) - y) <= (HALF_BF16 + 2 * NORM_REL) * np.abs(y)).all()
    s_x = torch.tensor([0.037], device="cuda")
    o = P.rmsnorm_quant(x.cuda(), gamma.cuda(), rc, EPS, B.SP24_INT8, s_x=s_x)
    v = y / float(s_x.double().cpu())
    rel = NORM_REL + 2.0 ** -24
    lo, hi = np.rint(np.clip(v * (1 - rel), -127, 127)), np.rint(np.clip(v * (1 + rel), -127, 127))
    got = o.y.cpu().numpy().astype(np.float64)
    assert ((got == lo) | (got == hi)).all()
    assert B.sp24_device_status() == B.SP24_OK


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("m,k", [(8192, 768), (8191, 272), (5001, 1040), (3000, 2048), (3000, 4096)])
def test_norm_backward_of_several_rows_a_group(m, k, dt):
    """Groups of threads that take several rows each, an uneven number among them."""
    h, gamma, dy, dh, rstd = back_inputs(m, k, dt, m + k)
    for d in (None, dh):
        dx, dg = P.rmsnorm_backward(dy.cuda(), h.cuda(), gamma.cuda(), rstd.cuda(),
                                    dH=None if d is None else d.cuda())
        assert_back(dx, dg, h, gamma, dy, d, rstd, dt is BF)
    assert B.sp24_device_status() == B.SP24_OK


def test_quantize_without_a_scale_is_an_argument_error():
    x = torch.zeros((4, 256), device="cuda")
    with pytest.raises(B.Sp24Error) as e:
        P.quantize(x, None)
    assert e.value.status == B.SP24_ERR_ARG
    with pytest.raises(ValueError, match="float32"):
        P.quantize(x.to(BF), torch.ones(1, device="cuda"))
    with pytest.raises(ValueError, match="float32"):
        P.act_scale(x.to(BF))
