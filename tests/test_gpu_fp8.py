"""GPU parity of the e4m3 layer and the RMS norm against the 64-bit oracle.

Quantisation and weight conversion round nothing but the code itself, so their
outputs equal the oracle's bit for bit.  Where arithmetic in fp32 comes first
(the norm), a code may differ only where the exact value lies within that
arithmetic's error of a rounding border.  Bounds:

* norm output y: the row sum has at most 8 * NV + 5 + 32 <= 70 roundings of
  positive terms, halved by the square root; mean, eps, the root and the
  products add at most 6: 41 half-steps of 2^-24, taken as NORM_REL = 64 * 2^-24;
* gemm: the fp32 sum takes K / 64 additions, each off by at most one unit
  2^-23 of a partial sum of at most sum |x w|, and as much again inside the
  instructions: SUM_REL(K) = 2 * (K / 64 + 1) * 2^-23 of sum |x w|; a bf16
  output adds half a step, 2^-8 of the value;
* backward: fp32 sums of up to 8 * NV + 5 + 32 (row) terms.
"""
import numpy as np
import pytest
import torch

from oracle import sp24_oracle as O
from structured_sparse_gemm_sp24_b200 import pipeline as P
from structured_sparse_gemm_sp24_b200 import sp24 as B
from tests import meta_layout as L

pytestmark = pytest.mark.gpu

NORM_REL = 64 * 2.0 ** -24
HALF_BF16 = 2.0 ** -8
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


def sum_rel(k):
    return 2 * (k / 64 + 1) * 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    B.lib()
    assert B.sp24_device_status() == B.SP24_OK


def f64(t):
    return t.detach().to(torch.float32 if t.element_size() == 1 else t.dtype).double().cpu().numpy()


def exps(e):
    """Exponents of a scale tensor (padding included)."""
    return e.view(torch.uint8).cpu().numpy().astype(np.int64) - 127


def rand(shape, dt, seed, scale=1.0, spread=2.0):
    """Values whose blocks differ in size by powers of ten, zeros among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    x = x * torch.exp(spread * torch.randn((shape[0], 1), generator=g))
    x = torch.where(torch.rand(shape, generator=g) < 0.05, torch.zeros(()), x)
    return x.to(dt)


def assert_scales(e, want, k):
    """Scale bytes [rows, padded blocks]: the blocks', then ones."""
    got = exps(e)
    kb = (k + 127) // 128
    assert got.shape[1] == 4 * ((k + 511) // 512)
    np.testing.assert_array_equal(got[:, :kb], want)
    assert (got[:, kb:] == 0).all()


def assert_codes_near(q, e, y, rel, k):
    """e4m3 codes q and exponents e of values known to a relative error rel."""
    kb = (k + 127) // 128
    ex = exps(e)[:, :kb]
    assert (exps(e)[:, kb:] == 0).all()
    amax = np.stack([np.abs(y[:, 128 * b:128 * b + 128]).max(1) for b in range(kb)], 1)
    lo, hi = O.block_exponent(amax * (1 - rel)), O.block_exponent(amax * (1 + rel))
    assert ((ex == lo) | (ex == hi)).all()
    v = y * np.ldexp(1.0, -np.repeat(ex, 128, 1)[:, :k])
    v = np.clip(v, -448, 448)
    a, b = O.e4m3_round(v * (1 - rel)), O.e4m3_round(np.clip(v * (1 + rel), -448, 448))
    got = f64(q)
    assert ((got == a) | (got == b)).all()


# ------------------------------------------------------------- quantisation
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("m,k", [(1, 16), (1, 128), (3, 144), (5, 1040), (7, 4096), (2, 4112),
                                 (33, 768), (300, 272), (1, 11008), (9, 20480), (1000, 512)])
def test_quantize_is_exact(m, k, dt):
    x = rand((m, k), dt, m * 7 + k)
    q, e = P.quantize_fp8(x.cuda())
    want_q, want_e = O.fp8_rows(f64(x))
    assert_scales(e, want_e, k)
    np.testing.assert_array_equal(f64(q), want_q)
    assert B.sp24_device_status() == B.SP24_OK


def test_quantize_borders_and_specials():
    """Largest values on and next to 448 * 2^e, ties of the code, subnormal and
    empty blocks, infinities and NaN."""
    k = 128 * 10
    x = torch.zeros((2, k), dtype=F32)
    b = x.view(2, 10, 128)
    b[:, 0, 0] = 448.0
    b[:, 1, 5] = float(np.nextafter(np.float32(448.0), np.float32(1e9)))
    b[:, 2, 127] = -448.0 * 2.0 ** 40
    b[:, 3, :9] = torch.tensor([256.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 27.0, 21.0])
    b[:, 4, 0] = 1e-45                       # subnormal
    b[:, 5, 1] = float(np.finfo(np.float32).max)
    # block 6 stays empty
    b[1, 7, 3] = float("inf")
    b[1, 8, 4] = float("nan")
    b[1, 9, 0] = 1.0
    q, e = P.quantize_fp8(x.cuda())
    want_q, want_e = O.fp8_rows(f64(x[:1]))
    assert_scales(e[:1], want_e, k)
    np.testing.assert_array_equal(f64(q[:1]), want_q)
    by = e.view(torch.uint8).cpu()
    assert by[1, 7] == 255 and by[1, 8] == 255
    codes = q.view(torch.uint8).cpu().view(2, 10, 128)
    assert (codes[1, 7] == 0x7F).all() and (codes[1, 8] == 0x7F).all()
    assert torch.equal(codes[1, :7], codes[0, :7])      # neighbours untouched
    assert f64(q)[1, 9 * 128] == 256.0 and exps(e)[1, 9] == -8


def test_quantize_offsets_past_32_bits():
    m, k = 70001, 32768                       # 2.29e9 elements
    x = torch.zeros((m, k), dtype=BF, device="cuda")
    tail = rand((3, k), BF, 5).cuda()
    x[-3:] = tail
    q, e = P.quantize_fp8(x)
    want_q, want_e = O.fp8_rows(f64(tail))
    assert_scales(e[-3:], want_e, k)
    np.testing.assert_array_equal(f64(q[-3:]), want_q)
    assert int(q[:-3].view(torch.uint8).max()) == 0
    del x, q


# ------------------------------------------------------- weight conversion
def convert_ref(w, mode, norms, mask_in):
    wf = f64(w)
    if mask_in is not None:
        wf = np.where(mask_in, wf, 0.0)
    keep = O.select(O.scores(wf, mode, norms), 2)
    return keep, O.fp8_weight(f64(w), keep)


def gather_kept(dense, keep):
    return dense[keep].reshape(dense.shape[0], -1)


@pytest.mark.parametrize("mode", [O.MAGNITUDE, O.WANDA])
@pytest.mark.parametrize("n,k,masked", [(8, 32, False), (128, 128, False), (200, 416, True),
                                        (1, 512, False), (129, 1024, False), (256, 544, True),
                                        (16, 36896, False)])
def test_convert_is_exact(n, k, masked, mode):
    w = rand((n, k), BF, n + k, 0.02)
    norms = None
    if mode == O.WANDA:
        norms = np.abs(np.random.default_rng(k).standard_normal(k)) + 0.1
    m1 = None
    if masked:
        m1 = O.select(O.scores(f64(w), mode, norms), 3)
    dn = None if norms is None else torch.from_numpy(norms).cuda()
    dm = None if m1 is None else torch.from_numpy(O.pack_mask(m1)).cuda()
    vals, meta, e, mask = P.prune_compress_fp8(
        w.cuda(), B.SP24_WANDA if norms is not None else B.SP24_MAGNITUDE, dn, dm, want_mask=True)
    keep, (dense, we) = convert_ref(w, mode, norms, m1)
    np.testing.assert_array_equal(O.unpack_mask(mask.cpu().numpy(), k), keep)
    assert_scales(e, we, k)
    np.testing.assert_array_equal(f64(vals), gather_kept(dense, keep))
    _, rm = O.compress(f64(w), keep)
    np.testing.assert_array_equal(L.decode(meta.cpu().numpy(), n, k, L.INT8), rm)
    assert L.padding_is_valid(meta.cpu().numpy(), n, k, L.INT8)
    # the same from the mask
    vals2, meta2, e2 = P.compress_fp8(w.cuda(), mask)
    assert torch.equal(vals2.view(torch.uint8), vals.view(torch.uint8))
    assert torch.equal(meta2, meta)
    assert torch.equal(e2.view(torch.uint8), e.view(torch.uint8))
    assert B.sp24_device_status() == B.SP24_OK


def test_convert_of_an_infinite_weight():
    """The block of an infinity or NaN is NaN, its neighbours and mask are not."""
    w = rand((256, 256), BF, 3, 0.02)
    clean = P.prune_compress_fp8(w.cuda())
    w[130, 7] = float("inf")
    w[5, 200] = float("nan")
    vals, meta, e = P.prune_compress_fp8(w.cuda())
    by, q = e.view(torch.uint8).cpu(), vals.view(torch.uint8).cpu()
    cq, cb = clean[0].view(torch.uint8).cpu(), clean[2].view(torch.uint8).cpu()
    assert by[1, 0] == 255 and by[0, 1] == 255 and by[0, 0] == cb[0, 0] and by[1, 1] == cb[1, 1]
    assert (q[128:, :64] == 0x7F).all() and (q[:128, 64:] == 0x7F).all()
    assert torch.equal(q[:128, :64], cq[:128, :64]) and torch.equal(q[128:, 64:], cq[128:, 64:])


def test_compress_reports_a_bad_group():
    w = rand((64, 64), BF, 3).cuda()
    mask = P.prune(w)
    mask[5, 3] = 0x37                         # three kept, two kept
    P.compress_fp8(w, mask)
    assert B.sp24_device_status() == B.SP24_ERR_PATTERN
    assert B.sp24_device_status() == B.SP24_OK


# --------------------------------------------------------------------- gemm
def product_case(m, n, k, seed=0):
    w = rand((n, k), BF, seed + 1, 0.02, 1.0)
    x = rand((m, k), F32, seed + 2, 1.0, 1.0)
    vals, meta, e_w = P.prune_compress_fp8(w.cuda())
    xq, e_x = P.quantize_fp8(x.cuda())
    keep = O.prune(f64(w), O.MAGNITUDE, 2)
    wq, we = O.fp8_weight(f64(w), keep)
    kb = (k + 127) // 128
    y, a = O.fp8_gemm(f64(xq), exps(e_x)[:, :kb], wq, we)
    return xq, e_x, vals, meta, e_w, y, a


def assert_product(got, y, a, k, bf16):
    d = np.abs(f64(got) - y)
    bound = sum_rel(k) * a + (HALF_BF16 * (np.abs(y) + sum_rel(k) * a) if bf16 else 0.0)
    bad = d > bound
    assert not bad.any(), (int(bad.sum()), d[bad][:3], y[bad][:3], bound[bad][:3])


GEMM_SIZES = [(1, 8, 32), (1, 128, 512), (1, 136, 544), (2, 1000, 1280), (16, 384, 4096),
              (17, 264, 800), (33, 256, 768), (64, 512, 256), (100, 72, 1056), (129, 640, 160),
              (128, 11008, 256), (200, 128, 4128), (3, 2048, 11008)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", GEMM_SIZES)
def test_gemm(m, n, k, kind):
    xq, e_x, vals, meta, e_w, y, a = product_case(m, n, k, m + n + k)
    out = P.gemm_fp8(xq, e_x, vals, meta, e_w, n,
                     B.SP24_OUT_F32 if kind == "f32" else B.SP24_OUT_BF16)
    assert B.sp24_device_status() == B.SP24_OK
    assert_product(out, y, a, k, kind == "bf16")


@pytest.mark.parametrize("impl", ["pair256", "pair240", "pair224", "splitk"])
@pytest.mark.parametrize("m,n,k", [(2500, 1056, 1312), (1233, 2056, 256), (700, 4104, 640)])
def test_gemm_kernels(m, n, k, impl, monkeypatch):
    """Every kernel on the same problem, both output types: several tiles per
    CTA, ragged sides, odd numbers of stages."""
    xq, e_x, vals, meta, e_w, y, a = product_case(m, n, k, 5)
    monkeypatch.setenv("SP24_GEMM_IMPL", impl)
    assert B.sp24_gemm_plan(m, n, k, B.SP24_FP8)["kernel"] == impl
    for kind in (B.SP24_OUT_BF16, B.SP24_OUT_F32):
        out = P.gemm_fp8(xq, e_x, vals, meta, e_w, n, kind)
        assert B.sp24_device_status() == B.SP24_OK
        assert_product(out, y, a, k, kind == B.SP24_OUT_BF16)


@pytest.mark.parametrize("split", [1, 2, 4, 8])
@pytest.mark.parametrize("m,n,k", [(5, 136, 2560), (20, 264, 2304), (40, 128, 4352), (100, 200, 3328)])
def test_gemm_splits(m, n, k, split, monkeypatch):
    """Every split, K ranges that start inside a scale word among them."""
    xq, e_x, vals, meta, e_w, y, a = product_case(m, n, k, 9)
    monkeypatch.setenv("SP24_SPLITK", str(split))
    out = P.gemm_fp8(xq, e_x, vals, meta, e_w, n, B.SP24_OUT_F32)
    assert B.sp24_device_status() == B.SP24_OK
    assert_product(out, y, a, k, False)


@pytest.mark.parametrize("m", [9, 30, 60, 110])
def test_gemm_more_row_tiles_than_sms(m):
    """Several CTAs on an SM (the small ring), every token tile width; the sizes
    are the plan's, so is the kernel."""
    n, k = 19080, 1312                        # 150 row tiles
    assert B.sp24_gemm_plan(m, n, k, B.SP24_FP8)["kernel"] == "splitk"
    xq, e_x, vals, meta, e_w, y, a = product_case(m, n, k, m)
    out = P.gemm_fp8(xq, e_x, vals, meta, e_w, n)
    assert B.sp24_device_status() == B.SP24_OK
    assert_product(out, y, a, k, True)


def test_gemm_same_bits_again_and_back_to_back():
    """Persistent tiles, many launches in a row: the same bits each time."""
    m, n, k = 4096, 2304, 2048
    w = P.prune_compress_fp8(rand((n, k), BF, 1, 0.02, 0.5).cuda())
    xq, e_x = P.quantize_fp8(rand((m, k), F32, 2).cuda())
    first = P.gemm_fp8(xq, e_x, *w, n)
    outs = [P.gemm_fp8(xq, e_x, *w, n) for _ in range(40)]
    assert B.sp24_device_status() == B.SP24_OK
    assert all(torch.equal(first, o) for o in outs)


def test_plan_uses_only_the_fp8_kernels(monkeypatch):
    for m, n, k in [(1, 4096, 4096), (64, 11008, 4096), (2048, 11008, 4096), (8192, 4096, 4096),
                    (300, 128, 512), (100000, 64, 256)]:
        p = B.sp24_gemm_plan(m, n, k, B.SP24_FP8)
        assert p["kernel"] in ("splitk", "pair256", "pair240", "pair224")
        assert p["split_k"] in (1, 2, 4, 8)
    for impl in ("single", "pair192", "pair128"):
        monkeypatch.setenv("SP24_GEMM_IMPL", impl)
        assert B.sp24_gemm_plan(4096, 4096, 4096, B.SP24_FP8)["kernel"].startswith("pair2")


def test_gemm_of_exact_sums_is_exact():
    """Small whole numbers with power-of-two scales: every sum is exact in fp32,
    so any wrong scale, position or K range shows."""
    m, n, k = 260, 520, 2176
    g = torch.Generator().manual_seed(1)
    kb, cols = 17, 20
    x = torch.randint(-3, 4, (m, k), generator=g).float()
    ex = torch.full((m, cols), 127, dtype=torch.uint8)
    ex[:, :kb] = torch.randint(125, 130, (m, kb), generator=g).to(torch.uint8)
    w = torch.randint(-3, 4, (n, k), generator=g).float().to(BF)
    mask = P.prune(w.cuda())
    vals, meta, _ = P.compress_fp8(w.cuda(), mask)
    keep = O.unpack_mask(mask.cpu().numpy(), k)
    kept = gather_kept(f64(w), keep)          # codes with our own scales
    vals = torch.from_numpy(kept).float().to(torch.float8_e4m3fn).cuda()
    ew = torch.full((5, cols), 127, dtype=torch.uint8)
    ew[:, :kb] = torch.randint(125, 130, (5, kb), generator=g).to(torch.uint8)
    y, _ = O.fp8_gemm(f64(x), ex.numpy()[:, :kb].astype(np.int64) - 127,
                      np.where(keep, f64(w), 0.0), ew.numpy()[:, :kb].astype(np.int64) - 127)
    xq = x.to(torch.float8_e4m3fn).cuda()
    out = P.gemm_fp8(xq, ex.cuda(), vals, meta, ew.cuda(), n, B.SP24_OUT_F32)
    np.testing.assert_array_equal(f64(out), y)
    for t in (1, 15, 50, 128):
        out = P.gemm_fp8(xq[:t].contiguous(), ex[:t].cuda(), vals, meta, ew.cuda(), n, B.SP24_OUT_F32)
        np.testing.assert_array_equal(f64(out), y[:t])


def test_gemm_nan_block_stays_in_its_row():
    x = rand((40, 640), F32, 3)
    x[7, 300] = float("inf")
    w = rand((136, 640), BF, 4, 0.02).cuda()
    vals, meta, e_w = P.prune_compress_fp8(w)
    xq, e_x = P.quantize_fp8(x.cuda())
    y = P.gemm_fp8(xq, e_x, vals, meta, e_w, 136).cpu()
    assert torch.isnan(y[7]).all()
    y[7] = 0
    assert torch.isfinite(y).all()


def test_gemm_leaves_the_rest_of_its_buffers():
    """Rows behind the last token and bytes behind Y keep what they held."""
    m, n, k = 37, 264, 544
    xq, e_x, vals, meta, e_w, y, a = product_case(m, n, k, 2)
    big = torch.full((m + 3, n), 7.0, dtype=BF, device="cuda")
    P.gemm_fp8(xq, e_x, vals, meta, e_w, n, out=big[:m])
    assert_product(big[:m], y, a, k, True)
    assert (big[m:] == 7).all()


def test_gemm_offsets_past_32_bits():
    m, n, k = 530000, 64, 4096                # X has 2.17e9 codes
    w = rand((n, k), BF, 1, 0.02, 0.5)
    vals, meta, e_w = P.prune_compress_fp8(w.cuda())
    xq = torch.zeros((m, k), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    e_x = torch.full((m, 32), 127, dtype=torch.uint8, device="cuda")
    tq, te = P.quantize_fp8(rand((5, k), F32, 2).cuda())
    xq[-5:] = tq
    e_x[-5:] = te.view(torch.uint8)
    out = P.gemm_fp8(xq, e_x, vals, meta, e_w, n)
    wq, we = O.fp8_weight(f64(w), O.prune(f64(w), O.MAGNITUDE, 2))
    y, a = O.fp8_gemm(f64(tq), exps(te), wq, we)
    assert_product(out[-5:], y, a, k, True)
    assert float(out[:-5].abs().max()) == 0.0


# ------------------------------------------------------------ norm, forward
NORM_SIZES = [(1, 16), (1, 4096), (3, 256), (5, 272), (9, 512), (17, 768), (2, 1024), (4, 1040),
              (700, 2064), (3, 8192), (2, 8208), (5, 11008), (2, 16384), (400, 128), (350, 8192)]


def stored_sum(x, r):
    return x if r is None else (x.float() + r.float()).to(x.dtype)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("m,k", NORM_SIZES)
def test_norm_fp8(m, k, res, dt):
    x = rand((m, k), dt, m + k)
    r = rand((m, k), dt, m + k + 1) if res else None
    gamma = (1 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(k))).to(dt)
    o = P.rmsnorm_quant(x.cuda(), gamma.cuda(), None if r is None else r.cuda(), EPS, want_rstd=True)
    h = stored_sum(x, r)
    assert torch.equal(o.h.cpu(), h)
    y, s = O.rmsnorm(f64(h), f64(gamma), EPS)
    np.testing.assert_allclose(f64(o.rstd), s, rtol=NORM_REL)
    assert_codes_near(o.y, o.e_y, y, NORM_REL, k)
    assert B.sp24_device_status() == B.SP24_OK


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("m,k", [(1, 4096), (6, 272), (40, 768), (11, 2064), (3, 16384)])
def test_norm_int8_and_bf16(m, k, dt):
    x, r = rand((m, k), dt, 1), rand((m, k), dt, 2)
    gamma = (1 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(k))).to(dt)
    s_x = torch.tensor([0.037], device="cuda")
    h = stored_sum(x, r)
    y, _ = O.rmsnorm(f64(h), f64(gamma), EPS)
    o = P.rmsnorm_quant(x.cuda(), gamma.cuda(), r.cuda(), EPS, B.SP24_INT8, s_x=s_x)
    v = y / float(s_x.double().cpu())
    rel = NORM_REL + 2.0 ** -24
    lo, hi = np.rint(np.clip(v * (1 - rel), -127, 127)), np.rint(np.clip(v * (1 + rel), -127, 127))
    got = o.y.cpu().numpy().astype(np.float64)
    assert ((got == lo) | (got == hi)).all()
    o = P.rmsnorm_quant(x.cuda(), gamma.cuda(), r.cuda(), EPS, B.SP24_BF16)
    assert (np.abs(f64(o.y) - y) <= (HALF_BF16 + 2 * NORM_REL) * np.abs(y)).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("m,k", [(297, 528), (296, 2048), (297, 2048), (297, 8192), (150, 12288),
                                 (3, 12304), (149, 16384)])
def test_norm_at_the_kernel_borders(m, k, dt):
    """Row lengths and counts on both sides of every choice of kernel."""
    x, r = rand((m, k), dt, m), rand((m, k), dt, k)
    gamma = (1 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(k))).to(dt)
    o = P.rmsnorm_quant(x.cuda(), gamma.cuda(), r.cuda(), EPS, want_rstd=True)
    h = stored_sum(x, r)
    assert torch.equal(o.h.cpu(), h)
    y, s = O.rmsnorm(f64(h), f64(gamma), EPS)
    np.testing.assert_allclose(f64(o.rstd), s, rtol=NORM_REL)
    assert_codes_near(o.y, o.e_y, y, NORM_REL, k)
    dy = rand((m, k), dt, 3, 1.0, 0.5)
    dx, dg = P.rmsnorm_backward(dy.cuda(), o.h, gamma.cuda(), o.rstd, dH=o.h)
    assert_back(dx, dg, h, gamma, dy, h, o.rstd.cpu(), dt is BF)


def test_norm_copies_the_stream_without_a_residual():
    x = rand((5, 528), BF, 1).cuda()
    h = torch.zeros_like(x)
    o = P.rmsnorm_quant(x, torch.ones(528, dtype=BF, device="cuda"), out_sum=h)
    assert o.h is h and torch.equal(h, x)


def test_norm_in_place_stream_and_zero_rows():
    m, k = 50, 1536
    x, r = rand((m, k), BF, 3).cuda(), rand((m, k), BF, 4).cuda()
    x[7] = 0
    r[7] = 0
    gamma = torch.ones(k, dtype=BF, device="cuda")
    want = P.rmsnorm_quant(x, gamma, r)
    for target in ("x", "r"):
        x2, r2 = x.clone(), r.clone()
        o = P.rmsnorm_quant(x2, gamma, r2, out_sum=x2 if target == "x" else r2)
        assert torch.equal(o.h, want.h)
        assert torch.equal(o.y.view(torch.uint8), want.y.view(torch.uint8))
        assert torch.equal(r2 if target == "x" else x2, r if target == "x" else x)
    assert int(want.y[7].view(torch.uint8).max()) == 0 and (exps(want.e_y)[7] == 0).all()


def test_norm_non_finite_rows_stay_alone():
    x = rand((6, 512), F32, 8)
    x[2, 5] = float("nan")
    x[4, 200] = float("inf")
    gamma = torch.ones(512, device="cuda")
    o = P.rmsnorm_quant(x.cuda(), gamma)
    by, q = o.e_y.view(torch.uint8).cpu(), o.y.view(torch.uint8).cpu()
    assert (by[2] == 255).all() and (q[2] == 0x7F).all()
    assert by[4, 1] == 255 and (q[4, 128:256] == 0x7F).all() and (q[4, 256:] & 0x7F == 0).all()
    clean = P.rmsnorm_quant(torch.nan_to_num(x, nan=1.0, posinf=1.0).cuda(), gamma)
    for i in (0, 1, 3, 5):
        assert torch.equal(q[i], clean.y.view(torch.uint8).cpu()[i])


# ----------------------------------------------------------- norm, backward
BACK_SIZES = [(1, 16), (1, 4096), (7, 256), (70, 272), (509, 768), (2000, 512), (13, 1024),
              (33, 1040), (1300, 2064), (5, 8192), (700, 8208), (3, 11008), (200, 16384)]


def back_inputs(m, k, dt, seed):
    h = rand((m, k), dt, seed, 1.0, 0.5)
    gamma = (1 + 0.2 * torch.randn(k, generator=torch.Generator().manual_seed(k))).to(dt)
    dy = rand((m, k), dt, seed + 1, 1.0, 0.5)
    dh = rand((m, k), dt, seed + 2, 1.0, 0.5)
    rstd = torch.from_numpy(1 / np.sqrt((f64(h) ** 2).mean(1) + EPS)).float()
    return h, gamma, dy, dh, rstd


def assert_back(dx, dg, h, gamma, dy, dh, rstd, bf16):
    """Row terms: g, xh and the mean carry at most 70 + 6 half-steps of 2^-24 of
    the sum of magnitudes; dgamma sums m products of 3 roundings, in chunks of
    a row of the workspace each (at most m additions in all)."""
    m, k = h.shape
    H, G, D, S = f64(h), f64(gamma), f64(dy), f64(rstd)
    want, wg = O.rmsnorm_backward(D, H, G, S, None if dh is None else f64(dh))
    xh = H * S[:, None]
    mag = S[:, None] * (np.abs(D * G) + np.abs(xh) * np.abs(D * G * xh).mean(1, keepdims=True))
    if dh is not None:
        mag = mag + np.abs(f64(dh))
    tol = 96 * 2.0 ** -24 * mag + (HALF_BF16 * np.abs(want) if bf16 else 0.0)
    assert (np.abs(f64(dx) - want) <= tol).all()
    tg = (min(m, 2000) + 8) * 2.0 ** -24 * np.abs(D * xh).sum(0)
    assert (np.abs(f64(dg) - wg) <= tg).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("m,k", BACK_SIZES)
def test_norm_backward(m, k, with_dh, dt):
    h, gamma, dy, dh, rstd = back_inputs(m, k, dt, m + k)
    dh = dh if with_dh else None
    args = (dy.cuda(), h.cuda(), gamma.cuda(), rstd.cuda())
    dx, dg = P.rmsnorm_backward(*args, dH=None if dh is None else dh.cuda())
    assert_back(dx, dg, h, gamma, dy, dh, rstd, dt is BF)
    dx2, dg2 = P.rmsnorm_backward(*args, dH=None if dh is None else dh.cuda())
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)      # same bits again


def test_norm_backward_against_differences():
    """Central differences of the forward (bf16-free: float32 stream) in 64 bits."""
    m, k = 3, 48
    h, gamma, dy, _, _ = back_inputs(m, k, F32, 6)
    o = P.rmsnorm_quant(h.cuda(), gamma.cuda(), eps=EPS, out_dtype=B.SP24_BF16, want_rstd=True)
    dx, dg = P.rmsnorm_backward(dy.cuda(), o.h, gamma.cuda(), o.rstd)
    H, G, D = f64(h), f64(gamma), f64(dy)
    loss = lambda hh, gg: float((O.rmsnorm(hh, gg, EPS)[0] * D).sum())  # noqa: E731
    for i, j in [(0, 0), (1, 17), (2, 47), (0, 31)]:
        d = 1e-5
        a, b = H.copy(), H.copy()
        a[i, j] += d
        b[i, j] -= d
        want = (loss(a, G) - loss(b, G)) / (2 * d)
        assert abs(float(dx[i, j]) - want) <= 1e-5 * (1 + abs(want)) * 10
    for j in (0, 20, 47):
        a, b = G.copy(), G.copy()
        a[j] += 1e-5
        b[j] -= 1e-5
        want = (loss(H, a) - loss(H, b)) / 2e-5
        assert abs(float(dg[j]) - want) <= 1e-4 * (1 + abs(want))


def test_norm_backward_in_place_and_no_rows():
    h, gamma, dy, dh, rstd = (t.cuda() for t in back_inputs(40, 2064, BF, 1))
    want, wg = P.rmsnorm_backward(dy, h, gamma, rstd, dH=dh)
    for which in (0, 1):
        a, b = dy.clone(), dh.clone()
        dx, dg = P.rmsnorm_backward(a, h, gamma, rstd, dH=b, out=(a, b)[which])
        assert torch.equal(dx, want) and torch.equal(dg, wg)
    e = torch.empty((0, 64), dtype=BF, device="cuda")
    dx, dg = P.rmsnorm_backward(e, e, gamma[:64].clone(), torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and (dg == 0).all()


# ------------------------------------------------------- together, as used
def test_decoder_step_of_fp8_layers():
    """norm -> up projection -> quantise -> down projection -> next norm, on a
    side stream, then captured and replayed with new inputs."""
    m, k, f = 19, 512, 1056
    wu, wd = rand((f, k), BF, 1, 0.05, 0.3), rand((k, f), BF, 2, 0.05, 0.3)
    gamma = torch.ones(k, dtype=BF, device="cuda")
    up, down = P.prune_compress_fp8(wu.cuda()), P.prune_compress_fp8(wd.cuda())
    x, r = rand((m, k), BF, 3, 1, 0.3).cuda(), rand((m, k), BF, 4, 1, 0.3).cuda()

    def step():
        o = P.rmsnorm_quant(x, gamma, r)
        u = P.gemm_fp8(o.y, o.e_y, *up, f)
        q, e = P.quantize_fp8(u)
        d = P.gemm_fp8(q, e, *down, k)
        return o, u, q, e, d, P.rmsnorm_quant(d, gamma, o.h)

    def check(o, u, q, e, d, last):
        h = stored_sum(x.cpu(), r.cpu())
        y, _ = O.rmsnorm(f64(h), np.ones(k), EPS)
        assert_codes_near(o.y, o.e_y, y, NORM_REL, k)
        for xq, ex, w, got, kk in ((o.y, o.e_y, wu, u, k), (q, e, wd, d, f)):
            wq, we = O.fp8_weight(f64(w), O.prune(f64(w), O.MAGNITUDE, 2))
            yy, a = O.fp8_gemm(f64(xq), exps(ex)[:, :(kk + 127) // 128], wq, we)
            assert_product(got, yy, a, kk, True)
        uq, ue = O.fp8_rows(f64(u))
        np.testing.assert_array_equal(f64(q), uq)
        assert_scales(e, ue, f)
        hh = stored_sum(d.cpu(), o.h.cpu())
        assert torch.equal(last.h.cpu(), hh)
        assert_codes_near(last.y, last.e_y, O.rmsnorm(f64(hh), np.ones(k), EPS)[0], NORM_REL, k)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    check(*got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    x.copy_(rand((m, k), BF, 13, 1, 0.3))
    r.copy_(rand((m, k), BF, 14, 1, 0.3))
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    check(*got)
    assert B.sp24_device_status() == B.SP24_OK


def test_norm_feeds_the_int8_product():
    """int8 output with a calibrated scale through sp24_gemm, forward and the
    straight-through gradient of the norm."""
    m, k, n = 24, 768, 256
    x = rand((m, k), BF, 1, 1, 0.3).cuda()
    gamma = torch.ones(k, dtype=BF, device="cuda")
    w = rand((n, k), BF, 2, 0.02, 0.3).cuda()
    vals, meta, s_w = P.prune_compress_int8(w)
    ref = P.rmsnorm_quant(x, gamma, out_dtype=B.SP24_BF16)
    s_x = P.act_scale(ref.y.float())
    o = P.rmsnorm_quant(x, gamma, out_dtype=B.SP24_INT8, s_x=s_x, want_rstd=True)
    y = P.gemm(o.y, vals, meta, n, B.SP24_INT8, s_x, s_w)
    acc = P.gemm(o.y, vals, meta, n, B.SP24_INT8, out_kind=B.SP24_OUT_INT32)
    want = (acc.float() * (s_x * s_w)).to(BF)
    assert torch.equal(y, want)
    keep = O.prune(f64(w), O.MAGNITUDE, 2)
    wd = torch.from_numpy(np.where(keep, f64(w), 0)).float().cuda()
    dy = torch.ones((m, n), device="cuda") @ wd
    dx, dg = P.rmsnorm_backward(dy.to(BF), o.h, gamma, o.rstd)
    assert_back(dx, dg, x.cpu(), gamma.cpu(), dy.to(BF).cpu(), None, o.rstd.cpu(), True)


def test_norm_of_rows_with_an_exact_root():
    """A row whose 1 / rms is a power of two: no remainder, so y is exact and ties
    go to the even code; rows of equal magnitudes and both signs."""
    k = 256
    x = torch.ones((3, k))
    x[0, ::2] = -1
    x[1] = 0.25
    x[2] = 0.25
    gamma = torch.tensor([1.0, 1.0625, 1.1875, -1.3125] * (k // 4))   # e4m3 ties among them
    o = P.rmsnorm_quant(x.cuda(), gamma.cuda(), eps=0.0, want_rstd=True)
    y = torch.sign(x.double()) * gamma.double()
    assert o.rstd.cpu().tolist() == [1.0, 4.0, 4.0]
    want_q, want_e = O.fp8_rows(y.numpy())
    assert_scales(o.e_y, want_e, k)
    np.testing.assert_array_equal(f64(o.y), want_q)


def test_norm_sum_of_subnormals_and_large_values():
    """bf16 sums keep subnormals and round once."""
    v = torch.tensor([1.0, 2.0 ** -8, 2.0 ** -9, 2.0 ** -130, 3 * 2.0 ** -133, 3e38, -0.0, 257.0])
    x = v.repeat(32).to(BF).view(1, 256)
    r = torch.tensor([2.0 ** -8, 1.0, 1.0, 2.0 ** -131, 2.0 ** -133, 1e36, -0.0, 0.5]).repeat(32)
    r = r.to(BF).view(1, 256)
    o = P.rmsnorm_quant(x.cuda(), torch.ones(256, dtype=BF, device="cuda"), r.cuda())
    assert torch.equal(o.h.cpu().view(torch.int16), (x.float() + r.float()).to(BF).view(torch.int16))


def test_two_streams_and_threads():
    """Calls on two streams at once give what they give alone."""
    import threading
    m, k, n = 300, 1040, 520
    k = 1056
    xs = [rand((m, k), BF, 20 + i, 1, 0.5).cuda() for i in range(2)]
    gamma = torch.ones(k, dtype=BF, device="cuda")
    w = P.prune_compress_fp8(rand((n, k), BF, 30, 0.02, 0.3).cuda())

    def one(x):
        o = P.rmsnorm_quant(x, gamma, x, want_rstd=True)
        y = P.gemm_fp8(o.y, o.e_y, *w, n)
        dx, dg = P.rmsnorm_backward(x, o.h, gamma, o.rstd)
        return [o.y.view(torch.uint8), o.e_y.view(torch.uint8), y, dx, dg]

    alone = [one(x) for x in xs]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(20):
                got[i] = one(xs[i])
        st.synchronize()

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    for i in range(2):
        for a, b in zip(alone[i], got[i]):
            assert torch.equal(a, b)


# ----------------------------------------------------------------- refusals
def test_binding_refuses_wrong_tensors():
    x = torch.zeros((4, 256), dtype=BF, device="cuda")
    gamma = torch.ones(256, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        P.quantize_fp8(x.to(torch.float16))
    with pytest.raises(ValueError):
        P.quantize_fp8(torch.zeros((4, 512), dtype=BF, device="cuda")[:, ::2])
    with pytest.raises(ValueError):
        P.quantize_fp8(x.cpu())
    with pytest.raises(ValueError):
        P.rmsnorm_quant(x, gamma.float())
    with pytest.raises(ValueError):
        P.rmsnorm_quant(x, gamma[:128].clone())
    with pytest.raises(ValueError):
        P.rmsnorm_quant(x, gamma, x[:2].clone())
    with pytest.raises(ValueError):
        P.rmsnorm_quant(x, gamma, out_scales=torch.empty((4, 2), dtype=torch.uint8, device="cuda"))
    with pytest.raises(B.Sp24Error) as e:
        P.rmsnorm_quant(x, gamma, out_dtype=B.SP24_INT8)
    assert e.value.status == B.SP24_ERR_ARG
    with pytest.raises(B.Sp24Error) as e:
        P.quantize_fp8(torch.zeros((4, 264), dtype=BF, device="cuda"))
    assert e.value.status == B.SP24_ERR_ALIGN
    big = torch.zeros((1, B.SP24_NORM_MAX_K + 16), dtype=BF, device="cuda")
    with pytest.raises(B.Sp24Error) as e:
        P.rmsnorm_quant(big, big[0].clone())
    assert e.value.status == B.SP24_ERR_UNSUPPORTED
    vals, meta, e_w = P.prune_compress_fp8(torch.zeros((64, 256), dtype=BF, device="cuda"))
    xq, e_x = P.quantize_fp8(x)
    with pytest.raises(ValueError):
        P.gemm_fp8(xq, e_x, vals, meta, e_w, 128)             # another N
    with pytest.raises(ValueError):
        P.gemm_fp8(xq, e_x[:2].contiguous(), vals, meta, e_w, 64)
    with pytest.raises(ValueError):
        P.gemm_fp8(xq, e_x, vals, meta[:1024].clone(), e_w, 64)
    with pytest.raises(B.Sp24Error) as e:
        P.gemm_fp8(xq, e_x, vals, meta, e_w, 64, out_kind=B.SP24_OUT_INT8)
    assert e.value.status == B.SP24_ERR_ARG
    assert B.sp24_device_status() == B.SP24_OK


@pytest.mark.parametrize("dt", [BF, F32])
def test_norm_of_an_overflowing_product(dt):
    """|y| past the largest float32 makes its block NaN, as an infinity does; y just
    below it stays finite."""
    k = 256
    x = torch.full((3, k), 2.0 ** -10, dtype=dt)
    x[:, 0] = 2.0 ** -6                         # y / gamma = 2^-6 s, of order 10
    gamma = torch.ones(k, dtype=dt)
    gamma[0] = 2.0 ** 126                       # y of 1e39: above 3.4e38
    q = P.rmsnorm_quant(x.cuda(), gamma.cuda(), eps=0.0)
    s = 1.0 / np.sqrt((f64(x) ** 2).mean(axis=1))
    assert (2.0 ** -6 * s * 2.0 ** 126 > 2.0 ** 128).all()
    assert (q.e_y.view(torch.uint8)[:, 0] == 255).all() and (q.y.view(torch.uint8)[:, :128] == 0x7F).all()
    assert (exps(q.e_y)[:, 1] < 10).all() and torch.isfinite(q.y[:, 128:].float()).all()
    gamma[0] = 2.0 ** 123                       # y of 1e38
    q = P.rmsnorm_quant(x.cuda(), gamma.cuda(), eps=0.0)
    want = 2.0 ** -6 * s * 2.0 ** 123
    got = f64(q.y)[:, 0] * 2.0 ** exps(q.e_y)[:, 0]
    assert (np.abs(got - want) <= want * (2.0 ** -4 + NORM_REL)).all()


@pytest.mark.parametrize("m", [4, 600])
@pytest.mark.parametrize("ex,ew", [(227, 27), (27, 227), (254, 3), (1, 254), (60, 68), (190, 60)])
def test_gemm_scales_far_apart(m, ex, ew):
    """Scales whose product is in range though neither is near one: exact (2^-126
    and 2^127 among them, and sums at the edge of float32's normal range)."""
    n, k = 256, 256
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-3, 4, (m, k), generator=g).float().to(torch.float8_e4m3fn).cuda()
    w = torch.randint(-3, 4, (n, k), generator=g).float().to(BF).cuda()
    vals, meta, e_w = P.compress_fp8(w, P.prune(w))
    full = lambda rows, v: torch.full((rows, 4), v, dtype=torch.uint8, device="cuda")
    one = P.gemm_fp8(x, full(m, 127), vals, meta, full(2, 127), n, B.SP24_OUT_F32)
    y = P.gemm_fp8(x, full(m, ex), vals, meta, full(2, ew), n, B.SP24_OUT_F32)
    assert B.sp24_device_status() == B.SP24_OK
    # the codes are whole multiples of 2^6 (three times 2^7 and below: 3 * 2^7 <= 448)
    np.testing.assert_array_equal(f64(y), f64(one) * 2.0 ** (ex - 127 + ew - 127))


@pytest.mark.parametrize("m", [65, 95, 96, 97, 191, 192, 193, 288])
@pytest.mark.parametrize("n,k", [(136, 800), (1032, 2048)])
def test_gemm_at_the_borders_of_96_token_tiles(m, n, k):
    xq, e_x, vals, meta, e_w, y, a = product_case(m, n, k, m)
    assert B.sp24_gemm_plan(m, n, k, B.SP24_FP8)["kernel"] == "splitk"
    for kind in (B.SP24_OUT_BF16, B.SP24_OUT_F32):
        out = P.gemm_fp8(xq, e_x, vals, meta, e_w, n, kind)
        assert B.sp24_device_status() == B.SP24_OK
        assert_product(out, y, a, k, kind == B.SP24_OUT_BF16)


@pytest.mark.parametrize("m", [148, 149, 500])
@pytest.mark.parametrize("k", [8208, 11008, 12288, 12304])
def test_norm_of_long_float_rows(m, k):
    """Float32 rows past the one-vector kernels, with the next row in registers
    (more rows than SMs, no residual) and without; every output type."""
    x, gamma = rand((m, k), F32, m + k), 1.0 + 0.1 * rand((1, k), F32, k)[0]
    r = rand((m, k), F32, 3 * m + k)
    sx = torch.tensor([0.05], device="cuda")
    for res in (None, r):
        h = x if res is None else x + res
        y, s = O.rmsnorm(f64(h), f64(gamma), EPS)
        rc = None if res is None else res.cuda()
        q = P.rmsnorm_quant(x.cuda(), gamma.cuda(), rc, EPS, want_rstd=True)
        assert torch.equal(q.h.cpu(), h)
        assert (np.abs(f64(q.rstd) - s) <= NORM_REL * s).all()
        e = np.repeat(exps(q.e_y)[:, :(k + 127) // 128], 128, axis=1)[:, :k]
        # half a code step, and the arithmetic's error
        step = np.maximum(2.0 ** -4 * np.abs(y) * (1 + NORM_REL), 2.0 ** (e - 10.0))
        assert (np.abs(f64(q.y) * 2.0 ** e - y) <= step + NORM_REL * np.abs(y)).all()
        b = P.rmsnorm_quant(x.cuda(), gamma.cuda(), rc, EPS, B.SP24_BF16)
        assert (np.abs(f64(b.y) - y) <= (HALF_BF16 + 2 * NORM_REL) * np.abs(y)).all()
        i = P.rmsnorm_quant(x.cuda(), gamma.cuda(), rc, EPS, B.SP24_INT8, s_x=sx)
        z = np.clip(y / float(sx.cpu()[0]), -127, 127)
        assert (np.abs(i.y.cpu().numpy() - z) <= 0.5 + 2 * NORM_REL * np.abs(z)).all()
    assert B.sp24_device_status() == B.SP24_OK
