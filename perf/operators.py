"""Measured cases of the 8-bit floating-point operators for 2:4 sparse layers.

Five operators that run next to each other in a decoder layer whose linear
weights are 2:4 sparse and whose matrix products run in e4m3 (4-bit exponent,
3-bit mantissa, largest finite value 448):

norm       h = x + r (rounded to x's type: the residual stream as stored),
           y = h * rsqrt(mean(h^2) + eps) * gamma, written as e4m3 codes with
           one power-of-two scale per row and 128 columns (or as int8 codes
           with one given scale, or as bf16).
norm_back  the gradient of norm to x (= to r) and gamma, the 8-bit rounding
           passed straight through, plus the gradient that reaches h directly.
quantize   the e4m3 codes and scales of an activation that no norm precedes.
weights    2:4 mask, e4m3 values, metadata and one power-of-two scale per
           128 x 128 block of a weight, from its bf16 values.
gemm       Y = X W'^T of quantised activations and a compressed weight, fp32 sums.

A scale is an e8m0 byte b that stands for 2^(b - 127); it is the smallest power
of two for which the block's largest magnitude fits into 448.  A row of scales
is padded to a multiple of four bytes with 127 (a scale of one).
"""
import math

import torch

own = False

FP8_MAX = 448.0
EPS = 1e-6

F8 = torch.float8_e4m3fn
E8 = torch.float8_e8m0fnu


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one token of a 4096-wide decoder layer: latency
        {"name": "norm_decode", "op": "norm", "m": 1, "k": 4096, "x": "bf16", "residual": True, "out": "fp8"},
        # float32 stream, odd token count, the wide dimension, no residual
        {"name": "norm_f32_ragged", "op": "norm", "m": 777, "k": 11008, "x": "f32", "residual": False, "out": "fp8"},
        # prompt of 8192 tokens
        {"name": "norm_prefill", "op": "norm", "m": 8192, "k": 4096, "x": "bf16", "residual": True, "out": "fp8"},
        # fine-tuning a 768-wide encoder layer on a short odd batch
        {"name": "back_small", "op": "norm_back", "m": 509, "k": 768, "x": "bf16", "residual": False},
        # fine-tuning the 4096-wide layer, residual gradient added
        {"name": "back_large", "op": "norm_back", "m": 8192, "k": 4096, "x": "bf16", "residual": True},
        # input of the down projection, a small batch of single tokens
        {"name": "quantize_batch", "op": "quantize", "m": 16, "k": 11008, "x": "bf16"},
        # input of the down projection, prompt
        {"name": "quantize_prefill", "op": "quantize", "m": 8192, "k": 11008, "x": "bf16"},
        # a weight whose sides end inside a block
        {"name": "weights_ragged", "op": "weights", "n": 1496, "k": 800, "score": "wanda"},
        # the up projection
        {"name": "weights_large", "op": "weights", "n": 11008, "k": 4096, "score": "magnitude"},
        # one token through the up projection: bound by the weight's bytes
        {"name": "gemm_decode", "op": "gemm", "m": 1, "n": 11008, "k": 4096, "out": "bf16"},
        # short odd prompt, sides that end inside tiles, float32 output
        {"name": "gemm_ragged", "op": "gemm", "m": 333, "n": 4104, "k": 4128, "out": "f32"},
        # prompt of 8192 tokens through the up projection: bound by the products
        {"name": "gemm_prefill", "op": "gemm", "m": 8192, "n": 11008, "k": 4096, "out": "bf16"},
    ]


def _log(rng, lo, hi, step):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_back", "quantize", "weights", "gemm", "gemm"])
    if op == "weights":
        return {"op": op, "n": _log(rng, 16, 11008, 8), "k": _log(rng, 64, 4096, 32),
                "score": rng.choice(["magnitude", "wanda"])}
    if op == "gemm":
        return {"op": op, "m": _log(rng, 1, 8192, 1), "n": _log(rng, 64, 11008, 8),
                "k": _log(rng, 128, 4096, 32), "out": rng.choice(["bf16", "bf16", "f32"])}
    k = _log(rng, 128, 8192 if op == "norm" else 11008 if op == "quantize" else 4096, 16)
    m = _log(rng, 1, 8192, 1)
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "quantize":
        return {"op": op, "m": m, "k": k, "x": x}
    case = {"op": op, "m": m, "k": k, "x": x, "residual": rng.random() < 0.5}
    if op == "norm":
        case["out"] = rng.choice(["fp8", "fp8", "int8", "bf16"])
    return case


# ------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _stream(g, m, k, dt):
    """A residual stream: rows of different size, a few large channels."""
    x = torch.randn((m, k), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((m, 1), generator=g, device="cuda"))
    gain = torch.where(torch.rand((1, k), generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return (x * gain).to(dt)


def _scale_cols(k):
    return 4 * ((k + 511) // 512)


def _weight(g, n, k):
    """N(0, 0.02) with one entry in a hundred twenty times as large."""
    w = 0.02 * torch.randn((n, k), generator=g, device="cuda")
    tail = torch.rand((n, k), generator=g, device="cuda") < 0.01
    return torch.where(tail, 20.0 * w, w).to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "weights":
        s["w"] = _weight(g, case["n"], case["k"])
        if case["score"] == "wanda":   # column norms of 128 calibration rows
            c = torch.randn((128, case["k"]), generator=g, device="cuda", dtype=torch.float64)
            s["norms"] = c.square().sum(0).sqrt()
        return s
    m, k = case["m"], case["k"]
    if op == "gemm":
        n = case["n"]
        # the weight as the program keeps it: compressed for the sparse product,
        # and the same values laid out densely for the plain one
        w = _weight(g, n, k)
        s["vals"], s["meta"], s["e_w"], s["dense"] = _convert(w, w.float().abs())
        s["x"], s["e_x"] = _to_fp8(_stream(g, m, k, torch.float32))
        s["y"] = torch.empty((m, n), dtype=_dtype(case["out"]), device="cuda")
        return s
    dt = _dtype(case["x"])
    s["x"] = _stream(g, m, k, dt)
    if op == "quantize":
        s["codes"] = torch.empty((m, k), dtype=F8, device="cuda")
        s["e"] = torch.empty((m, _scale_cols(k)), dtype=E8, device="cuda")
        return s
    s["gamma"] = (1.0 + 0.1 * torch.randn(k, generator=g, device="cuda")).to(dt)
    if op == "norm":
        s["r"] = _stream(g, m, k, dt) if case["residual"] else None
        s["s_x"] = torch.full((1,), 6.0 / 127.0, device="cuda") * (
            1.0 + 0.1 * torch.rand(1, generator=g, device="cuda"))
        if case["out"] == "fp8":
            s["y"] = torch.empty((m, k), dtype=F8, device="cuda")
            s["e"] = torch.empty((m, _scale_cols(k)), dtype=E8, device="cuda")
        else:
            s["y"] = torch.empty((m, k), device="cuda",
                                 dtype=torch.int8 if case["out"] == "int8" else torch.bfloat16)
            s["e"] = None
        s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
        return s
    s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS).float()
    s["dy"] = torch.randn((m, k), generator=g, device="cuda").to(dt)
    s["dh"] = torch.randn((m, k), generator=g, device="cuda").to(dt) if case["residual"] else None
    return s


# -------------------------------------------------------------- plain forms
def _pow2(e):
    """2^e as float32 for whole e in [-126, 127], from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e; 0 for an empty block.  448 is 0.875 * 2^9."""
    f, x = torch.frexp(amax)
    e = x - 9 + (f > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.zeros_like(e)).clamp(-126, 127)


def _pad_scales(e, k):
    """Exponents [rows, blocks] as e8m0 [rows, padded blocks]."""
    b = torch.full((e.shape[0], _scale_cols(k)), 127, dtype=torch.uint8, device=e.device)
    b[:, : e.shape[1]] = (e + 127).to(torch.uint8)
    return b.view(E8)


def _blocks(y):
    """[m, k] as [m, blocks, 128], zeros past k."""
    m, k = y.shape
    kb = (k + 127) // 128
    return torch.nn.functional.pad(y, (0, kb * 128 - k)).view(m, kb, 128)


def _to_fp8(y):
    """e4m3 codes and e8m0 scales of a float32 [m, k]."""
    m, k = y.shape
    b = _blocks(y)
    e = _exponent(b.abs().amax(2))
    q = (b * _pow2(-e)[:, :, None]).to(F8)
    return q.view(m, -1)[:, :k].contiguous(), _pad_scales(e, k)


def _from_fp8(q, e):
    k = q.shape[1]
    return q.float() * e.float().repeat_interleave(128, 1)[:, :k]


def _keep(score):
    """2:4 mask of [n, k] scores: a position stays if fewer than two others of
    its group beat it; ties go to the lower index."""
    s = score.view(score.shape[0], -1, 4)
    a, b = s[..., :, None], s[..., None, :]              # does b beat a?
    i = torch.arange(4, device=s.device)
    lower = i[None, :] < i[:, None]
    beaten = (b > a) | ((b == a) & lower)
    return (beaten.sum(-1) < 2).view(score.shape)


def _convert(w, score):
    """(values [n, k/2], metadata, scales, dense masked codes) of a weight.

    The metadata is the row-major operand layout of 8-bit values: chunks of 128
    rows x 128 positions (ordered row block first), 16 bytes per row, one nibble
    lo | hi << 2 per group of four; rows and groups past the edge hold (0, 1)."""
    n, k = w.shape
    nb, kb = (n + 127) // 128, (k + 127) // 128
    keep = _keep(score)
    wf = torch.where(keep, w.float(), torch.zeros((), device=w.device))
    pad = torch.nn.functional.pad(wf, (0, kb * 128 - k, 0, nb * 128 - n))
    tiles = pad.view(nb, 128, kb, 128)
    e = _exponent(tiles.abs().amax((1, 3)))
    q = (tiles * _pow2(-e)[:, None, :, None]).to(F8).view(nb * 128, kb * 128)[:n, :k].contiguous()
    grp = keep.view(n, k // 4, 4)
    lo = grp.to(torch.int32).argmax(2)
    hi = 3 - grp.flip(2).to(torch.int32).argmax(2)
    at = torch.stack((lo, hi), 2)
    vals = q.view(torch.uint8).view(n, k // 4, 4).gather(2, at).view(n, k // 2).contiguous().view(F8)
    code = torch.full((nb * 128, kb * 32), 4, dtype=torch.int32, device=w.device)
    code[:n, : k // 4] = (lo | (hi << 2)).to(torch.int32)
    byte = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)
    meta = byte.view(nb, 128, kb, 16).permute(0, 2, 1, 3).contiguous().view(-1)
    return vals, meta, _pad_scales(e, k), q


def _plain_norm(s):
    x = s["x"].float()
    h = x if s["r"] is None else (x + s["r"].float()).to(s["x"].dtype).float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["gamma"].float()
    got = {} if s["r"] is None else {"h": h.to(s["x"].dtype)}
    if s["out"] == "fp8":
        got["y"], got["e"] = _to_fp8(y)
    elif s["out"] == "int8":   # the codes as numbers
        got["y"] = torch.round(y / s["s_x"]).clamp(-127, 127).to(torch.bfloat16)
    else:
        got["y"] = y.to(torch.bfloat16)
    return got


def _plain_back(s):
    h, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xh = h * rstd
    g = dy * s["gamma"].float()
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum(0)}


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_back":
        return _plain_back(s)
    if op == "quantize":
        q, e = _to_fp8(s["x"].float())
        return {"y": q, "e": e}
    if op == "weights":
        score = s["w"].float().abs()
        if s["score"] == "wanda":
            score = score.double() * s["norms"]
        vals, meta, e, _ = _convert(s["w"], score)
        return {"vals": vals, "meta": meta, "e": e}
    x = _from_fp8(s["x"], s["e_x"])
    w = _from_fp8(s["dense"], s["e_w"].float().repeat_interleave(128, 0)[: s["n"]])
    return {"y": (x @ w.t()).to(_dtype(s["out"]))}


def _run_own(s):
    from structured_sparse_gemm_sp24_b200 import pipeline as P, sp24 as B
    op = s["op"]
    if op == "norm":
        kind = {"fp8": B.SP24_FP8, "int8": B.SP24_INT8, "bf16": B.SP24_BF16}[s["out"]]
        o = P.rmsnorm_quant(s["x"], s["gamma"], residual=s["r"], eps=EPS, out_dtype=kind,
                            s_x=s["s_x"] if s["out"] == "int8" else None,
                            out=s["y"], out_scales=s["e"], out_sum=s["h"])
        got = {} if s["r"] is None else {"h": o.h}
        got["y"] = o.y.to(torch.bfloat16) if s["out"] == "int8" else o.y
        if s["out"] == "fp8":
            got["e"] = o.e_y
        return got
    if op == "norm_back":
        dx, dgamma = P.rmsnorm_backward(s["dy"], s["x"], s["gamma"], s["rstd"], dH=s["dh"])
        return {"dx": dx, "dgamma": dgamma}
    if op == "quantize":
        y, e = P.quantize_fp8(s["x"], out=s["codes"], out_scales=s["e"])
        return {"y": y, "e": e}
    if op == "weights":
        if s["score"] == "wanda":
            vals, meta, e = P.prune_compress_fp8(s["w"], B.SP24_WANDA, norms=s["norms"])
        else:
            vals, meta, e = P.prune_compress_fp8(s["w"])
        return {"vals": vals, "meta": meta, "e": e}
    kind = B.SP24_OUT_F32 if s["out"] == "f32" else B.SP24_OUT_BF16
    return {"y": P.gemm_fp8(s["x"], s["e_x"], s["vals"], s["meta"], s["e_w"], s["n"],
                            out_kind=kind, out=s["y"])}


# ------------------------------------------------------------- 64-bit values
def _exact_pow2(e):
    """2^e as float64 for whole e, from its bits (a power function may be an ulp off)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_round(v):
    """float64 values in [-448, 448] to the nearest e4m3 value, ties to even."""
    _, x = torch.frexp(v)                                 # |v| in [2^(x-1), 2^x)
    step = _exact_pow2((x - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_scale(amax):
    """The smallest power of two t with amax <= 448 t; 1 for an empty block."""
    _, x = torch.frexp(amax)
    t = _exact_pow2(x - 10)                               # 448 t < 2^(x-1) <= amax
    for _ in range(2):
        t = torch.where(FP8_MAX * t < amax, 2.0 * t, t)
    return torch.where(amax > 0, t, torch.ones_like(t))


def _exact_codes(y):
    m, k = y.shape
    sc = torch.ones((m, _scale_cols(k)), dtype=torch.float64, device=y.device)
    q = torch.empty_like(y)
    for c in range(0, k, 128):
        part = y[:, c:c + 128]
        t = _exact_scale(part.abs().amax(1))
        sc[:, c // 128] = t
        q[:, c:c + 128] = _exact_round(part / t[:, None])
    return q, sc


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x, got = s["x"].double(), {}
        if s["r"] is not None:
            got["h"] = x + s["r"].double()
            # bf16 values add exactly in 64 bits, so one rounding gives the stored sum
            x = got["h"].to(s["x"].dtype).double()
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / case["k"] + EPS) * s["gamma"].double()
        if case["out"] == "fp8":
            got["y"], got["e"] = _exact_codes(y)
        elif case["out"] == "int8":
            got["y"] = torch.round(y / s["s_x"].double()).clamp(-127, 127)
        else:
            got["y"] = y
        return got
    if op == "norm_back":
        h, r = s["x"].double(), s["rstd"].double()[:, None]
        dy, ga = s["dy"].double(), s["gamma"].double()
        dot = (dy * ga * h).sum(1, keepdim=True)
        dx = r * dy * ga - h * dot * r.pow(3) / case["k"]
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dgamma": (dy * h * r).sum(0)}
    if op == "quantize":
        y, e = _exact_codes(s["x"].double())
        return {"y": y, "e": e}
    if op == "weights":
        w = s["w"].double()
        n, k = w.shape
        score = w.abs() * (s["norms"] if case["score"] == "wanda" else 1.0)
        # the first two of a stable sort by falling score, back in rising order
        top = score.view(n, k // 4, 4).sort(dim=2, descending=True, stable=True).indices[..., :2]
        top = top.sort(dim=2).values
        kept = w.view(n, k // 4, 4).gather(2, top).view(n, k // 2)
        e = torch.ones(((n + 127) // 128, _scale_cols(k)), dtype=torch.float64, device=w.device)
        vals = torch.empty_like(kept)
        for c in range(0, k // 2, 64):
            for r in range(0, n, 128):
                part = kept[r:r + 128, c:c + 64]
                t = _exact_scale(part.abs().max())
                e[r // 128, c // 64] = t
                vals[r:r + 128, c:c + 64] = _exact_round(part / t)
        return {"vals": vals, "meta": None, "e": e}
    n, k = case["n"], case["k"]
    x, w = s["x"].double(), s["dense"].double()
    for c in range(0, k, 128):
        x[:, c:c + 128] *= s["e_x"][:, c // 128].double()[:, None]
        w[:, c:c + 128] *= s["e_w"][:, c // 128].double().repeat_interleave(128)[:n, None]
    return {"y": x @ w.t()}


# --------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "weights":
        n, k = case["n"], case["k"]
        nb, kb = (n + 127) // 128, (k + 127) // 128
        b = 2 * n * k + n * k // 2 + nb * kb * 2048 + nb * _scale_cols(k)
        return {"bytes": b + (8 * k if case["score"] == "wanda" else 0), "flops": 8 * n * k}
    m, k = case["m"], case["k"]
    if op == "gemm":
        n = case["n"]
        nb, kb = (n + 127) // 128, (k + 127) // 128
        b = m * k + m * _scale_cols(k) + n * k // 2 + nb * kb * 2048 + nb * _scale_cols(k)
        return {"bytes": b + m * n * (4 if case["out"] == "f32" else 2), "flops": m * n * k}
    t = 4 if case["x"] == "f32" else 2
    if op == "quantize":
        return {"bytes": m * k * (t + 1) + m * _scale_cols(k), "flops": 3 * m * k}
    if op == "norm":
        o = 2 if case["out"] == "bf16" else 1
        b = m * k * (t + o + (2 * t if case["residual"] else 0)) + k * t
        return {"bytes": b + (m * _scale_cols(k) if case["out"] == "fp8" else 0), "flops": 6 * m * k}
    b = m * k * t * (4 if case["residual"] else 3) + 4 * m + k * t + 4 * k
    return {"bytes": b, "flops": 10 * m * k}
