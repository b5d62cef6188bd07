// libsp24: RMS norm with the residual's addition and an 8-bit output
// (sp24_rmsnorm_quant), its gradient (sp24_rmsnorm_backward), and the block
// quantisation of an activation that no norm precedes (sp24_quantize_fp8).
//
//   h = round(x + r)                       the residual stream as stored
//   s = 1 / sqrt(mean(h^2) + eps)          fp32 within a warp, fp64 across
//   y = h * gamma * s                      rounded once to fp32
//   e4m3: one power-of-two scale per row and 128 columns (fp8.cuh)
//   int8: clamp(rint(y / s_x), -127, 127), the rule of sp24_quantize
//   bf16: y rounded
//
// Bound by HBM: each element of x and r is read once and h and y are written
// once; a row lives in registers between its sum and its output.  A thread
// holds NV vectors of 8 columns (16 bytes of bf16), T threads apart, so 16
// neighbouring lanes hold a 128-column block and its maximum is four shuffles.
// Rows of up to 512 columns take one warp (no barrier); longer rows a block
// of T threads and one barrier.  The grid is persistent, and a row's loads are
// issued before the previous row is reduced and written.

#include "fp8.cuh"
#include "sp24_host.h"

namespace sp24 {

// ------------------------------------------------------------ pairs of fp32
// The arithmetic works on pairs (one instruction for two elements): these
// kernels spend about as long issuing as waiting for memory.
struct Pair {
  uint64_t v;
};
__device__ __forceinline__ Pair pair(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Pair pair(float a) { return pair(a, a); }
__device__ __forceinline__ void split(Pair p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Pair fma2_rz(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Eight e4m3 codes of four pairs times a power of two.
__device__ __forceinline__ uint2 e4m3x8(const Pair (&f)[4], float scale) {
  const Pair s = pair(scale);
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) split(mul2(f[i], s), y[2 * i], y[2 * i + 1]);
  return make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
}

// ------------------------------------------------------- 8-element vectors
// Loads that leave no line in L1 (each element is read once).
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

template <typename T>
struct Vec8;

template <>
struct Vec8<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void zero() { q = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = ld_stream16(p); }
  __device__ __forceinline__ void load_cached(const __nv_bfloat16* p) {
    q = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void load_shared(const __nv_bfloat16* p) {
    q = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = q; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void get(Pair (&f)[4]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  // += v, each sum rounded once (the bf16 adder rounds the exact sum)
  __device__ __forceinline__ void add(const Vec8& v) {
    q.x = add2(q.x, v.q.x);
    q.y = add2(q.y, v.q.y);
    q.z = add2(q.z, v.q.z);
    q.w = add2(q.w, v.q.w);
  }
  __device__ __forceinline__ static uint32_t add2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {   // round to nearest even
    q = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
};

template <>
struct Vec8<float> {
  uint4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const float* p) {
    a = ld_stream16(p);
    b = ld_stream16(p + 4);
  }
  __device__ __forceinline__ void load_cached(const float* p) {
    a = __ldg(reinterpret_cast<const uint4*>(p));
    b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void load_shared(const float* p) {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<uint4*>(p)[0] = a;
    reinterpret_cast<uint4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
  __device__ __forceinline__ void get(Pair (&f)[4]) const {
    float g[8];
    get(g);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pair(g[2 * i], g[2 * i + 1]);
  }
  __device__ __forceinline__ void add(const Vec8& v) {
    float f[8], g[8];
    get(f);
    v.get(g);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fadd_rn(f[i], g[i]);
    set(f);
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3]));
    b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                   __float_as_uint(f[7]));
  }
};

// Largest magnitude of eight values as float bits; a NaN among them gives a NaN.
__device__ __forceinline__ uint32_t amax8(const float (&f)[8]) {
  float a, b, c;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(f[0]), "f"(f[1]), "f"(f[2]));
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(b) : "f"(f[3]), "f"(f[4]), "f"(f[5]));
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(c) : "f"(f[6]), "f"(f[7]), "f"(a));
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(b), "f"(c), "f"(c));
  return __float_as_uint(a);
}

// Largest value of the 16 lanes that hold a block.
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Sum over the `warps` warps of a row, the same value in all threads: each
// warp's by shuffles, then the warps' in order through `part`, of which two
// rows' buffers alternate so that one barrier (hardware barrier `bar`, of the
// row's threads) is enough.
// S is the type of the sum across warps: double keeps the last additions, whose
// roundings no averaging hides, out of the result.
template <bool kWarpRow, typename S>
__device__ __forceinline__ S row_sum(float v, S* part, int warp, int warps, uint32_t bar) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if constexpr (kWarpRow) return static_cast<S>(v);
  if ((threadIdx.x & 31) == 0) part[warp] = static_cast<S>(v);
  named_barrier(bar, 32 * warps);
  if (warps > 8) {   // one value a lane, and shuffles, instead of a long chain
    const int lane = threadIdx.x & 31;
    S u = lane < warps ? part[lane] : S(0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
    return u;
  }
  S t[4] = {S(0), S(0), S(0), S(0)};
  for (int i = 0; i < warps; i += 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < warps) t[j] += part[i + j];
  }
  return (t[0] + t[1]) + (t[2] + t[3]);
}

// ------------------------------------------------------------------ forward
struct NormArgs {
  const void* x;
  const void* r;        // residual (optional)
  const void* gamma;
  void* h;              // x + r as stored (optional)
  void* y;
  uint8_t* e;           // e4m3: scale bytes [m][scale_cols]
  float* rstd;          // optional
  const float* s_x;     // int8: the given scale
  int64_t m, k;
  double inv_k;         // 1 / k
  float eps;
  int scale_cols;
};

// h of one vector: x + r rounded to the stream's type (x without r), and its
// squares added to `sum` in fp32.  The norm is that of the stored sum.
template <typename T>
__device__ __forceinline__ Vec8<T> norm_sum(const Vec8<T>& x, const Vec8<T>& r, bool res, Pair& sum) {
  Vec8<T> h = x;
  if (res) h.add(r);
  Pair f[4];
  h.get(f);
#pragma unroll
  for (int j = 0; j < 4; ++j) sum = fma2(f[j], f[j], sum);
  return h;
}

// y = h * gamma * s of one vector, rounded once.  s comes as hi + lo; the product
// of two bf16 values is exact in fp32, that of two floats is taken with its
// remainder.
//
// kOdd: rounded to odd (truncated, last bit set if that left something), for a y
// that is rounded again to a code: every border between codes is an even fp32
// number, so y stays on the side of the border that the exact product is on, and
// only the error of s can still move a code (8192 x 4096: 1 to 23 of 33.5 million
// codes differ from those of 64 bits, 20 to 27 with y rounded to nearest, 19 to
// 38 in plain fp32).
// `last` is the bit to set in both halves.  An s that is no power of two has no
// finite binary fraction, so its products count as inexact and the bit is set in
// all (a zero becomes the smallest subnormal; a product that is exact all the same,
// 3 * 2/3, is moved by the error of s).  With a power of two only float32 products
// that fp32 does not hold are inexact, those with a remainder (kAsk).  Rows of this
// kind are rare: they are done again after the others, as the question in every
// row, or a loop of its own there, costs registers (777 x 11008: 15.3 us a call;
// 14.0 this way and 13.9 without).
enum Rounding { kNearest, kOdd, kAsk };

__device__ __forceinline__ bool norm_pow2(float2 s) {
  return s.y == 0.0f && (__float_as_uint(s.x) & 0x007FFFFFu) == 0u;
}

template <Rounding R>
__device__ __forceinline__ Pair norm_round(Pair p, Pair s, Pair rest, uint64_t last) {
  if constexpr (R == kNearest) return fma2(p, s, rest);
  Pair y = fma2_rz(p, s, rest);
  y.v |= last;
  return y;
}
template <Rounding R>
__device__ __forceinline__ void norm_scale(const Vec8<__nv_bfloat16>& h, const Vec8<__nv_bfloat16>& g,
                                           float2 s, Pair (&y)[4]) {
  const uint64_t last = norm_pow2(s) ? 0ull : 0x0000000100000001ull;
  Pair fg[4];
  h.get(y);
  g.get(fg);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Pair p = mul2(y[j], fg[j]);
    y[j] = norm_round<R>(p, pair(s.x), mul2(p, pair(s.y)), last);
  }
}
template <Rounding R>
__device__ __forceinline__ void norm_scale(const Vec8<float>& h, const Vec8<float>& g, float2 s,
                                           Pair (&y)[4]) {
  Pair fg[4];
  h.get(y);
  g.get(fg);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Pair p = mul2(y[j], fg[j]);
    const Pair e = fma2(y[j], fg[j], mul2(p, pair(-1.0f)));
    uint64_t last = 0x0000000100000001ull;
    if constexpr (R == kAsk) {
      float e0, e1;
      split(e, e0, e1);
      last = (e0 != 0.0f ? 1ull : 0ull) | (e1 != 0.0f ? 1ull << 32 : 0ull);
    }
    y[j] = norm_round<R>(p, pair(s.x), fma2(p, pair(s.y), mul2(e, pair(s.x))), last);
  }
}

// y of one vector (columns 8c ..) of row `row` and its output.  All lanes of a
// warp call it, `ok` where the columns exist: 16 neighbouring lanes hold a
// 128-column block.
template <typename T, int OUT, Rounding R = OUT == SP24_FP8 ? kOdd : kNearest>
__device__ __forceinline__ void norm_out(const NormArgs& a, const Vec8<T>& h, const Vec8<T>& g,
                                         float2 rs, int64_t row, int c, bool ok, float sx, float rsx) {
  Pair y[4];
  norm_scale<R>(h, g, rs, y);
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) split(y[j], f[2 * j], f[2 * j + 1]);
  const int64_t at = row * a.k + 8 * c;
  if constexpr (OUT == SP24_FP8) {
    // (a NaN statistic makes NaNs of the zeros past the row)
    uint32_t amax = block_max(ok ? amax8(f) : 0u);
    if (amax == 1u) amax = 0u;            // a block of zeros, rounded to odd
    if (amax == 0x7F7FFFFFu) amax += 1u;  // truncation holds an overflow at the largest float
    const uint32_t byte = scale_byte(amax);
    const float inv = scale_inverse(byte);
    if (ok) {
      const uint2 q = e4m3x8(y, inv);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + at) = q;
      if ((threadIdx.x & 15) == 0) a.e[row * a.scale_cols + (c >> 4)] = static_cast<uint8_t>(byte);
    }
  } else if constexpr (OUT == SP24_INT8) {
    if (ok) {
      uint2 q;
      q.x = q8(f[0], sx, rsx) | (q8(f[1], sx, rsx) << 8) | (q8(f[2], sx, rsx) << 16) |
            (q8(f[3], sx, rsx) << 24);
      q.y = q8(f[4], sx, rsx) | (q8(f[5], sx, rsx) << 8) | (q8(f[6], sx, rsx) << 16) |
            (q8(f[7], sx, rsx) << 24);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + at) = q;
    }
  } else {
    if (ok) {
      Vec8<__nv_bfloat16> o;
      o.set(f);
      o.store(static_cast<__nv_bfloat16*>(a.y) + at);
    }
  }
}

// 1 / sqrt(mean + eps) as hi + lo: the rounded root of the rounded argument and
// one Newton step from its residual 1 - v hi^2, formed with exact products.  A
// root that is 0, infinite or NaN stands as it is.
__device__ __forceinline__ float2 norm_rstd(double sum, const NormArgs& a) {
  const double v = __fma_rn(sum, a.inv_k, static_cast<double>(a.eps));
  const float vh = __double2float_rn(v);
  const float vl = __double2float_rn(v - static_cast<double>(vh));
  const float r = __frsqrt_rn(vh);
  const float t = __fmul_rn(r, r), tl = __fmaf_rn(r, r, -t);
  const float e = __fmaf_rn(-vl, t, __fmaf_rn(-vh, tl, __fmaf_rn(-vh, t, 1.0f)));
  const float lo = __fmul_rn(0.5f * r, e);
  return make_float2(r, fabsf(lo) < r ? lo : 0.0f);   // (false for inf, NaN)
}

// Per row: 1 / rms, and (e4m3) the padding of the scale row, by thread t of the row.
template <int OUT>
__device__ __forceinline__ void norm_row_end(const NormArgs& a, int64_t row, int t, float2 rs) {
  if (a.rstd != nullptr && t == 0) a.rstd[row] = rs.x + rs.y;
  if constexpr (OUT == SP24_FP8) {
    const int kb = static_cast<int>((a.k + 127) >> 7);
    if (t < a.scale_cols - kb) a.e[row * a.scale_cols + kb + t] = static_cast<uint8_t>(kScaleOne);
  }
}

// Rows straight from global memory: short rows (one warp each) and few rows.
// kRes: a residual may be given (its vectors take registers).
template <typename T, int OUT, int NV, bool kWarpRow, int MAXT, int MINB, bool kRes = true>
__global__ void __launch_bounds__(MAXT, MINB) norm_kernel(const NormArgs a) {
  pdl_launch_dependents();
  pdl_wait_prior();
  __shared__ double part[2][32];
  const int t = kWarpRow ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int nt = kWarpRow ? 32 : static_cast<int>(blockDim.x);
  const int per_cta = kWarpRow ? static_cast<int>(blockDim.x >> 5) : 1;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * per_cta + (kWarpRow ? threadIdx.x >> 5 : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * per_cta;
  const bool res = kRes && a.r != nullptr;
  const int c_end = static_cast<int>(a.k / 8);
  const float sx = OUT == SP24_INT8 ? *a.s_x : 1.0f;
  const float rsx = __frcp_rn(sx);

  Vec8<T> x[NV], r[NV];
  auto load = [&](int64_t row) {
    const T* xp = static_cast<const T*>(a.x) + row * a.k;
    const T* rp = static_cast<const T*>(a.r) + row * a.k;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * nt;
      x[i].zero();
      if (res) r[i].zero();
      if (c < c_end) {
        x[i].load(xp + 8 * c);
        if (res) r[i].load(rp + 8 * c);
      }
    }
  };
  // the next row is loaded before this one is reduced, where the registers
  // allow (two float32 rows of two vectors and their residuals would spill)
  constexpr bool kAhead = sizeof(T) * NV <= 4 || kWarpRow || !kRes;
  if (kAhead && first < a.m) load(first);
  // e4m3 codes of float32 rows whose s is a power of two: see norm_scale
  constexpr bool kAskAgain = OUT == SP24_FP8 && sizeof(T) == 4;
  bool again = false;
  uint32_t buf = 0;
  for (int64_t row = first; row < a.m; row += step, buf ^= 1u) {
    if (!kAhead) load(row);
    Vec8<T> h[NV];
    Pair sum2 = pair(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * nt;
      h[i] = norm_sum<T>(x[i], r[i], res, sum2);
      if (a.h != nullptr && c < c_end) h[i].store(static_cast<T*>(a.h) + row * a.k + 8 * c);
    }
    if (kAhead && row + step < a.m) load(row + step);
    float sum, odd;
    split(sum2, sum, odd);
    const float2 rs = norm_rstd(
        row_sum<kWarpRow, double>(sum + odd, part[buf], threadIdx.x >> 5, blockDim.x >> 5, 0), a);
    norm_row_end<OUT>(a, row, t, rs);
    if (kAskAgain) again |= rs.y == 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * nt;
      Vec8<T> g;
      g.zero();
      if (c < c_end) g.load_cached(static_cast<const T*>(a.gamma) + 8 * c);
      norm_out<T, OUT>(a, h[i], g, rs, row, c, c < c_end, sx, rsx);
    }
  }
  if constexpr (kAskAgain) {   // rows with such an s are written again (the same
    if (!again) return;        // answer in all of a row's threads)
    for (int64_t row = first; row < a.m; row += step, buf ^= 1u) {
      // h is read again, as stored (x may be overwritten by it)
      const T* hp = static_cast<const T*>(a.h != nullptr ? a.h : a.x) + row * a.k;
      const bool add = res && a.h == nullptr;
      Vec8<T> h[NV];
      Pair sum2 = pair(0.0f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = t + i * nt;
        Vec8<T> v, w;
        v.zero();
        w.zero();
        if (c < c_end) {
          v.load(hp + 8 * c);
          if (add) w.load(static_cast<const T*>(a.r) + row * a.k + 8 * c);
        }
        h[i] = norm_sum<T>(v, w, add, sum2);
      }
      float sum, odd;
      split(sum2, sum, odd);
      const float2 rs = norm_rstd(
          row_sum<kWarpRow, double>(sum + odd, part[buf], threadIdx.x >> 5, blockDim.x >> 5, 0), a);
      if (!norm_pow2(rs)) continue;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = t + i * nt;
        Vec8<T> g;
        g.zero();
        if (c < c_end) g.load_cached(static_cast<const T*>(a.gamma) + 8 * c);
        norm_out<T, OUT, kAsk>(a, h[i], g, rs, row, c, c < c_end, sx, rsx);
      }
    }
  }
}

// ------------------------------------------------------------ quantisation
// e4m3 codes of [m][k] by blocks of 128 columns.  A half-warp takes a block and
// a thread kQuantUnroll of its vectors of 8 columns, all loaded before the first
// is used; blocks are numbered through the rows, so consecutive half-warps read
// consecutive memory whatever the row length.  One pass per CTA (8192 x 11008
// bf16: 49.0 us, 5.5 TB/s; a grid of resident CTAs that loop 52.9, eight vectors
// a thread 52.3, two 51.9).
constexpr int kQuantUnroll = 4;
constexpr int kQuantThreads = 256;

// Quotient by a fixed divisor of numbers below 2^31 (the round-up method of
// Granlund and Montgomery, "Division by invariant integers using multiplication",
// 1994): with l = ceil(log2 d) and mul = floor(2^32 (2^l - d) / d) + 1 it is
// (mulhi(n, mul) + n) >> l.
struct FastDiv {
  uint32_t mul, shift;
  FastDiv(uint32_t d = 1) {
    shift = 0;
    while ((uint64_t(1) << shift) < d) ++shift;
    mul = static_cast<uint32_t>((((uint64_t(1) << shift) - d) << 32) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return (__umulhi(n, mul) + n) >> shift;
  }
};

struct QuantArgs {
  const void* x;
  uint8_t* y;
  uint8_t* e;
  int64_t k;
  uint32_t blocks;      // m * kb
  uint32_t kb;          // blocks of a row
  FastDiv by_kb;
  uint32_t pad_cols;    // 128 * kb - k
  uint32_t pad_scales;  // scale columns past kb
};

// Largest magnitude of eight values, as float bits.
__device__ __forceinline__ uint32_t amax8(const Vec8<__nv_bfloat16>& v) {
  constexpr uint32_t kM = 0x7FFF7FFFu;
  const uint32_t m = max_u16x2(max_u16x2(v.q.x & kM, v.q.y & kM), max_u16x2(v.q.z & kM, v.q.w & kM));
  return max(m & 0xFFFFu, m >> 16) << 16;
}
__device__ __forceinline__ uint32_t amax8(const Vec8<float>& v) {
  constexpr uint32_t kM = 0x7FFFFFFFu;
  return max(max(max(v.a.x & kM, v.a.y & kM), max(v.a.z & kM, v.a.w & kM)),
             max(max(v.b.x & kM, v.b.y & kM), max(v.b.z & kM, v.b.w & kM)));
}

template <typename T>
__global__ void __launch_bounds__(kQuantThreads) quantize_fp8_kernel(const QuantArgs a) {
  pdl_launch_dependents();
  pdl_wait_prior();
  constexpr uint32_t kHalves = kQuantThreads / 16;
  const uint32_t hw = threadIdx.x >> 4, t = threadIdx.x & 15;
  // 32-bit block numbers: m * kb < 2^31, checked by the host
  const uint32_t b0 = blockIdx.x * (kHalves * kQuantUnroll) + hw;
  Vec8<T> x[kQuantUnroll];
  int64_t at[kQuantUnroll];   // element of the thread's vector, -1 past the row or the end
#pragma unroll
  for (int u = 0; u < kQuantUnroll; ++u) {
    const uint32_t b = b0 + u * kHalves;
    const uint32_t row = a.by_kb(b);
    // columns end inside a row's last block only (a column may pass 32 bits)
    const bool ok = b < a.blocks && (b - row * a.kb + 1 < a.kb || 8 * t + a.pad_cols < 128);
    at[u] = ok ? static_cast<int64_t>(b) * 128 + 8 * t - static_cast<int64_t>(row) * a.pad_cols : -1;
    x[u].zero();
    if (ok) x[u].load(static_cast<const T*>(a.x) + at[u]);
  }
#pragma unroll
  for (int u = 0; u < kQuantUnroll; ++u) {
    const uint32_t amax = block_max(amax8(x[u]));
    const uint32_t byte = scale_byte(amax);
    const float inv = scale_inverse(byte);
    if (at[u] >= 0) {
      Pair f[4];
      x[u].get(f);
      const uint2 q = e4m3x8(f, inv);
      *reinterpret_cast<uint2*>(a.y + at[u]) = q;
      if (t == 0) {   // the scale, and after a row's last block the row's padding
        const uint32_t b = b0 + u * kHalves, row = a.by_kb(b);
        uint8_t* e = a.e + b + static_cast<int64_t>(row) * a.pad_scales;
        e[0] = static_cast<uint8_t>(byte);
        if (b - row * a.kb == a.kb - 1)
          for (uint32_t i = 1; i <= a.pad_scales; ++i) e[i] = static_cast<uint8_t>(kScaleOne);
      }
    }
  }
}

// ----------------------------------------------------------------- backward
// With t = dy * h:  dgamma = sum over rows of t * rstd, and
//   dx = rstd * dy * gamma - h * c [+ dh],  c = rstd^3 * mean(t * gamma),
// which is rstd * (g - xh * mean(g * xh)) with g = dy * gamma, xh = h * rstd.
// Bound by HBM: dy, h (and dh) are read once and dx is written once.
//
// A block holds groups of T threads, a row each at a time; a thread keeps the
// dgamma sums of its columns over all its rows.  At the end the groups' sums are
// added in order through shared memory and the block writes one row of the
// workspace; dgamma_kernel adds those rows in order (no atomics: the same
// inputs give the same bits).  Groups keep the workspace short (509 x 768: 5.1
// us with four rows a block, 9.3 with one; 2000 x 768 with five 8.3 and 10.5).
struct BackArgs {
  const void* dy;
  const void* dh;       // optional
  const void* h;
  const void* gamma;
  const float* rstd;
  void* dx;
  float* part;          // [gridDim.x][k]
  int64_t m, k;
};

constexpr int kBackSlots = 4;      // most rows in flight of a block of the ring kernel

template <typename T, int NV>
__global__ void __launch_bounds__(512) norm_back_kernel(const BackArgs a, int group_threads) {
  pdl_launch_dependents();
  pdl_wait_prior();
  __shared__ float part[2][32];
  extern __shared__ float s_acc[];   // [groups][k], one group: unused
  const int groups = static_cast<int>(blockDim.x) / group_threads;
  const int grp = static_cast<int>(threadIdx.x) / group_threads;
  const int t = static_cast<int>(threadIdx.x) - grp * group_threads;
  const int warps = group_threads >> 5;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + grp;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int c_end = static_cast<int>(a.k / 8);
  const float inv_k = __fdiv_rn(1.0f, static_cast<float>(a.k));
  const bool has_dh = a.dh != nullptr;

  Pair acc[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = pair(0.0f);

  // the next row's dy and h are loaded before this one is reduced, where the
  // registers allow
  constexpr bool kAhead = NV <= 2;
  Vec8<T> dy[NV], h[NV];
  float rs_next = 0.0f;
  auto load = [&](int64_t row) {
    const int64_t base = row * a.k;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * group_threads;
      dy[i].zero();
      h[i].zero();
      if (c < c_end) {
        dy[i].load(static_cast<const T*>(a.dy) + base + 8 * c);
        h[i].load(static_cast<const T*>(a.h) + base + 8 * c);
      }
    }
    rs_next = a.rstd[row];
  };
  if (kAhead && first < a.m) load(first);
  uint32_t buf = 0;
  for (int64_t row = first; row < a.m; row += step, buf ^= 1u) {
    if (!kAhead) load(row);
    const float rs = rs_next;
    Vec8<T> cdy[NV], ch[NV], dh[NV];
    Pair dot2 = pair(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * group_threads;
      cdy[i] = dy[i];
      ch[i] = h[i];
      if (kAhead && has_dh && c < c_end) dh[i].load(static_cast<const T*>(a.dh) + row * a.k + 8 * c);
      Vec8<T> g;
      g.zero();
      if (c < c_end) g.load_cached(static_cast<const T*>(a.gamma) + 8 * c);
      Pair fd[4], fh[4], fg[4];
      cdy[i].get(fd);
      ch[i].get(fh);
      g.get(fg);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Pair p = mul2(fd[j], fh[j]);
        acc[i][j] = fma2(p, pair(rs), acc[i][j]);
        dot2 = fma2(p, fg[j], dot2);
      }
    }
    if (kAhead && row + step < a.m) load(row + step);
    float dot, odd;
    split(dot2, dot, odd);
    dot = row_sum<false, float>(dot + odd, part[buf] + grp * warps, t >> 5, warps, 1 + grp);
    const float coef = -(dot * inv_k) * rs * rs * rs;
    T* out = static_cast<T*>(a.dx) + row * a.k;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * group_threads;
      if (c < c_end) {
        Vec8<T> g, o;
        g.load_cached(static_cast<const T*>(a.gamma) + 8 * c);
        if (!kAhead && has_dh) dh[i].load(static_cast<const T*>(a.dh) + row * a.k + 8 * c);
        Pair fd[4], fh[4], fg[4], fo[4];
        cdy[i].get(fd);
        ch[i].get(fh);
        g.get(fg);
        if (has_dh) {
          dh[i].get(fo);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) fo[j] = pair(0.0f);
        }
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          split(fma2(mul2(fd[j], fg[j]), pair(rs), fma2(fh[j], pair(coef), fo[j])), f[2 * j],
                f[2 * j + 1]);
        o.set(f);
        o.store(out + 8 * c);
      }
    }
  }
  float* dst = a.part + static_cast<int64_t>(blockIdx.x) * a.k;
  float* sums = groups > 1 ? s_acc + grp * a.k : dst;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t + i * group_threads;
    if (c < c_end) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) split(acc[i][j], f[2 * j], f[2 * j + 1]);
      float4* q = reinterpret_cast<float4*>(sums + 8 * c);
      q[0] = make_float4(f[0], f[1], f[2], f[3]);
      q[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
  if (groups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < a.k; c += blockDim.x) {
      float s = 0.0f;
      for (int i = 0; i < groups; ++i) s += s_acc[i * a.k + c];
      dst[c] = s;
    }
  }
}

// The same for rows too long for the registers: one row a block at a time, the
// rows in `slots` slots of dy, h (and dh) in shared memory, filled by bulk copies
// that run ahead (2000 x 11008 with dh: 37.5 us; four vectors a thread in
// registers 72.7.  8192 x 4096: 49.7 against 50.4; 8192 x 768: 18.2 against 15.1).
// A slot is read in both passes over its row; it is refilled after the next
// row's sum, whose barrier says that the block has left it.
template <typename T, int NV>
__global__ void __launch_bounds__(1024) norm_back_ring_kernel(const BackArgs a, int slots) {
  pdl_launch_dependents();
  extern __shared__ __align__(128) uint8_t ring[];   // gamma, then the slots
  __shared__ float part[2][32];
  __shared__ uint64_t full[kBackSlots];
  const int t = static_cast<int>(threadIdx.x), nt = static_cast<int>(blockDim.x);
  const int64_t first = blockIdx.x, step = gridDim.x;
  const int c_end = static_cast<int>(a.k / 8);
  const float inv_k = __fdiv_rn(1.0f, static_cast<float>(a.k));
  const bool has_dh = a.dh != nullptr;
  const uint32_t row_bytes = static_cast<uint32_t>(a.k * sizeof(T));
  const uint32_t slot_bytes = row_bytes * (has_dh ? 3 : 2);
  const T* gamma = reinterpret_cast<const T*>(ring);
  if (t == 0) {
    for (int i = 0; i < slots; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  pdl_wait_prior();
  for (int c = t; c < c_end; c += nt) {
    Vec8<T> g;
    g.load_cached(static_cast<const T*>(a.gamma) + 8 * c);
    g.store(reinterpret_cast<T*>(ring) + 8 * c);
  }
  __syncthreads();
  auto fill = [&](int64_t row, int slot) {
    uint8_t* dst = ring + row_bytes + slot * slot_bytes;
    mbar_arrive_expect_tx(&full[slot], slot_bytes);
    bulk_load(dst, static_cast<const T*>(a.dy) + row * a.k, row_bytes, &full[slot]);
    bulk_load(dst + row_bytes, static_cast<const T*>(a.h) + row * a.k, row_bytes, &full[slot]);
    if (has_dh)
      bulk_load(dst + 2 * row_bytes, static_cast<const T*>(a.dh) + row * a.k, row_bytes, &full[slot]);
  };
  if (t == 0)
    for (int i = 0; i < slots && first + i * step < a.m; ++i) fill(first + i * step, i);

  Pair acc[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = pair(0.0f);

  int slot = 0, prev = 0;
  uint32_t ph = 0, buf = 0;
  for (int64_t row = first; row < a.m; row += step, buf ^= 1u) {
    const float rs = __ldg(a.rstd + row);
    mbar_wait(&full[slot], ph);
    const T* dy = reinterpret_cast<const T*>(ring + row_bytes + slot * slot_bytes);
    const T* h = dy + a.k;
    Pair dot2 = pair(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * nt;
      if (c < c_end) {
        Vec8<T> vd, vh, vg;
        vd.load_shared(dy + 8 * c);
        vh.load_shared(h + 8 * c);
        vg.load_shared(gamma + 8 * c);
        Pair fd[4], fh[4], fg[4];
        vd.get(fd);
        vh.get(fh);
        vg.get(fg);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const Pair p = mul2(fd[j], fh[j]);
          acc[i][j] = fma2(p, pair(rs), acc[i][j]);
          dot2 = fma2(p, fg[j], dot2);
        }
      }
    }
    float dot, odd;
    split(dot2, dot, odd);
    dot = row_sum<false, float>(dot + odd, part[buf], t >> 5, nt >> 5, 0);
    // the previous row's slot: its next row is `slots` rows after that row
    if (t == 0 && row != first) {
      const int64_t next = row + (slots - 1) * step;
      if (next < a.m) {
        fence_async_shared();
        fill(next, prev);
      }
    }
    const float coef = -(dot * inv_k) * rs * rs * rs;
    T* out = static_cast<T*>(a.dx) + row * a.k;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * nt;
      if (c < c_end) {
        Vec8<T> vd, vh, vg, o;
        vd.load_shared(dy + 8 * c);
        vh.load_shared(h + 8 * c);
        vg.load_shared(gamma + 8 * c);
        Pair fd[4], fh[4], fg[4], fo[4];
        vd.get(fd);
        vh.get(fh);
        vg.get(fg);
        if (has_dh) {
          o.load_shared(h + a.k + 8 * c);
          o.get(fo);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) fo[j] = pair(0.0f);
        }
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          split(fma2(mul2(fd[j], fg[j]), pair(rs), fma2(fh[j], pair(coef), fo[j])), f[2 * j],
                f[2 * j + 1]);
        o.set(f);
        o.store(out + 8 * c);
      }
    }
    prev = slot;
    if (++slot == slots) {
      slot = 0;
      ph ^= 1u;
    }
  }
  float* dst = a.part + static_cast<int64_t>(blockIdx.x) * a.k;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t + i * nt;
    if (c < c_end) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) split(acc[i][j], f[2 * j], f[2 * j + 1]);
      float4* q = reinterpret_cast<float4*>(dst + 8 * c);
      q[0] = make_float4(f[0], f[1], f[2], f[3]);
      q[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
}

// dgamma[c] = sum over p rows of part, 32 columns per block: 32 groups of 8
// threads (one float4 each) take every 32nd row, then the groups are added in
// order.
__global__ void __launch_bounds__(256) dgamma_kernel(const float* part, int p, int64_t k,
                                                     float* dgamma) {
  pdl_launch_dependents();
  pdl_wait_prior();
  __shared__ float s[32][33];
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 7) * 4;
  const int grp = threadIdx.x >> 3;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < k) {
#pragma unroll 8
    for (int i = grp; i < p; i += 32) {
      const float4 q = __ldcg(reinterpret_cast<const float4*>(part + static_cast<int64_t>(i) * k + c));
      v.x += q.x;
      v.y += q.y;
      v.z += q.z;
      v.w += q.w;
    }
  }
  float* d = &s[grp][(threadIdx.x & 7) * 4];
  d[0] = v.x;
  d[1] = v.y;
  d[2] = v.z;
  d[3] = v.w;
  __syncthreads();
  if (threadIdx.x < 32) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    if (col < k) dgamma[col] = t;
  }
}

// -------------------------------------------------------------- launching
// Resident blocks per SM of a kernel at `threads` threads, asked once per
// device and block size (the gradient's groups take at most 64 bytes of shared
// memory a thread, 128 KB of a full SM, so its size never decides the answer and
// the grid depends on the sizes of the call alone).
struct Occupancy {
  std::atomic<int> per_sm[64][33];   // zero-initialised (static storage)
};

static sp24_status resident_blocks(const void* kern, Occupancy& o, int threads, size_t smem, int* out) {
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return cuda_fail("cudaGetDevice", e);
  std::atomic<int>& slot = o.per_sm[dev & 63][threads / 32];
  int n = slot.load(std::memory_order_acquire);
  if (n == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem);
    if (e != cudaSuccess) return cuda_fail("cudaOccupancyMaxActiveBlocksPerMultiprocessor", e);
    if (n < 1) return SP24_ERR_UNSUPPORTED;
    slot.store(n, std::memory_order_release);
  }
  *out = n;
  return SP24_OK;
}

template <typename T, int OUT, int NV, bool kWarpRow, int MAXT, int MINB, bool kRes = true>
static sp24_status launch_norm_t(const NormArgs& a, int threads, cudaStream_t s) {
  auto kern = norm_kernel<T, OUT, NV, kWarpRow, MAXT, MINB, kRes>;
  static Occupancy occ;
  int per_sm = 0;
  SP24_TRY(resident_blocks(reinterpret_cast<const void*>(kern), occ, threads, 0, &per_sm));
  const int64_t per_cta = kWarpRow ? threads / 32 : 1;
  const int64_t ctas = (a.m + per_cta - 1) / per_cta;
  const int64_t cap = static_cast<int64_t>(sm_count()) * per_sm;
  return launch_kernel(kern, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)), dim3(threads), 0,
                       s, 1, a);
}

static int round32(int64_t v) { return static_cast<int>((v + 31) / 32 * 32); }

template <typename T, int OUT>
static sp24_status launch_norm(const NormArgs& a, cudaStream_t s) {
  const int64_t c = a.k / 8;   // vectors of a row
  if (c <= 32) return launch_norm_t<T, OUT, 1, true, 256, 1>(a, 256, s);
  if (c <= 64) return launch_norm_t<T, OUT, 2, true, 256, 1>(a, 256, s);
  // One vector a thread where a block can have that many threads: always for
  // float32 (2000 x 4096 with residual: 19.6 us, two vectors 23.6) and up to
  // 1024 columns (4096 x 768: 5.9 us, a warp with four vectors 7.2), for bf16
  // otherwise only when the rows are few; with many rows two vectors a thread keep more
  // bytes in flight (8192 x 4096: 39.7 us, one vector 45.1, four 41.8).
  if (c <= 1024 && (c <= 128 || sizeof(T) == 4 || a.m <= 2 * sm_count()))
    return launch_norm_t<T, OUT, 1, false, 1024, 1>(a, round32(c), s);
  // Long float32 rows without a residual, more than one an SM: three vectors a
  // thread in two blocks an SM, whose 64 registers hold the next row as well but
  // for a few values (8 bytes of spills for e4m3, 36 for the other outputs).
  // Against two vectors without the next row: 777 x 11008 to e4m3 13.9 and 17.1 us,
  // to int8 17.1 and 19.7, to bf16 12.8 and 15.4; 1000 x 9216 15.0 and 17.9; 2000 x
  // 11008 29.2 and 39.3.  With a residual, or a row an SM, two vectors (100 x 11008:
  // 3.9 us, three 5.1).
  if constexpr (sizeof(T) == 4) {
    if (c > 1024 && c <= 1536 && a.r == nullptr && a.m > sm_count())
      return launch_norm_t<T, OUT, 3, false, 512, 2, false>(a, round32((c + 2) / 3), s);
  }
  return launch_norm_t<T, OUT, 2, false, 1024, 1>(a, round32((c + 1) / 2), s);
}

template <typename T>
static sp24_status launch_norm_out(const NormArgs& a, int out, cudaStream_t s) {
  switch (out) {
    case SP24_FP8: return launch_norm<T, SP24_FP8>(a, s);
    case SP24_INT8: return launch_norm<T, SP24_INT8>(a, s);
    default: return launch_norm<T, SP24_BF16>(a, s);
  }
}

template <typename T>
static sp24_status launch_quantize(const QuantArgs& a, cudaStream_t s) {
  const uint32_t per_cta = kQuantThreads / 16 * kQuantUnroll;
  return launch_kernel(quantize_fp8_kernel<T>, dim3((a.blocks + per_cta - 1) / per_cta),
                       dim3(kQuantThreads), 0, s, 1, a);
}

// Rows of the dgamma workspace: at most this many blocks run the backward.
constexpr int64_t kBackMaxCtas = 640;

template <typename T, int NV>
static sp24_status launch_back_t(const BackArgs& a, int group_threads, float* dgamma,
                                 cudaStream_t s) {
  auto kern = norm_back_kernel<T, NV>;
  static Occupancy occ;
  // as many groups as 512 threads hold (their hardware barriers are 1 .. 15),
  // fewer where the rows are few
  int64_t groups = 512 / group_threads;
  if (groups > 15) groups = 15;
  const int64_t spread = (a.m + sm_count() - 1) / sm_count();
  if (groups > spread) groups = spread < 1 ? 1 : spread;
  const int threads = static_cast<int>(groups) * group_threads;
  const size_t smem = groups > 1 ? static_cast<size_t>(groups) * a.k * 4 : 0;
  int per_sm = 0;
  SP24_TRY(resident_blocks(reinterpret_cast<const void*>(kern), occ, threads, smem, &per_sm));
  int64_t ctas = (a.m + groups - 1) / groups;
  const int64_t cap = static_cast<int64_t>(sm_count()) * per_sm;
  if (ctas > cap) ctas = cap;
  if (ctas > kBackMaxCtas) ctas = kBackMaxCtas;
  if (ctas > 0)
    SP24_TRY(launch_kernel(kern, dim3(static_cast<unsigned>(ctas)), dim3(threads), smem, s, 1, a,
                           group_threads));
  return launch_kernel(dgamma_kernel, dim3(static_cast<unsigned>((a.k + 31) / 32)), dim3(256), 0, s,
                       1, static_cast<const float*>(a.part), static_cast<int>(ctas), a.k, dgamma);
}

// Shared memory of the ring kernel: gamma and the slots.
constexpr int64_t kBackRing = 224 * 1024;

template <typename T, int NV>
static sp24_status launch_back_ring(const BackArgs& a, int threads, int slots, float* dgamma,
                                    cudaStream_t s) {
  auto kern = norm_back_ring_kernel<T, NV>;
  static std::atomic<uint64_t> smem_set{0};   // one bit per device
  SP24_TRY(set_smem_once(reinterpret_cast<const void*>(kern), static_cast<int>(kBackRing), smem_set));
  const size_t smem = (1 + static_cast<size_t>(slots) * (a.dh ? 3 : 2)) * a.k * sizeof(T);
  const int64_t cap = sm_count() < kBackMaxCtas ? sm_count() : kBackMaxCtas;
  const int64_t ctas = a.m < cap ? a.m : cap;
  if (ctas > 0)
    SP24_TRY(launch_kernel(kern, dim3(static_cast<unsigned>(ctas)), dim3(threads), smem, s, 1, a,
                           slots));
  return launch_kernel(dgamma_kernel, dim3(static_cast<unsigned>((a.k + 31) / 32)), dim3(256), 0, s,
                       1, static_cast<const float*>(a.part), static_cast<int>(ctas), a.k, dgamma);
}

template <typename T>
static sp24_status launch_back(const BackArgs& a, float* dgamma, cudaStream_t s) {
  const int64_t c = a.k / 8;   // vectors of a row
  if (c <= 256) return launch_back_t<T, 1>(a, round32(c), dgamma, s);
  if (c <= 1024) return launch_back_t<T, 2>(a, round32((c + 1) / 2), dgamma, s);
  const int64_t row = a.k * static_cast<int64_t>(sizeof(T));
  const int64_t slots = (kBackRing - row) / ((a.dh ? 3 : 2) * row);
  if constexpr (sizeof(T) == 4)   // two float32 rows may not fit (bf16 rows always do)
    if (slots < 2) return launch_back_t<T, 4>(a, round32((c + 3) / 4), dgamma, s);
  static_assert(kBackRing >= 7 * SP24_NORM_MAX_K * 2, "two bf16 rows of dy, h and dh, and gamma");
  return launch_back_ring<T, 2>(a, round32((c + 1) / 2),
                                static_cast<int>(slots < kBackSlots ? slots : kBackSlots), dgamma, s);
}

}  // namespace sp24

using namespace sp24;

extern "C" {

sp24_status sp24_rmsnorm_quant(const void* X, const void* R, const void* gamma, int64_t M,
                               int64_t K, int x_dtype, float eps, int out_dtype, const float* s_x,
                               void* H, void* Y, uint8_t* e_y, float* rstd, void* stream) {
  if (M < 0 || K < 1 || (x_dtype != SP24_BF16 && x_dtype != SP24_F32) ||
      (out_dtype != SP24_FP8 && out_dtype != SP24_INT8 && out_dtype != SP24_BF16) || !(eps >= 0.0f))
    return SP24_ERR_ARG;
  if (K % 16 != 0) return SP24_ERR_ALIGN;
  if (K > SP24_NORM_MAX_K) return SP24_ERR_UNSUPPORTED;
  if (M == 0) return SP24_OK;
  if (!X || !gamma || !Y || (out_dtype == SP24_FP8 && !e_y) || (out_dtype == SP24_INT8 && !s_x))
    return SP24_ERR_ARG;
  if (!aligned16(X) || !aligned16(gamma) || !aligned16(Y) || (R && !aligned16(R)) ||
      (H && !aligned16(H)) || (out_dtype == SP24_FP8 && !aligned16(e_y)))
    return SP24_ERR_ALIGN;
  SP24_TRY(check_device());
  NormArgs a{};
  a.x = X;
  a.r = R;
  a.gamma = gamma;
  a.h = H;
  a.y = Y;
  a.e = e_y;
  a.rstd = rstd;
  a.s_x = s_x;
  a.m = M;
  a.k = K;
  a.inv_k = 1.0 / static_cast<double>(K);
  a.eps = eps;
  a.scale_cols = static_cast<int>(4 * ((K + 511) / 512));
  return x_dtype == SP24_F32 ? launch_norm_out<float>(a, out_dtype, as_stream(stream))
                             : launch_norm_out<__nv_bfloat16>(a, out_dtype, as_stream(stream));
}

sp24_status sp24_quantize_fp8(const void* X, int64_t M, int64_t K, int x_dtype, void* Xq,
                              uint8_t* e_x, void* stream) {
  if (M < 0 || K < 1 || (x_dtype != SP24_BF16 && x_dtype != SP24_F32)) return SP24_ERR_ARG;
  if (K % 16 != 0) return SP24_ERR_ALIGN;
  if (M == 0) return SP24_OK;
  if (!X || !Xq || !e_x) return SP24_ERR_ARG;
  if (!aligned16(X) || !aligned16(Xq) || !aligned16(e_x)) return SP24_ERR_ALIGN;
  const int64_t kb = K / 128 + (K % 128 != 0);
  if (kb > 0x7FFFFFFF / M) return SP24_ERR_UNSUPPORTED;   // more blocks than 32 bits number
  SP24_TRY(check_device());
  QuantArgs a{};
  a.x = X;
  a.y = static_cast<uint8_t*>(Xq);
  a.e = e_x;
  a.k = K;
  a.blocks = static_cast<uint32_t>(M * kb);
  a.kb = static_cast<uint32_t>(kb);
  a.by_kb = FastDiv(a.kb);
  a.pad_cols = static_cast<uint32_t>(128 * kb - K);
  a.pad_scales = static_cast<uint32_t>(4 * ((K + 511) / 512) - kb);
  return x_dtype == SP24_F32 ? launch_quantize<float>(a, as_stream(stream))
                             : launch_quantize<__nv_bfloat16>(a, as_stream(stream));
}

size_t sp24_rmsnorm_backward_workspace_bytes(int64_t M, int64_t K) {
  if (M < 0 || K < 1 || K > SP24_NORM_MAX_K) return 0;
  const int64_t rows = M < 1 ? 1 : (M < kBackMaxCtas ? M : kBackMaxCtas);
  return static_cast<size_t>(rows) * static_cast<size_t>(K) * sizeof(float);
}

sp24_status sp24_rmsnorm_backward(const void* dY, const void* dH, const void* H, const void* gamma,
                                  const float* rstd, int64_t M, int64_t K, int x_dtype, void* dX,
                                  float* dgamma, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  if (M < 0 || K < 1 || (x_dtype != SP24_BF16 && x_dtype != SP24_F32)) return SP24_ERR_ARG;
  if (K % 16 != 0) return SP24_ERR_ALIGN;
  if (K > SP24_NORM_MAX_K) return SP24_ERR_UNSUPPORTED;
  if (!dgamma || !workspace || workspace_bytes < sp24_rmsnorm_backward_workspace_bytes(M, K))
    return SP24_ERR_ARG;
  if (M > 0 && (!dY || !H || !gamma || !rstd || !dX)) return SP24_ERR_ARG;
  if (!aligned16(dgamma) || !aligned16(workspace) || (M > 0 && (!aligned16(dY) || !aligned16(H) ||
      !aligned16(gamma) || !aligned16(dX))) || (dH && !aligned16(dH)))
    return SP24_ERR_ALIGN;
  SP24_TRY(check_device());
  BackArgs a{};
  a.dy = dY;
  a.dh = dH;
  a.h = H;
  a.gamma = gamma;
  a.rstd = rstd;
  a.dx = dX;
  a.part = static_cast<float*>(workspace);
  a.m = M;
  a.k = K;
  return x_dtype == SP24_F32 ? launch_back<float>(a, dgamma, as_stream(stream))
                             : launch_back<__nv_bfloat16>(a, dgamma, as_stream(stream));
}

}  // extern "C"
