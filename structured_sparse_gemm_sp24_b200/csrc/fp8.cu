// libsp24: e4m3 conversion of a 2:4 weight (sp24_prune_compress_fp8,
// sp24_compress_fp8).
//
// The mask is that of sp24_prune (n_keep = 2); the kept values of each 128 x
// 128 block of W share one power-of-two scale (fp8.cuh); values, metadata and
// scales are what sp24_gemm_fp8 reads.  HBM-bound: 2NK bytes in, NK/2 values,
// NK/8 metadata and (asked for) NK/8 mask bytes out.
//
// One CTA per 128 x 128 block: every 16-byte vector of W (8 K-positions) is
// loaded once and stays in registers between the block's maximum and its
// conversion.  Thread t takes vector t % 16 of block rows t / 16 + 16 j, so a
// half-warp reads 256 contiguous bytes; the metadata (the int8 layout: 16
// bytes per row) and the mask bytes leave through shared memory in 16-byte
// pieces.

#include "fp8.cuh"
#include "sp24_host.h"

namespace sp24 {

constexpr int kConvThreads = 256;
constexpr int kConvRows = 128 / (kConvThreads / 16);   // vectors per thread

struct ConvertArgs {
  const uint16_t* w;
  int64_t n, k;
  const double* norms;       // Wanda
  const uint8_t* mask_in;    // mask to apply (kPrune: optional, dropped weights score 0)
  uint8_t* mask_out;         // optional
  uint32_t* vals;            // 4 codes per vector
  uint8_t* meta;
  uint8_t* e_w;              // [ceil(n/128)][scale_cols]
  int kblocks;
  int scale_cols;
};

// Magnitude selection of two groups of four at once: q.x, q.y hold the first
// group (positions 0..3), q.z, q.w the second.  Position p of both groups is
// put into the halves of one word as a 15-bit magnitude, so comparisons run two
// at a time with the free top bit of each half as the guard: the top bit of
// (x | 8000) - y says x >= y.  With a >= b the ordered positions 0, 1 and c >= d
// the ordered 2, 3 (ties to the lower index), the two kept are
//   0, 1 if b >= c;  2, 3 if d > a;  the larger of either pair otherwise.
// Returns the two metadata nibbles lo | hi << 2 in one byte; `top` receives the
// largest magnitude of either group (always kept).
__device__ __forceinline__ uint32_t select2_mag(const uint4& q, uint32_t& top) {
  constexpr uint32_t kG = 0x80008000u, kM = 0x7FFF7FFFu;
  const uint32_t x = q.x & kM, y = q.y & kM, z = q.z & kM, w = q.w & kM;
  const uint32_t p0 = __byte_perm(x, z, 0x5410), p1 = __byte_perm(x, z, 0x7632);
  const uint32_t p2 = __byte_perm(y, w, 0x5410), p3 = __byte_perm(y, w, 0x7632);
  const uint32_t a = max_u16x2(p0, p1), b = min_u16x2(p0, p1);
  const uint32_t c = max_u16x2(p2, p3), d = min_u16x2(p2, p3);
  const uint32_t ge01 = (p0 | kG) - p1;   // flags in bits 15 and 31
  const uint32_t ge23 = (p2 | kG) - p3;
  const uint32_t first = (b | kG) - c;    // keep 0, 1
  const uint32_t not_last = (a | kG) - d; // clear: keep 2, 3
  top = max_u16x2(a, c);
  const uint32_t lo0 = ~first & not_last & ~ge01, lo1 = ~not_last;
  const uint32_t hi0 = first | ~not_last | ~ge23, hi1 = ~first;
  const uint32_t t = ((lo0 >> 15) & 0x00010001u) | ((lo1 >> 14) & 0x00020002u) |
                     ((hi0 >> 13) & 0x00040004u) | ((hi1 >> 12) & 0x00080008u);
  return (t | (t >> 12)) & 0xFFu;
}

// Kept pair of a group (w0, w1 its four bf16) from its metadata nibble.
__device__ __forceinline__ uint32_t gather_code(uint32_t w0, uint32_t w1, uint32_t code) {
  return __byte_perm(w0, w1, 0x1010u + 0x22u * (code & 3u) + 0x880u * (code & 12u));
}

// kPrune: the mask is formed here (kWanda: scores |w| * norm; kMaskIn: positions
// dropped by mask_in score 0), else mask_in is the mask.
template <bool kPrune, bool kWanda, bool kMaskIn>
__global__ void __launch_bounds__(kConvThreads) convert_fp8_kernel(const ConvertArgs a) {
  pdl_launch_dependents();
  pdl_wait_prior();
  __shared__ __align__(16) uint8_t s_meta[2048];
  __shared__ __align__(16) uint8_t s_mask[2048];
  __shared__ uint32_t s_max[kConvThreads / 32];
  const int tid = threadIdx.x;
  const int rt = static_cast<int>(blockIdx.x / a.kblocks);
  const int kb = static_cast<int>(blockIdx.x) - rt * a.kblocks;
  const int bb = tid & 15, m0 = tid >> 4;
  const int64_t kvec = a.k / 8;
  const int64_t v = static_cast<int64_t>(kb) * 16 + bb;
  const int64_t row0 = static_cast<int64_t>(rt) * 128 + m0;
  // rows m0, m0 + 16, ... of the block that exist (for this thread's columns)
  const int64_t left = v < kvec ? a.n - row0 : 0;
  const int rows = left <= 0 ? 0 : (left >= 128 ? kConvRows : static_cast<int>((left + 15) / 16));

  uint4 q[kConvRows];
  const uint4* src = reinterpret_cast<const uint4*>(a.w) + row0 * kvec + v;
#pragma unroll
  for (int j = 0; j < kConvRows; ++j) {
    q[j] = make_uint4(0u, 0u, 0u, 0u);
    if (j < rows) q[j] = __ldcs(src + 16 * j * kvec);
  }
  double nrm[8];
  if constexpr (kWanda) {
#pragma unroll
    for (int e = 0; e < 8; ++e) nrm[e] = rows > 0 ? __ldg(a.norms + 8 * v + e) : 0.0;
  }

  uint32_t bad = 0, amax = 0;
  uint32_t p0[kConvRows], p1[kConvRows];   // kept pairs of the two groups
#pragma unroll
  for (int j = 0; j < kConvRows; ++j) {
    uint32_t code = 0x44u;                 // padding: positions (0, 1)
    if constexpr (kPrune && !kWanda && !kMaskIn) {
      uint32_t top;
      code = select2_mag(q[j], top);       // (zeros keep 0, 1)
      amax = max_u16x2(amax, top);          // both halves hold magnitudes
    } else {
      uint32_t keep = 0x33u;
      if (j < rows) {
        uint32_t in = 0xFFu;
        if (!kPrune || kMaskIn) in = a.mask_in[(row0 + 16 * j) * kvec + v];
        if constexpr (!kPrune) keep = in;
        else if constexpr (kWanda) keep = mask_byte<true>(q[j], in, nrm, 2);
        else keep = keep_nibble_mag<true>(q[j].x, q[j].y, in & 15u, 2) |
                    (keep_nibble_mag<true>(q[j].z, q[j].w, in >> 4, 2) << 4);
        code = nibble_code(keep & 15u, bad) | (nibble_code(keep >> 4, bad) << 4);
      }
    }
    p0[j] = gather_code(q[j].x, q[j].y, code & 15u);
    p1[j] = gather_code(q[j].z, q[j].w, code >> 4);
    if constexpr (!(kPrune && !kWanda && !kMaskIn))
      amax = max_u16x2(amax, max_u16x2(p0[j] & 0x7FFF7FFFu, p1[j] & 0x7FFF7FFFu));
    s_meta[(m0 + 16 * j) * 16 + bb] = static_cast<uint8_t>(code);
    if (a.mask_out)
      s_mask[(m0 + 16 * j) * 16 + bb] = static_cast<uint8_t>(
          (1u << (code & 3u)) | (1u << ((code >> 2) & 3u)) | (16u << ((code >> 4) & 3u)) |
          (16u << (code >> 6)));
  }
  // a bf16's bits are the upper half of its float's
  amax = max(amax & 0xFFFFu, amax >> 16) << 16;
  amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kConvThreads / 32; ++i) amax = max(amax, s_max[i]);
  const uint32_t byte = scale_byte(amax);
  const float inv = scale_inverse(byte);
  uint32_t* dst = a.vals + row0 * kvec + v;
#pragma unroll
  for (int j = 0; j < kConvRows; ++j) {
    if (j < rows) {
      const uint32_t c = e4m3x4(__uint_as_float(p0[j] << 16) * inv,
                          __uint_as_float(p0[j] & 0xFFFF0000u) * inv,
                          __uint_as_float(p1[j] << 16) * inv,
                          __uint_as_float(p1[j] & 0xFFFF0000u) * inv);
      __stcs(dst + 16 * j * kvec, c);
    }
  }
  if (tid < 128) {
    uint4* md = reinterpret_cast<uint4*>(a.meta + static_cast<int64_t>(blockIdx.x) * 2048);
    __stcs(md + tid, reinterpret_cast<const uint4*>(s_meta)[tid]);
  } else if (a.mask_out) {
    const int m = tid - 128;
    const int64_t row = static_cast<int64_t>(rt) * 128 + m;
    const int64_t v0 = static_cast<int64_t>(kb) * 16;
    const int nb = static_cast<int>(kvec - v0 < 16 ? kvec - v0 : 16);   // K % 32: multiple of 4
    if (row < a.n) {
      uint32_t* mo = reinterpret_cast<uint32_t*>(a.mask_out + row * kvec + v0);
      for (int e = 0; e < nb / 4; ++e) mo[e] = reinterpret_cast<const uint32_t*>(s_mask)[m * 4 + e];
    }
  }
  // this block's scale, and the row's padding after the last block
  if (tid == 0) a.e_w[static_cast<int64_t>(rt) * a.scale_cols + kb] = static_cast<uint8_t>(byte);
  if (kb == a.kblocks - 1 && tid > 0 && kb + tid < a.scale_cols)
    a.e_w[static_cast<int64_t>(rt) * a.scale_cols + kb + tid] = static_cast<uint8_t>(kScaleOne);
  if (!kPrune && bad) raise_error(kErrPatternBit);
}

static sp24_status launch_convert_fp8(bool prune, bool wanda, ConvertArgs a, cudaStream_t s) {
  const int64_t kblocks = (a.k + 127) / 128;
  const int64_t nblocks = ((a.n + 127) / 128) * kblocks;
  if (nblocks > 0x7FFFFFFF) return SP24_ERR_UNSUPPORTED;
  a.kblocks = static_cast<int>(kblocks);
  a.scale_cols = static_cast<int>(4 * ((a.k + 511) / 512));
  const dim3 grid(static_cast<unsigned>(nblocks));
  const dim3 block(kConvThreads);
  if (!prune) return launch_kernel(convert_fp8_kernel<false, false, true>, grid, block, 0, s, 1, a);
  if (wanda)
    return a.mask_in ? launch_kernel(convert_fp8_kernel<true, true, true>, grid, block, 0, s, 1, a)
                     : launch_kernel(convert_fp8_kernel<true, true, false>, grid, block, 0, s, 1, a);
  return a.mask_in ? launch_kernel(convert_fp8_kernel<true, false, true>, grid, block, 0, s, 1, a)
                   : launch_kernel(convert_fp8_kernel<true, false, false>, grid, block, 0, s, 1, a);
}

}  // namespace sp24

using namespace sp24;

extern "C" {

sp24_status sp24_prune_compress_fp8(const void* W, int64_t N, int64_t K, int mode,
                                    const double* norms, const uint8_t* mask_in,
                                    uint8_t* mask_out, void* vals, void* meta, uint8_t* e_w,
                                    void* stream) {
  if (N < 0 || K < 0 || (mode != SP24_MAGNITUDE && mode != SP24_WANDA)) return SP24_ERR_ARG;
  if (N == 0 || K == 0) return SP24_OK;
  if (!W || !vals || !meta || !e_w || (mode == SP24_WANDA && !norms)) return SP24_ERR_ARG;
  if (K % 32 != 0) return SP24_ERR_ALIGN;
  if (!aligned16(W) || !aligned16(vals) || !aligned16(meta) || !aligned16(e_w) ||
      (mask_in && !aligned16(mask_in)) || (mask_out && !aligned16(mask_out)) ||
      (norms && !aligned16(norms)))
    return SP24_ERR_ALIGN;
  SP24_TRY(check_device());
  ConvertArgs a{};
  a.w = static_cast<const uint16_t*>(W);
  a.n = N;
  a.k = K;
  a.norms = norms;
  a.mask_in = mask_in;
  a.mask_out = mask_out;
  a.vals = static_cast<uint32_t*>(vals);
  a.meta = static_cast<uint8_t*>(meta);
  a.e_w = e_w;
  return launch_convert_fp8(true, mode == SP24_WANDA, a, as_stream(stream));
}

sp24_status sp24_compress_fp8(const void* W, const uint8_t* mask, int64_t N, int64_t K, void* vals,
                              void* meta, uint8_t* e_w, void* stream) {
  if (N < 0 || K < 0) return SP24_ERR_ARG;
  if (N == 0 || K == 0) return SP24_OK;
  if (!W || !mask || !vals || !meta || !e_w) return SP24_ERR_ARG;
  if (K % 32 != 0) return SP24_ERR_ALIGN;
  if (!aligned16(W) || !aligned16(mask) || !aligned16(vals) || !aligned16(meta) || !aligned16(e_w))
    return SP24_ERR_ALIGN;
  SP24_TRY(check_device());
  ConvertArgs a{};
  a.w = static_cast<const uint16_t*>(W);
  a.n = N;
  a.k = K;
  a.mask_in = mask;
  a.vals = static_cast<uint32_t*>(vals);
  a.meta = static_cast<uint8_t*>(meta);
  a.e_w = e_w;
  return launch_convert_fp8(false, false, a, as_stream(stream));
}

}  // extern "C"
