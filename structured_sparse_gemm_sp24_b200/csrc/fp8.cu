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

template <bool kPrune, bool kWanda>
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
  const bool kv_ok = v < kvec;

  uint4 q[kConvRows];
#pragma unroll
  for (int j = 0; j < kConvRows; ++j) {
    const int64_t row = row0 + 16 * j;
    q[j] = make_uint4(0u, 0u, 0u, 0u);
    if (kv_ok && row < a.n)
      q[j] = __ldcs(reinterpret_cast<const uint4*>(a.w + row * a.k) + v);
  }
  double nrm[8];
  if constexpr (kWanda) {
#pragma unroll
    for (int e = 0; e < 8; ++e) nrm[e] = kv_ok ? __ldg(a.norms + 8 * v + e) : 0.0;
  }

  uint32_t bad = 0, amax = 0;
  uint32_t p0[kConvRows], p1[kConvRows];   // kept pairs of the two groups
#pragma unroll
  for (int j = 0; j < kConvRows; ++j) {
    const int64_t row = row0 + 16 * j;
    uint32_t lo0 = 0, hi0 = 1, lo1 = 0, hi1 = 1, keep = 0;
    if (kv_ok && row < a.n) {
      uint32_t in = 0xFFu;
      if (a.mask_in) in = a.mask_in[row * kvec + v];
      if constexpr (kPrune && !kWanda) {
        top2_positions_mag<true>(q[j].x, q[j].y, in & 15u, lo0, hi0);
        top2_positions_mag<true>(q[j].z, q[j].w, in >> 4, lo1, hi1);
        keep = (1u << lo0) | (1u << hi0) | (((1u << lo1) | (1u << hi1)) << 4);
      } else {
        if constexpr (kPrune) keep = mask_byte<true>(q[j], in, nrm, 2);
        else keep = in;
        uint32_t badv = 0;
        const uint32_t c0 = nibble_code(keep & 15u, badv);
        const uint32_t c1 = nibble_code(keep >> 4, badv);
        if (!kPrune) bad |= badv;
        lo0 = c0 & 3u; hi0 = c0 >> 2; lo1 = c1 & 3u; hi1 = c1 >> 2;
      }
    }
    p0[j] = gather_pair(q[j].x, q[j].y, lo0, hi0);
    p1[j] = gather_pair(q[j].z, q[j].w, lo1, hi1);
    s_meta[(m0 + 16 * j) * 16 + bb] = static_cast<uint8_t>(lo0 | (hi0 << 2) | (lo1 << 4) | (hi1 << 6));
    s_mask[(m0 + 16 * j) * 16 + bb] = static_cast<uint8_t>(keep);
    // |value| bits of a bf16 are its float's upper half
    amax = max(amax, max((p0[j] << 16) & 0x7FFF0000u, p0[j] & 0x7FFF0000u));
    amax = max(amax, max((p1[j] << 16) & 0x7FFF0000u, p1[j] & 0x7FFF0000u));
  }
  amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kConvThreads / 32; ++i) amax = max(amax, s_max[i]);
  const uint32_t byte = scale_byte(amax);
  const float inv = scale_inverse(byte == kScaleNan ? kScaleOne : byte);
#pragma unroll
  for (int j = 0; j < kConvRows; ++j) {
    const int64_t row = row0 + 16 * j;
    if (kv_ok && row < a.n) {
      uint32_t c = e4m3x4(__uint_as_float(p0[j] << 16) * inv,
                          __uint_as_float(p0[j] & 0xFFFF0000u) * inv,
                          __uint_as_float(p1[j] << 16) * inv,
                          __uint_as_float(p1[j] & 0xFFFF0000u) * inv);
      if (byte == kScaleNan) c = kCodeNan4;
      __stcs(a.vals + row * kvec + v, c);
    }
  }
  if (tid < 128) {
    uint4* dst = reinterpret_cast<uint4*>(a.meta + static_cast<int64_t>(blockIdx.x) * 2048);
    __stcs(dst + tid, reinterpret_cast<const uint4*>(s_meta)[tid]);
  } else if (a.mask_out) {
    const int m = tid - 128;
    const int64_t row = static_cast<int64_t>(rt) * 128 + m;
    const int64_t v0 = static_cast<int64_t>(kb) * 16;
    const int nb = static_cast<int>(kvec - v0 < 16 ? kvec - v0 : 16);   // K % 32: multiple of 4
    if (row < a.n) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.mask_out + row * kvec + v0);
      for (int e = 0; e < nb / 4; ++e) dst[e] = reinterpret_cast<const uint32_t*>(s_mask)[m * 4 + e];
    }
  }
  // this block's scale, and the row's padding after the last block
  if (tid == 0) a.e_w[static_cast<int64_t>(rt) * a.scale_cols + kb] = static_cast<uint8_t>(byte);
  if (kb == a.kblocks - 1 && tid > 0 && kb + tid < a.scale_cols)
    a.e_w[static_cast<int64_t>(rt) * a.scale_cols + kb + tid] = static_cast<uint8_t>(kScaleOne);
  if (bad) raise_error(kErrPatternBit);
}

static sp24_status launch_convert_fp8(bool prune, bool wanda, ConvertArgs a, cudaStream_t s) {
  const int64_t kblocks = (a.k + 127) / 128;
  const int64_t nblocks = ((a.n + 127) / 128) * kblocks;
  if (nblocks > 0x7FFFFFFF) return SP24_ERR_UNSUPPORTED;
  a.kblocks = static_cast<int>(kblocks);
  a.scale_cols = static_cast<int>(4 * ((a.k + 511) / 512));
  const dim3 grid(static_cast<unsigned>(nblocks));
  if (!prune) return launch_kernel(convert_fp8_kernel<false, false>, grid, dim3(kConvThreads), 0, s, 1, a);
  if (wanda) return launch_kernel(convert_fp8_kernel<true, true>, grid, dim3(kConvThreads), 0, s, 1, a);
  return launch_kernel(convert_fp8_kernel<true, false>, grid, dim3(kConvThreads), 0, s, 1, a);
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
