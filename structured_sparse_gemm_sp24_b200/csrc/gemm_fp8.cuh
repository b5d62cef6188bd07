// Block scales of the e4m3 product (sp24_gemm_fp8), shared by the split-K and
// the CTA-pair kernels.  Included by gemm_sp.cu.
//
// Y[m][n] = sum over K blocks b of 128 of 2^(ex[m][b] + ew[n / 128][b]) *
//           sum over the kept k of block b of x[m][k] * w[n][k],
// with ex, ew the exponents of the e8m0 scale bytes.  The tensor core applies
// both powers of two to every K = 64 instruction's products before the fp32
// sum (kind::mxf8f6f4), so the scales cost no pass over the accumulator: with
// scales applied in registers each 128-position block of a 128 x 256 tile
// would take 32768 fused multiply-adds, as long as its sparse MMAs.  Powers of
// two also make the scaling exact.
//
// Scale words.  Global memory holds one byte per row and block, rows padded to
// whole 32-bit words (four blocks, 512 K-positions: two ring stages).  Tensor
// memory wants row r's word in lane r % 32, column r / 32, so the loader warp
// reads 32 token rows per load (lane = row % 32), one word each, joins the
// words of rows 32 apart into the 16 bytes of a lane and writes them with one
// store; the MMA thread copies the tile with tcgen05.cp (the four lane
// quadrants get the same data).  A weight tile's 128 rows share one word: its
// tile is 8 rows of 16 bytes that the copy reads four times (row-group stride
// 0).
#pragma once

namespace sp24 {

// kBuf: scale buffers in tensor memory.
template <int kDtype, int BN, int kBuf>
struct SfCfg {
  static constexpr bool kOn = kDtype == SP24_FP8;
  static constexpr int kTiles = (BN + 127) / 128;              // 128-token scale tiles
  static constexpr int kABytes = 128;                          // 8 rows x 16 bytes
  static constexpr int kSmemBuf = kOn ? kABytes + 512 * kTiles : 0;
  static constexpr int kBufCols = 4 * kTiles + 4;              // tokens, then weight rows
  static constexpr int kCols = kOn ? kBuf * kBufCols : 0;
  static constexpr int kBufs = kBuf;
};

// Whether stage kb of a K range starting at kb0 begins a scale word.
__device__ __forceinline__ bool sf_load_stage(int kb, int kb0) { return kb == kb0 || (kb & 1) == 0; }

// A loader warp's words of one tile: words word0 .. word0 + G - 1 of the tokens
// tok0 + lane + 32 j and of the tile's weight row block.
template <int BN, int G>
struct SfWords {
  static constexpr int kRows = (BN + 31) / 32;
  uint32_t x[kRows][G];
  uint32_t w[G];

  // Words past the row (word0 + g >= words) and rows past the ends read as
  // scale 1 (their accumulator columns and lanes are not stored).  With G = 4
  // and rows of whole 16-byte pieces one load fetches the four words.
  __device__ __forceinline__ void load(const uint32_t* e_x, const uint32_t* e_w, int64_t words,
                                       int64_t word0, int64_t tok0, int64_t m, int64_t rt,
                                       int64_t row_tiles, int lane) {
    const bool vec = G == 4 && (words & 3) == 0;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int64_t t = tok0 + 32 * j + lane;
      const bool ok = t < m && 32 * j + lane < BN;
      fetch(x[j], e_x + t * words + word0, ok, vec, words - word0);
    }
    fetch(w, e_w + rt * words + word0, rt < row_tiles, vec, words - word0);
  }

  __device__ __forceinline__ static void fetch(uint32_t (&d)[G], const uint32_t* p, bool ok, bool vec,
                                               int64_t left) {
    if constexpr (G == 4) {
      if (vec) {
        const uint4 q = ok ? __ldg(reinterpret_cast<const uint4*>(p))
                           : make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        d[0] = q.x;
        d[1] = q.y;
        d[2] = q.z;
        d[3] = q.w;
        return;
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) d[g] = ok && g < left ? __ldg(p + g) : 0x7F7F7F7Fu;
  }

  // Writes the tiles of the words, one scale buffer after another (each the
  // weight tile, then the token tiles).
  __device__ __forceinline__ void store(uint8_t* buf, int buf_bytes, int lane) const {
#pragma unroll
    for (int g = 0; g < G; ++g, buf += buf_bytes) {
      if (lane < 8) *reinterpret_cast<uint4*>(buf + 16 * lane) = make_uint4(w[g], w[g], w[g], w[g]);
#pragma unroll
      for (int t = 0; t < (kRows + 3) / 4; ++t) {
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = 4 * t + i < kRows ? 4 * t + i : 0;
          v[i] = 4 * t + i < kRows ? x[j][g] : 0x7F7F7F7Fu;
        }
        *reinterpret_cast<uint4*>(buf + 128 + 512 * t + 16 * lane) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
    fence_async_shared();
    __syncwarp();
  }
};

// Copies one scale buffer to tensor memory: token tiles at `col`, the weight
// tile after them.
template <class Sf, bool kPair>
__device__ __forceinline__ void sf_copy(uint32_t tmem_col, uint32_t buf_addr) {
#pragma unroll
  for (int t = 0; t < Sf::kTiles; ++t) {
    const uint64_t d = smem_desc(buf_addr + 128 + 512 * t, 128, 128, kSwizzleNone);
    if constexpr (kPair) tc_cp_scales_pair(tmem_col + 4 * t, d);
    else tc_cp_scales(tmem_col + 4 * t, d);
  }
  const uint64_t d = smem_desc(buf_addr, 128, 0, kSwizzleNone);
  if constexpr (kPair) tc_cp_scales_pair(tmem_col + 4 * Sf::kTiles, d);
  else tc_cp_scales(tmem_col + 4 * Sf::kTiles, d);
}

}  // namespace sp24
