// libsp24: sparse GEMM Y = X * W'^T on the 5th-generation tensor cores
// (tcgen05.mma.sp), for bf16 (fp32 accumulate), int8 (int32 accumulate) and
// block-scaled e4m3 (fp32 accumulate).
//
// [Orin ch.7] "Chapter 7: 2:4 Structured Sparsity" 2.1 Step 3: the sparse
// tensor core multiplies only the kept weights, each with the activation its
// 2-bit position selects; [Sparse-accel forum] (oeforum.com): INT8 x 2:4.
//
// Operand roles.  The sparse operand of tcgen05.mma.sp is A (the MMA's M
// side), so the kernel computes one 128 (output channels) x BN (tokens) tile
// of Y^T = W' * X^T per CTA:
//   A = compressed W tile: 128 rows x 128 bytes per stage (bf16: 64 values =
//       128 logical K; int8: 128 values = 256 logical K), TMA, 128B swizzle;
//   B = X tile: BN rows x 256 bytes per stage as two 128B-swizzled halves;
//   E = metadata chunk(s) (2048 bytes per 128 logical K), one bulk copy, then
//       tcgen05.cp into tensor memory, where tcgen05.mma.sp reads it;
//   D = fp32 / int32 accumulator in tensor memory: lane = output channel,
//       column = token.
// Each stage issues 4 MMAs (K = 32 for kind::f16, 64 for kind::i8 and
// kind::mxf8f6f4, which share the int8 tile and metadata layouts); all
// advance A by 32 bytes and B by 64 bytes inside the swizzle atoms.
//
// Kernels: gemm_splitk.cuh (split-K), gemm_persistent.cuh (single-SM
// persistent), gemm_pair.cuh (CTA-pair persistent), each with its launch;
// gemm_epilogue.cuh (epilogue of both persistent kernels).  This file holds
// the launch plan, the dispatch and the C entry points.

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "sp24_device.cuh"
#include "sp24_host.h"
#include "tma_host.h"

namespace sp24 {

struct GemmArgs {
  const uint8_t* meta;
  const float* s_x;
  const float* s_w;
  const float* s_y;
  const uint32_t* e_x;   // e4m3: scale words (gemm_fp8.cuh)
  const uint32_t* e_w;
  int64_t sf_words;
  void* y;
  int64_t m, n, k;
  int kblocks;        // stages over the whole K
  int kb_per_split;   // stages per split CTA
  int out_kind;
};

}  // namespace sp24

#include "gemm_fp8.cuh"
#include "gemm_splitk.cuh"
#include "gemm_epilogue.cuh"
#include "gemm_persistent.cuh"
#include "gemm_pair.cuh"

namespace sp24 {

// ----------------------------------------------------------------- host side
namespace {

// Which kernel to use: SP24_GEMM_IMPL = pair256 | pair240 | pair224 | pair192 |
// pair128 | single | splitk (tuning override; default chooses by problem size).
enum Impl : int { kSplitK = 0, kPair256 = 1, kPair128 = 2, kSingle = 3, kPair224 = 4,
                  kPair192 = 5, kPair240 = 6 };

int impl_override() {
  const char* e = std::getenv("SP24_GEMM_IMPL");
  if (!e) return -1;
  if (std::strcmp(e, "pair256") == 0) return kPair256;
  if (std::strcmp(e, "pair128") == 0) return kPair128;
  if (std::strcmp(e, "single") == 0) return kSingle;
  if (std::strcmp(e, "pair224") == 0) return kPair224;
  if (std::strcmp(e, "pair192") == 0) return kPair192;
  if (std::strcmp(e, "pair240") == 0) return kPair240;
  if (std::strcmp(e, "splitk") == 0) return kSplitK;
  return -1;
}

// SP24_SPLITK = 1..8: K slices of the split-K kernel (tuning override; 0 =
// choose by shape).
int split_override() {
  const char* e = std::getenv("SP24_SPLITK");
  if (!e) return 0;
  const int v = std::atoi(e);
  return (v >= 1 && v <= 8) ? v : 0;
}

const char* impl_name(int impl) {
  switch (impl) {
    case kPair256: return "pair256";
    case kPair240: return "pair240";
    case kPair224: return "pair224";
    case kPair192: return "pair192";
    case kPair128: return "pair128";
    case kSingle: return "single";
    default: return "splitk";
  }
}

int pair_tokens(int impl) {
  switch (impl) {
    case kPair256: return 256;
    case kPair240: return 240;
    case kPair224: return 224;
    case kPair192: return 192;
    default: return 128;
  }
}

// Estimated run time (us, B200 under load) of a persistent variant: waves of
// output tiles over the SMs (resident pairs) x per-tile time, i.e. k-blocks x
// the measured cost of one k-block plus the part of the epilogue the variant
// cannot overlap with the next tile.  Used only to rank the variants.  e4m3:
// 0.59, 0.535 and 0.515 us a k-block of 256-, 240- and 224-token tiles (8192 x
// 11008 x 4096: 194, 180 us; 8192 x 4096 x 4096: 73, 68, 66 us; the first has
// room for three ring stages only).  A k-block's time follows the bytes that it
// brings into an SM (16 KB of weights, 4 of metadata, 128 a token) and not the
// tensor pipe alone: 8192 x 11008 x 4096 on 240 tokens takes 809 clocks a k-block
// under the power cap, 727 with the token loads only, 661 with the weights' only
// and 580 on resident operands, where the pipe needs 480.
double est_time(int impl, int64_t m, int64_t n, int kblocks, int sms, int pairs, bool fp8) {
  const auto waves = [](int64_t tiles, int64_t units) {
    return static_cast<double>((tiles + units - 1) / units);
  };
  const double kb = kblocks;
  const int64_t prow = (n + 255) / 256;
  const double c256 = fp8 ? 0.59 : 0.50, c240 = fp8 ? 0.535 : 0.50, c224 = fp8 ? 0.515 : 0.50;
  switch (impl) {
    case kPair256:   // one accumulator: the next tile waits for the epilogue's
                     // tensor-memory loads (~0.8 us a tile, measured)
      return waves(prow * ((m + 255) / 256), pairs) * (c256 * kb + 0.8);
    case kPair240:   // two accumulators: only the last drain is exposed
      return waves(prow * ((m + 239) / 240), pairs) * std::max(c240 * kb, 1.5) + 2.0;
    case kPair224:
      return waves(prow * ((m + 223) / 224), pairs) * std::max(c224 * kb, 1.4) + 2.0;
    default:         // 128 x 128 single-SM tile, two accumulators
      return waves(((n + 127) / 128) * ((m + 127) / 128), sms) * std::max(0.48 * kb, 1.6);
  }
}

struct Plan {
  int impl;            // Impl
  int bn;              // split-K kernel: tokens per tile
  int split;           // split-K kernel: K slices (= cluster size)
  bool small_ring;     // split-K kernel: the ring that lets several CTAs share an SM
  int64_t ctas;        // CTAs launched
  int cluster;         // CTAs per cluster
  int tile_tokens;     // tokens (rows of X and Y) per output tile
  int tile_channels;   // output channels (rows of W) per output tile
};

// The launch plan.  At least 128 tokens and at least one 128 x 128 tile per
// SM: a persistent kernel, the variant with the lowest estimated time (or the
// SP24_GEMM_IMPL override).  Otherwise (few tokens or less than one wave of
// tiles): the split-K kernel, BN from the token count and K split as far as
// all CTAs still fit one wave (SP24_SPLITK overrides the split).  Measured on
// B200: M = 128 x 11008 x 4096 (86 tiles) takes 22.5 us split-K, 24.6 us on
// the persistent kernel (e4m3, with the lean issue loop: 11.2 us split-K, 12.5 us
// on 224-token pairs).
// Split-K rings: the full ring (one CTA per SM) and a small one with which
// several split CTAs share an SM (so that a split spreads a few row tiles
// over every SM without a second wave).  Shared memory per SM on sm_100 is
// 228 KiB, of which each resident CTA also takes 1 KiB.  No CTA's allocation of
// tensor memory may ever wait on another's: a CTA allocates before it waits for
// the previous kernel, and the CTAs of a cluster wait for one another.  So the
// CTAs that fit an SM by shared memory, of whatever types and token counts, need
// at most 512 columns together (the worst mix is two 128-token CTAs of 256), and
// any other kernel that uses tensor memory leaves no room beside it.
constexpr int kSmemPerSm = 228 * 1024;
constexpr int small_ring_stages(int bn) { return bn == 16 ? 3 : 2; }

struct CtaNeeds {
  int smem, columns;
};
template <class C>
constexpr CtaNeeds needs_of() {
  return {C::kSmemBytes + 1024, C::kTmemCols};
}
template <int kDtype, int BN>
constexpr CtaNeeds kSmallRing = needs_of<GemmCfg<kDtype, BN, small_ring_stages(BN)>>();
constexpr CtaNeeds kSmallRings[] = {
    kSmallRing<SP24_BF16, 16>, kSmallRing<SP24_BF16, 32>, kSmallRing<SP24_BF16, 64>,
    kSmallRing<SP24_BF16, 128>, kSmallRing<SP24_INT8, 16>, kSmallRing<SP24_INT8, 32>,
    kSmallRing<SP24_INT8, 64>, kSmallRing<SP24_INT8, 128>, kSmallRing<SP24_FP8, 16>,
    kSmallRing<SP24_FP8, 32>, kSmallRing<SP24_FP8, 64>, kSmallRing<SP24_FP8, 128>};

// Most columns that small-ring CTAs number `from` and up can need in `smem` bytes.
constexpr int most_columns(int smem, int from = 0) {
  int best = 0;
  for (int i = from; i < 12; ++i)
    if (kSmallRings[i].smem <= smem) {
      const int c = kSmallRings[i].columns + most_columns(smem - kSmallRings[i].smem, i);
      best = c > best ? c : best;
    }
  return best;
}
static_assert(most_columns(kSmemPerSm) <= 512, "an allocation of tensor memory could wait");

template <class C>
constexpr bool fills_sm() {
  return most_columns(kSmemPerSm - needs_of<C>().smem) == 0;
}
template <int kDtype>
constexpr bool full_rings_fill_sm() {
  return fills_sm<GemmCfg<kDtype, 16, 8>>() && fills_sm<GemmCfg<kDtype, 32, 7>>() &&
         fills_sm<GemmCfg<kDtype, 64, 6>>() && fills_sm<GemmCfg<kDtype, 128, 4>>();
}
static_assert(full_rings_fill_sm<SP24_BF16>() && full_rings_fill_sm<SP24_INT8>() &&
                  full_rings_fill_sm<SP24_FP8>() && fills_sm<GemmCfg<SP24_FP8, 96, 5>>(),
              "a split-K CTA with the full ring shares its SM");
// (the pair and single-SM variants with the least shared memory)
static_assert(fills_sm<PairCfg<SP24_BF16, 192, 4, SP24_OUT_BF16, 2>>() &&
                  fills_sm<PairCfg<SP24_INT8, 240, 3, SP24_OUT_INT32, 2>>() &&
                  fills_sm<PairCfg<SP24_FP8, 256, 3, SP24_OUT_BF16, 1>>() &&
                  fills_sm<PairCfg<SP24_FP8, 224, 3, SP24_OUT_F32, 2>>() &&
                  fills_sm<PersistCfg<SP24_BF16, 112, 4, SP24_OUT_BF16>>() &&
                  fills_sm<PersistCfg<SP24_INT8, 112, 3, SP24_OUT_INT32>>() &&
                  fills_sm<PersistCfg<SP24_INT8, 112, 4, SP24_OUT_INT8>>(),
              "a persistent CTA shares its SM");

template <int kDtype>
int small_ring_smem(int bn) {
  switch (bn) {
    case 16: return GemmCfg<kDtype, 16, small_ring_stages(16)>::kSmemBytes;
    case 32: return GemmCfg<kDtype, 32, small_ring_stages(32)>::kSmemBytes;
    case 64: return GemmCfg<kDtype, 64, small_ring_stages(64)>::kSmemBytes;
    default: return GemmCfg<kDtype, 128, small_ring_stages(128)>::kSmemBytes;
  }
}

int small_ring_ctas_per_sm(int dtype, int bn) {
  const int smem = dtype == SP24_BF16 ? small_ring_smem<SP24_BF16>(bn)
                   : dtype == SP24_FP8 ? small_ring_smem<SP24_FP8>(bn)
                                       : small_ring_smem<SP24_INT8>(bn);
  return kSmemPerSm / (smem + 1024);
}

sp24_status make_plan(int64_t m, int64_t n, int kblocks, int dtype, Plan* p) {
  const int sms = sm_count();
  const int64_t row_tiles = (n + 127) / 128;
  int forced = impl_override();
  // the e4m3 product has the split-K kernel and the 256, 240 and 224-token pairs
  const bool fp8 = dtype == SP24_FP8;
  if (fp8 && (forced == kSingle || forced == kPair192 || forced == kPair128)) forced = -1;
  // (an SP24_GEMM_IMPL override applies from half a wave of tiles, as the
  // kernel-family tests expect)
  const int64_t tiles128 = row_tiles * ((m + 127) / 128);
  // e4m3 has no single-SM kernel: what a pair tile cannot fill goes to split-K,
  // unless its tiles are more than a launch's y and z number (16 bits each).  For
  // 129 to 255 tokens that is not the best choice where the 128-token tiles pass
  // one wave (160 x 11008 x 4096: 16.8 us, 224-token pairs 12.8; 160 x 22016 x 4096
  // 29.7 and 20.3); at 128 tokens it is (11008: 11.5 and 12.5, 22016: 18.6 and 20.1).
  const bool fp8_split =
      fp8 && forced < 0 && (m < 256 || n < 256) && row_tiles <= 65535 && m <= 65535 * 128;
  const bool enough = m >= 128 || (fp8 && row_tiles > 65535);
  if (forced != kSplitK && enough && tiles128 >= (forced >= 0 ? sms / 2 : sms) && !fp8_split) {
    int pairs = 0;
    SP24_TRY(pair_capacity(&pairs));
    int impl = forced;
    if (impl < 0) {
      impl = kSingle;   // pair tiles need both dimensions to fill them
      if (fp8 || (m >= 256 && n >= 256)) {
        double best = fp8 ? 1e30 : est_time(kSingle, m, n, kblocks, sms, pairs, false);
        for (int c : {kPair256, kPair240, kPair224}) {
          const double t = est_time(c, m, n, kblocks, sms, pairs, fp8);
          if (t < best) {
            best = t;
            impl = c;
          }
        }
      }
    }
    p->impl = impl;
    p->bn = 128;
    p->split = 1;
    p->small_ring = false;
    if (impl == kSingle) {
      const int64_t tiles = row_tiles * ((m + 127) / 128);
      p->ctas = tiles < sms ? tiles : sms;
      p->cluster = 1;
      p->tile_tokens = 128;
      p->tile_channels = 128;
    } else {
      const int tok = pair_tokens(impl);
      const int64_t tiles = ((n + 255) / 256) * ((m + tok - 1) / tok);
      p->ctas = 2 * (tiles < pairs ? tiles : pairs);
      p->cluster = 2;
      p->tile_tokens = tok;
      p->tile_channels = 256;
    }
    return SP24_OK;
  }
  int bn = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
  int64_t base = row_tiles * ((m + bn - 1) / bn);
  // The split.  With the issue loop that built every descriptor anew a stage took
  // the issuing thread about the same time whatever the token count (measured on
  // B200: ~0.44 us per 128-channel x 128-K stage at 16 tokens, ~0.5 us at 256), so
  // at few tokens the kernel was bound by the stages the busiest SM runs:
  // ceil(CTAs / SMs) x stages per CTA.  The plan
  // takes the split among 1, 2, 4, 8 (at least 4 stages per CTA) that
  // minimises it, the fewer CTAs on a tie; more than one CTA per SM takes
  // the small ring.  E.g. M = 16, 11008 x 4096 (86 row tiles, 32 stages):
  // split 1 on 86 SMs runs 32 stages on the busiest SM, split 4 (344 CTAs,
  // 3 per SM) 24 -- 9.8 against 13.9 us a launch back to back.  Splits of 3,
  // 5, 6 and 7 run correctly (SP24_SPLITK) but measured no better: at 3 CTAs
  // per SM a GPC holds fewer 5-CTA clusters than the 86 tiles need
  // (cudaOccupancyMaxActiveClusters: 82), and the second wave costs more
  // than the shorter K loop saves.  With the lean loop the model no longer holds
  // where a split shares SMs: 11008 x 4096, weights from HBM, split 1 and 4, bf16
  // M = 1 11.2 and 10.8 us, 16 11.2 and 11.3, 64 12.5 and 14.3, int8 8.1 and 8.6, 8.3
  // and 8.9, 10.5 and 11.7.  It still picks the best split where CTAs do not share
  // (4096 x 4096, split 4: bf16 M = 16 6.7 us, 1 9.5, 8 7.1; int8 5.1, 6.6, 5.5), and
  // another split would change the bf16 sums' order.
  int split = 1;
  int64_t best = -1;
  const int cap = small_ring_ctas_per_sm(dtype, bn);
  // e4m3 (with the lean issue loop): the largest split that keeps one CTA per
  // SM; sharing an SM costs more than it spreads (11008 x 4096: M = 1 8.25 us
  // with split 1 on 86 CTAs, 8.17 with 4; M = 16 8.3 and 8.7; M = 64 9.3 and 11.6;
  // 4096 x 4096, M = 1: split 1 6.6, 4 4.8, 8 5.0).  Above 64 tokens a stage takes
  // the time of its rows' way into the SM (128 of weights, two halves of bn), so
  // 96-token tiles are taken where they make the busiest SM load fewer: M = 333
  // x 4104 x 4128 10.3 us on 132 CTAs, 11.9 with 128 tokens on 99; M = 80 x 4096 x
  // 4096 6.9 and 7.6; M = 192 x 8192 x 4096 8.2 and 8.8; M = 288 x 5376 x 11008
  // 15.6 and 16.7.
  const auto one_per_sm = [&](int64_t tiles) {
    int sp = 1;
    while (sp < 8 && kblocks >= 8 * sp && tiles * 2 * sp <= sms) sp *= 2;
    return sp;
  };
  if (fp8) {
    split = one_per_sm(base);
    if (bn == 128) {
      const int64_t base96 = row_tiles * ((m + 95) / 96);
      const int split96 = one_per_sm(base96);
      const auto rows = [&](int tokens, int sp) {
        return static_cast<int64_t>((kblocks + sp - 1) / sp) * (128 + 2 * tokens);
      };
      if (base96 <= sms && rows(96, split96) < rows(128, split)) {
        bn = 96;
        base = base96;
        split = split96;
      }
    }
  }
  for (int sp = 1; !fp8 && sp <= 8; sp *= 2) {
    if (sp > 1 && kblocks < 4 * sp) break;
    const int64_t per_sm = (base * sp + sms - 1) / sms;
    if (sp > 1 && per_sm > cap) break;
    const int64_t cost = per_sm * ((kblocks + sp - 1) / sp);
    if (best < 0 || cost < best) {
      best = cost;
      split = sp;
    }
  }
  const int so = split_override();
  if (so > 0 && so <= kblocks) {
    split = fp8 ? (so >= 8 ? 8 : so >= 4 ? 4 : so >= 2 ? 2 : 1) : so;
    // (e4m3 CTAs share an SM only where the tiles alone are more than the SMs)
    while (fp8 && split > 1 && base * split > sms) split /= 2;
  }
  p->impl = kSplitK;
  p->bn = bn;
  p->split = split;
  p->small_ring = base * split > sms && bn != 96;
  p->ctas = base * split;
  p->cluster = split;
  p->tile_tokens = bn;
  p->tile_channels = 128;
  return SP24_OK;
}

template <int kDtype, int BN, int ST>
sp24_status launch_split(int split, const CUtensorMap& ma, const CUtensorMap& mb,
                         const GemmArgs& a, cudaStream_t s) {
  if constexpr (kDtype == SP24_FP8) {   // powers of two only (the plan takes no other)
    switch (split) {
      case 1: return launch_gemm_cfg<kDtype, BN, ST, 1>(ma, mb, a, s);
      case 2: return launch_gemm_cfg<kDtype, BN, ST, 2>(ma, mb, a, s);
      case 4: return launch_gemm_cfg<kDtype, BN, ST, 4>(ma, mb, a, s);
      default: return launch_gemm_cfg<kDtype, BN, ST, 8>(ma, mb, a, s);
    }
  } else {
    switch (split) {
      case 1: return launch_gemm_cfg<kDtype, BN, ST, 1>(ma, mb, a, s);
      case 2: return launch_gemm_cfg<kDtype, BN, ST, 2>(ma, mb, a, s);
      case 3: return launch_gemm_cfg<kDtype, BN, ST, 3>(ma, mb, a, s);
      case 4: return launch_gemm_cfg<kDtype, BN, ST, 4>(ma, mb, a, s);
      case 5: return launch_gemm_cfg<kDtype, BN, ST, 5>(ma, mb, a, s);
      case 6: return launch_gemm_cfg<kDtype, BN, ST, 6>(ma, mb, a, s);
      case 7: return launch_gemm_cfg<kDtype, BN, ST, 7>(ma, mb, a, s);
      default: return launch_gemm_cfg<kDtype, BN, ST, 8>(ma, mb, a, s);
    }
  }
}

// The small ring (e4m3 takes it without a split only).
template <int kDtype, int BN>
sp24_status launch_small(int split, const CUtensorMap& ma, const CUtensorMap& mb,
                         const GemmArgs& a, cudaStream_t s) {
  constexpr int kStages = small_ring_stages(BN);
  if constexpr (kDtype == SP24_FP8) {
    return split == 1 ? launch_gemm_cfg<kDtype, BN, kStages, 1>(ma, mb, a, s) : SP24_ERR_UNSUPPORTED;
  } else {
    return launch_split<kDtype, BN, kStages>(split, ma, mb, a, s);
  }
}

template <int kDtype>
sp24_status dispatch(const void* x, const void* vals, GemmArgs a, cudaStream_t s) {
  Plan p;
  SP24_TRY(make_plan(a.m, a.n, a.kblocks, kDtype, &p));
  a.kb_per_split = (a.kblocks + p.split - 1) / p.split;
  const int bn = p.bn;
  const int el = kDtype == SP24_BF16 ? 2 : 1;
  const CUtensorMapDataType dt =
      kDtype == SP24_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const uint32_t box_cols = 128 / el;
  CUtensorMap ma, mb;
  SP24_TRY(make_map(&ma, vals, dt, el, static_cast<uint64_t>(a.k / 2),
                    static_cast<uint64_t>(a.n), box_cols, 128));
  const int pairs = static_cast<int>(p.ctas / 2);
  if constexpr (kDtype == SP24_FP8) {
    // one stage fewer at 256 tokens (and with 32-bit output): the scale buffers
    switch (p.impl) {
      case kPair256: return launch_pair_out<kDtype, 256, 3, 3, 1>(ma, a, x, pairs, s);
      case kPair240: return launch_pair_out<kDtype, 240, 4, 3, 2>(ma, a, x, pairs, s);
      case kPair224: return launch_pair_out<kDtype, 224, 4, 3, 2>(ma, a, x, pairs, s);
      default: break;
    }
  } else {
    switch (p.impl) {
      case kPair256: return launch_pair_out<kDtype, 256, 4, 3, 1>(ma, a, x, pairs, s);
      case kPair240: return launch_pair_out<kDtype, 240, 4, 3, 2>(ma, a, x, pairs, s);
      case kPair224: return launch_pair_out<kDtype, 224, 4, 4, 2>(ma, a, x, pairs, s);
      case kPair192: return launch_pair_out<kDtype, 192, 4, 4, 2>(ma, a, x, pairs, s);
      case kPair128:
        if constexpr (kDtype == SP24_BF16) {
          return launch_pair<kDtype, 128, 6, SP24_OUT_BF16, 2>(ma, a, x, pairs, s);
        } else {
          if (a.out_kind == SP24_OUT_INT32)
            return launch_pair<kDtype, 128, 5, SP24_OUT_INT32, 2>(ma, a, x, pairs, s);
          if (a.out_kind == SP24_OUT_INT8)
            return launch_pair<kDtype, 128, 6, SP24_OUT_INT8, 2>(ma, a, x, pairs, s);
          return launch_pair<kDtype, 128, 5, SP24_OUT_BF16, 2>(ma, a, x, pairs, s);
        }
      default: break;
    }
  }
  SP24_TRY(make_map(&mb, x, dt, el, static_cast<uint64_t>(a.k), static_cast<uint64_t>(a.m),
                    box_cols, static_cast<uint32_t>(bn)));
  if constexpr (kDtype != SP24_FP8) {
    if (p.impl == kSingle) {
      if constexpr (kDtype == SP24_BF16) {
        return launch_persistent<kDtype, 128, 4, SP24_OUT_BF16>(ma, mb, a, s);
      } else {
        if (a.out_kind == SP24_OUT_INT32)
          return launch_persistent<kDtype, 128, 3, SP24_OUT_INT32>(ma, mb, a, s);
        if (a.out_kind == SP24_OUT_INT8)
          return launch_persistent<kDtype, 128, 4, SP24_OUT_INT8>(ma, mb, a, s);
        return launch_persistent<kDtype, 128, 4, SP24_OUT_BF16>(ma, mb, a, s);
      }
    }
  }
  const int split = p.split;

#define SP24_GEMM_CASE(BN_, ST_)                                                          \
  if (bn == BN_) {                                                                        \
    if (p.small_ring) return launch_small<kDtype, BN_>(split, ma, mb, a, s);               \
    return launch_split<kDtype, BN_, ST_>(split, ma, mb, a, s);                             \
  }
  SP24_GEMM_CASE(16, 8)
  SP24_GEMM_CASE(32, (kDtype == SP24_FP8 ? 7 : 8))   // the scale buffers take one stage
  SP24_GEMM_CASE(64, 6)
  SP24_GEMM_CASE(128, 4)
  if constexpr (kDtype == SP24_FP8) {
    if (bn == 96) return launch_split<kDtype, 96, 5>(split, ma, mb, a, s);
  }
#undef SP24_GEMM_CASE
  return SP24_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace sp24

using namespace sp24;

extern "C" sp24_status sp24_gemm(const void* X, int64_t M, int64_t K, const void* vals,
                                 const void* meta, int64_t N, int dtype, const float* s_x,
                                 const float* s_w, int out_kind, const float* s_y, void* Y,
                                 void* stream) {
  if (M < 0 || N < 0 || K < 0 || (dtype != SP24_BF16 && dtype != SP24_INT8)) return SP24_ERR_ARG;
  if (dtype == SP24_BF16 && out_kind != SP24_OUT_BF16) return SP24_ERR_ARG;
  if (dtype == SP24_INT8 && out_kind != SP24_OUT_BF16 && out_kind != SP24_OUT_INT32 &&
      out_kind != SP24_OUT_INT8)
    return SP24_ERR_ARG;
  if (M == 0 || N == 0) return SP24_OK;
  if (!X || !vals || !meta || !Y) return SP24_ERR_ARG;
  if (dtype == SP24_INT8 && out_kind != SP24_OUT_INT32 && (!s_x || !s_w)) return SP24_ERR_ARG;
  if (dtype == SP24_INT8 && out_kind == SP24_OUT_INT8 && !s_y) return SP24_ERR_ARG;
  if (K < 16 || N % 8 != 0 || K % (dtype == SP24_BF16 ? 16 : 32) != 0) return SP24_ERR_ALIGN;
  if (out_kind == SP24_OUT_INT8 && dtype == SP24_INT8 && N % 16 != 0) return SP24_ERR_ALIGN;
  if (!aligned16(X) || !aligned16(vals) || !aligned16(meta) || !aligned16(Y) ||
      (s_w && !aligned16(s_w)))
    return SP24_ERR_ALIGN;
  if (K > (int64_t(1) << 31) || M > (int64_t(1) << 31) || N > (int64_t(1) << 31))
    return SP24_ERR_UNSUPPORTED;
  SP24_TRY(check_device());
  if (!get_encoder()) return cuda_fail("cudaGetDriverEntryPoint", "cuTensorMapEncodeTiled");
  GemmArgs a;
  a.meta = static_cast<const uint8_t*>(meta);
  a.s_x = s_x;
  a.s_w = s_w;
  a.s_y = s_y;
  a.e_x = a.e_w = nullptr;
  a.sf_words = 0;
  a.y = Y;
  a.m = M;
  a.n = N;
  a.k = K;
  a.out_kind = out_kind;
  const int kl = dtype == SP24_BF16 ? 128 : 256;
  a.kblocks = static_cast<int>((K + kl - 1) / kl);
  a.kb_per_split = a.kblocks;
  if (dtype == SP24_BF16) return dispatch<SP24_BF16>(X, vals, a, as_stream(stream));
  return dispatch<SP24_INT8>(X, vals, a, as_stream(stream));
}

extern "C" sp24_status sp24_gemm_fp8(const void* X, const uint8_t* e_x, int64_t M, int64_t K,
                                     const void* vals, const void* meta, const uint8_t* e_w,
                                     int64_t N, int out_kind, void* Y, void* stream) {
  if (M < 0 || N < 0 || K < 0 || (out_kind != SP24_OUT_BF16 && out_kind != SP24_OUT_F32))
    return SP24_ERR_ARG;
  if (M == 0 || N == 0) return SP24_OK;
  if (!X || !e_x || !vals || !meta || !e_w || !Y) return SP24_ERR_ARG;
  if (K < 32 || K % 32 != 0 || N % 8 != 0) return SP24_ERR_ALIGN;
  if (!aligned16(X) || !aligned16(e_x) || !aligned16(vals) || !aligned16(meta) ||
      !aligned16(e_w) || !aligned16(Y))
    return SP24_ERR_ALIGN;
  constexpr int64_t kMax = 0x7FFFFFFF - 512;   // tile coordinates are 32-bit
  if (K > kMax || M > kMax || N > kMax)
    return SP24_ERR_UNSUPPORTED;
  SP24_TRY(check_device());
  if (!get_encoder()) return cuda_fail("cudaGetDriverEntryPoint", "cuTensorMapEncodeTiled");
  GemmArgs a;
  a.meta = static_cast<const uint8_t*>(meta);
  a.s_x = a.s_w = a.s_y = nullptr;
  a.e_x = reinterpret_cast<const uint32_t*>(e_x);
  a.e_w = reinterpret_cast<const uint32_t*>(e_w);
  a.sf_words = (K + 511) / 512;
  a.y = Y;
  a.m = M;
  a.n = N;
  a.k = K;
  a.out_kind = out_kind;
  a.kblocks = static_cast<int>((K + 255) / 256);
  a.kb_per_split = a.kblocks;
  return dispatch<SP24_FP8>(X, vals, a, as_stream(stream));
}

extern "C" sp24_status sp24_gemm_plan(int64_t M, int64_t N, int64_t K, int dtype,
                                      sp24_gemm_plan_t* plan) {
  if (!plan || M < 1 || N < 1 || K < 16 ||
      (dtype != SP24_BF16 && dtype != SP24_INT8 && dtype != SP24_FP8))
    return SP24_ERR_ARG;
  if (K > (int64_t(1) << 31) || M > (int64_t(1) << 31) || N > (int64_t(1) << 31))
    return SP24_ERR_UNSUPPORTED;
  SP24_TRY(check_device());
  const int kl = dtype == SP24_BF16 ? 128 : 256;
  Plan p;
  SP24_TRY(make_plan(M, N, static_cast<int>((K + kl - 1) / kl), dtype, &p));
  std::memset(plan, 0, sizeof(*plan));
  std::snprintf(plan->kernel, sizeof(plan->kernel), "%s", impl_name(p.impl));
  plan->tile_tokens = p.tile_tokens;
  plan->tile_channels = p.tile_channels;
  plan->split_k = p.split;
  plan->ctas = p.ctas;
  plan->cluster = p.cluster;
  return SP24_OK;
}
