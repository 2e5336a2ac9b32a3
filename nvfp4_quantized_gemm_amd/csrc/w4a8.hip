// MXFP8 quantize, and the product of MXFP8 activations with MXFP4 weights (W4A8), for gfx950.
//
// Y[m][n] = sum_k a[m][k] Xa[m][k / 32] b[n][k] Xb[n][k / 32]: E4M3 codes times E2M1 codes under
// E8M0 scales, exact products (of operands from 2^-133 on), fp32 sums.
#include <cmath>
#include <type_traits>

#include "epilogue.hpp"
#include "launch.hpp"
#include "mx8.hpp"

namespace nvfp4 {

// A lane takes 8 consecutive elements, 4 adjacent lanes a block, and has two such segments in flight.
// Bound by memory, 3.03 B per bf16 element: 16384 x 8192 in 61 us (6.6 TB/s; one segment 70, four 63), 4096 x
// 4608 in 11.6 us (12.6, 11.5), 4096 x 1152 in 4.3 us (4.4, 4.7).
template <int DT, bool DENSE>
__global__ __launch_bounds__(256) void k_mx8_quantize(const void *__restrict__ x, int64_t ld, uint64_t nseg,
                                                      FastDiv bpr, uint8_t *__restrict__ codes,
                                                      uint8_t *__restrict__ scales) {
  constexpr int U = 2;
  const uint64_t g0 = (uint64_t)blockIdx.x * (256 * U) + threadIdx.x;
  Vec8<DT> v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t g = g0 + 256 * u;
    if (g >= nseg) break;
    int64_t off = (int64_t)g * 8;
    if (!DENSE) {
      const uint32_t blk = (uint32_t)(g >> 2), row = fastdiv(blk, bpr);
      off = (int64_t)row * ld + (int64_t)(blk - row * bpr.d) * kMx8Blk + 8 * (int64_t)(g & 3);
    }
    v[u].template load<true>(x, off);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t g = g0 + 256 * u;
    if (g >= nseg) break;  // whole blocks are in or out
    float f[8];
    v[u].get(f);
    const uint32_t b = mx8_scale_byte(mx8_amax_bits(f));
    *reinterpret_cast<u32x2 *>(codes + 8 * g) = mx8_encode8(f, b);
    if ((g & 3) == 0) scales[g >> 2] = (uint8_t)b;
  }
}

// One thread per output element.
template <int OUT>
__global__ __launch_bounds__(256) void k_w4a8_generic(const uint8_t *__restrict__ a, const uint8_t *__restrict__ as,
                                                      const uint8_t *__restrict__ b, const uint8_t *__restrict__ bs,
                                                      int64_t M, int64_t N, int64_t K, void *__restrict__ c,
                                                      int64_t ldc) {
  for (int64_t t = blockIdx.x * 256ll + threadIdx.x; t < M * N; t += (int64_t)gridDim.x * 256) {
    const int64_t m = t / N, n = t % N;
    float acc = 0.0f;
    for (int64_t k = 0; k < K; k += kMx8Blk) {
      const int ea = as[(m * K + k) / kMx8Blk], eb = bs[(n * K + k) / kMx8Blk];
      float part = 0.0f;
      for (int i = 0; i < kMx8Blk; i += 2) {
        const uint32_t w = b[(n * K + k + i) / 2];
        const f32x2 q = fp4_decode2_f32<0>(w);
        part = fmaf(e4m3_to_f32(a[m * K + k + i]), q.x, part);
        part = fmaf(e4m3_to_f32(a[m * K + k + i + 1]), q.y, part);
      }
      // both scales in one exponent: their product alone may leave fp32 where the scaled sum does not
      acc += ea == 255 || eb == 255 ? NAN : ldexpf(part, ea + eb - 254);
    }
    if (OUT == 0) static_cast<float *>(c)[m * ldc + n] = acc;
    else static_cast<__bf16 *>(c)[m * ldc + n] = (__bf16)acc;
  }
}

// ---- tiled product ------------------------------------------------------------------------------------
//
// The matrix instruction that takes E4M3 and E2M1 codes with E8M0 scales as they are sums groups of eight
// products in a window of 13 bits below the group's largest: measured, a product under 2^-13 of it is
// dropped, and a product over wide-ranging values came out 3e-5 of sum |a b| off.  That is no fp32 sum, so
// the codes are widened to bf16 with their scale (exact down to 2^-133: at most 4 significant bits; one conversion
// instruction per two values) and multiplied by v_mfma_f32_32x32x16_bf16, at half the rate.
//
// Operands of a 64-k step: lane (r, h) = (l % 32, l / 32) takes block h of row r: 32 activation bytes, 16
// weight bytes, one scale each; its 32 values make four matrix instructions of 8 k from either block.  In
// 16-byte pieces of a 128-k chunk (8 per activation row, 4 per weight row) step t takes activation
// pieces 4 t + 2 h and the next, and weight piece 2 t + h: both operands stream from their canonical
// layouts by LDS-DMA.
//
// R x C tile (rows of Y, columns) per workgroup of KG groups of WM x WN waves.  Each group takes its own
// run of chunks of 128 k through its own ring of S LDS stages, and the groups' sums are added in LDS in
// order: small tiles have few waves and much latency, and the groups overlap it without more traffic.
//   activation [R rows][8 pieces]   weight [C rows][4 pieces]
// A DMA copies 8 activation rows' 128 bytes or 16 weight rows' 64, neighbouring lanes neighbouring pieces
// (with rows in neighbouring lanes each lane is a request of its own, and the address unit was what bound
// every tile size: 64 x 8192 x 8192 took 28 us, and 16 with this).  Piece p of row r lies in slot
// p ^ (r / 2 % 8), or p ^ (r / 4 % 4) of a weight row, so that the 16 rows of a read pass lie in 16
// different bank groups.  Scales: blocks of 4 chunks (16 bytes of a row) in two slots, one row per lane: a
// 16-byte DMA lane, four 4-byte ones ([64 rows' chunk 0][chunk 1]..), or, where rows of scales are not
// aligned, registers that are written to LDS two chunks later.
//
// A chunk is two 64-k steps.  While step 0 multiplies, step 1's operands are read; in the middle one
// barrier says that the next chunk has landed everywhere and that this one's stage is free, the DMA of
// the chunk after the next two starts into it, and while step 1 multiplies the next chunk's step 0 is read.
// Rows past M or N repeat the last one and are never stored.  Past K (the end of the last chunk where K is
// no multiple of 128, and the chunks that a short group has too many) pieces are read from inside the row
// and the weight's words masked to zero: products with finite codes are then 0.
//
// Measured: 8192^3 in 0.74 to 0.77 ms, 1.43 to 1.49 PFLOP/s (a bf16 torch.matmul of that size: 1.30), bound by
// power: 76 % of the cycles in the matrix cores at 1.88 GHz.  With few tiles a 128 x 128 workgroup alone on
// its CU keeps them 62 % busy: a chunk is about 260 instructions a wave, 4 clocks each, beside 1024 clocks of
// products, and two workgroups on a CU (or two groups of one) get little more out of it.

namespace {

typedef uint32_t u32_any __attribute__((aligned(1)));

// Byte i of a word of scale bytes as the float the conversions take: they read its exponent field alone
// (checked over random other bits), so turning the byte there is all.  turn = scale_turn(i).
__device__ __forceinline__ uint32_t scale_turn(int i) { return (8 * i + 9) & 31; }
__device__ __forceinline__ float scale_at(uint32_t word, uint32_t turn) {
  return __uint_as_float(__builtin_amdgcn_alignbit(word, word, turn));
}
// 8 E4M3 codes of words lo, hi, or the 8 E2M1 codes of a word, times their scale: exact in bf16, but for E4M3
// under scale bytes 0 to 2, whose steps of 2^-136 to 2^-134 are below bf16's least number, 2^-133.
__device__ __forceinline__ bf16x8 widen_act(uint32_t lo, uint32_t hi, float X) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, X, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, X, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, X, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, X, true);
  return bf16x8{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}
__device__ __forceinline__ bf16x8 widen_weight(uint32_t w, float X) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, X, 0);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, X, 1);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, X, 2);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, X, 3);
  return bf16x8{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

// Bytes 4 w .. 4 w + 3 of a row of nb scale bytes; past the end 2^0.
__device__ __forceinline__ uint32_t scale_word(const uint8_t *row, int w, int nb) {
  if (4 * w + 4 <= nb) return *reinterpret_cast<const u32_any *>(row + 4 * w);
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) v |= (uint32_t)(4 * w + i < nb ? row[4 * w + i] : 127) << (8 * i);
  return v;
}

// The same without a branch, for rows of at least 4 bytes, in two parts: the load, and (when it is back)
// the shift.  Past the end 0, a finite scale.
__device__ __forceinline__ uint32_t scale_word_raw(const uint8_t *row, int w, int nb) {
  return *reinterpret_cast<const u32_any *>(row + min(4 * w, nb - 4));
}
__device__ __forceinline__ uint32_t scale_word_shift(uint32_t raw, int w, int nb) {
  return raw >> (8 * (4 * w - min(4 * w, nb - 4)));
}

// store_tile for rows of Y that are not 16-byte aligned: the slab goes through the same staging, and
// neighbouring lanes store neighbouring columns, one element each (777 x 1001, fp32: 1.6 us less than
// four single stores from each lane's 16 bytes).
template <int CW, int TM, int TN, typename OutT>
__device__ __forceinline__ void store_tile_unaligned(const f32x16 (&acc)[TM][TN], OutT *__restrict__ C, int64_t ldc,
                                                     int M, int N, int row0, int col0, uint8_t *lds, int lane) {
  constexpr int kPitch = EpiPitch<CW, 4>::kPitch;
  const int lr = lane & 31, lh = lane >> 5;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4 *>(lds + lr * kPitch + (j * 32 + 8 * g + 4 * lh) * 4) =
            f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
    wave_lds_sync();
    constexpr int kCols = CW < 64 ? CW : 64, kRows = 64 / kCols;
    const int c = lane % kCols, r0 = lane / kCols;
#pragma unroll
    for (int h = 0; h < CW / kCols; ++h) {
      const int col = col0 + h * kCols + c;
#pragma unroll 8
      for (int r = r0; r < 32; r += kRows) {
        const int row = row0 + 32 * i + r;
        const float v = *reinterpret_cast<const float *>(lds + r * kPitch + (h * kCols + c) * 4);
        if (row < M && col < N) C[(int64_t)row * ldc + col] = (OutT)v;
      }
    }
    wave_lds_sync();
  }
}

template <int R, int C, int WM_, int WN_, int KG_, int S_>
struct TileCfg {
  static constexpr int kR = R, kC = C, WM = WM_, WN = WN_, KG = KG_, S = S_;
  static constexpr int kSlots = S > 3 ? 3 : 2;  // scale blocks: the one in use and those on their way
  static constexpr int kG = WM * WN, kWaves = kG * KG, kThreads = 64 * kWaves;
  static constexpr int kTM = R / 32 / WM, kTN = C / 32 / WN;
  static constexpr int kA = R * 128, kB = C * 64, kStage = kA + kB;
  static constexpr int kScaleUnits = (R + C + 63) / 64, kSlot = kScaleUnits * 1024;  // of 64 rows
  static constexpr int kSU = (kScaleUnits + kG - 1) / kG;                            // per wave, at most
  static constexpr int kScales = S * kStage, kGroup = kScales + kSlots * kSlot, kLds = KG * kGroup;
  static constexpr int kNA = R / 8 / kG, kNB = C / 16 / kG, kDmas = kNA + kNB;  // DMAs per wave and chunk
  static constexpr int kPart = kTM * kTN * 4096;                               // a wave's sums
  static constexpr int kEpi = (KG - 1) * kG * kPart, kEpiWave = 32 * EpiPitch<C / WN, 4>::kPitch;
  static constexpr int kWavesPerEu = ((kLds <= 80 * 1024 ? 2 : 1) * kWaves + 3) / 4;
  static_assert(kNA * kG == R / 8 && kNB * kG == C / 16, "even DMA split");
  static_assert(kTM * WM * 32 == R && kTN * WN * 32 == C, "wave tiling");
  static_assert(S >= 3 && S <= 8 && kLds <= 160 * 1024 && kEpi + kG * kEpiWave <= kLds, "LDS fits");
};

}  // namespace

// SX: how a row's scale bytes of 4 chunks are loaded -- 16: one 16-byte DMA lane (K % 512 == 0, 16-byte
// aligned arrays, runs of whole blocks), 4: four 4-byte ones (K % 128 == 0), 1: unaligned words, bytes at
// the end (TAIL).  run: chunks per group.
template <int OUT, class Cfg, int SX>
__global__ __launch_bounds__(Cfg::kThreads) __attribute__((amdgpu_waves_per_eu(Cfg::kWavesPerEu, Cfg::kWavesPerEu))) void k_w4a8(
    const uint8_t *__restrict__ a, const uint8_t *__restrict__ as, const uint8_t *__restrict__ b,
    const uint8_t *__restrict__ bs, int M, int N, int K, void *__restrict__ c, int64_t ldc, int tiles_m, int tiles_n,
    int run) {
  constexpr int TM = Cfg::kTM, TN = Cfg::kTN, S = Cfg::S, G = Cfg::kG, KG = Cfg::KG, WN = Cfg::WN;
  constexpr bool TAIL = SX == 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KG == 1 ? 0 : wave_all / G, wave = KG == 1 ? wave_all : wave_all % G;
  const int wm = wave / WN, wn = wave % WN;
  const int lr = lane & 31, lh = lane >> 5;

  // tiles in XCD-aware grouped order: workgroups go round the 8 XCDs, so each XCD gets a run of tiles
  const int ntiles = tiles_m * tiles_n;
  int bid = blockIdx.x;
  {
    const int full = (ntiles / 8) * 8;
    if (bid < full) bid = (bid % 8) * (full / 8) + bid / 8;
  }
  int tmi, tni;
  grouped_tile<4>(bid, tiles_m, tiles_n, tmi, tni);
  const int m0 = tmi * Cfg::kR, n0 = tni * Cfg::kC;
  const int nk = (K + 127) / 128, nb = K / 32;
  const int k0 = kg * run;  // this group's chunks: k0 .. k0 + run - 1, those past nk with zero weights
  uint8_t *const ring = smem + kg * Cfg::kGroup;

  const uint8_t *a_tile = a + (int64_t)m0 * K, *b_tile = b + (int64_t)n0 * (K / 2);
  // DMA d of the activation: rows 8 d + lane / 8; of the weight: rows 16 d + lane / 4.  The pieces are
  // swizzled.
  uint32_t oa[Cfg::kNA], ob[Cfg::kNB], pa[Cfg::kNA];
  const uint32_t pb = (lane & 3) ^ ((lane >> 4) & 3);
#pragma unroll
  for (int i = 0; i < Cfg::kNA; ++i) {
    const int d = wave + G * i, row = 8 * d + (lane >> 3);
    pa[i] = (lane & 7) ^ ((row >> 1) & 7);
    oa[i] = (uint32_t)(min(m0 + row, M - 1) - m0) * (uint32_t)K + 16 * pa[i];
  }
#pragma unroll
  for (int i = 0; i < Cfg::kNB; ++i) {
    const int row = 16 * (wave + G * i) + (lane >> 2);
    ob[i] = (uint32_t)(min(n0 + row, N - 1) - n0) * (uint32_t)(K / 2) + 16 * pb;
  }
  // DMAs first .. last - 1 of a chunk (the activation's, then the weight's)
  auto issue = [&](int kc, int stage, int first, int last) {
    uint8_t *st = ring + stage * Cfg::kStage;
    const int want = k0 + min(kc, run - 1), k = KG == 1 ? want : min(want, nk - 1);
#pragma unroll
    for (int i = 0; i < Cfg::kNA; ++i) {
      if (i < first || i >= last) continue;
      // TAIL: not past the row's last piece
      const uint32_t o = TAIL ? oa[i] + min(128 * k, K - 16 - 16 * (int)pa[i]) : oa[i];
      g2l16((TAIL ? a_tile : a_tile + (int64_t)k * 128) + o, st + (wave + G * i) * 1024);
    }
#pragma unroll
    for (int i = 0; i < Cfg::kNB; ++i) {
      if (Cfg::kNA + i < first || Cfg::kNA + i >= last) continue;
      const uint32_t o = TAIL ? ob[i] + min(64 * k, K / 2 - 16 - 16 * (int)pb) : ob[i];
      g2l16((TAIL ? b_tile : b_tile + (int64_t)k * 64) + o, st + Cfg::kA + (wave + G * i) * 1024);
    }
  };
  // all ones where this lane's block of step t of the run's chunk kc lies inside K, else 0 (SX = 16: the
  // groups share the chunks evenly, as 4 divides their number and KG divides 4)
  static_assert(4 % KG == 0, "even groups");
  auto inside = [&](int kc, int t) {
    if constexpr (TAIL || (KG > 1 && SX != 16)) return (k0 + kc) * 128 + 64 * t + 32 * lh < K ? ~0u : 0u;
    else return ~0u;
  };

  // scales: unit u (wave u % G) is rows 64 u .. of the activation's, then the weight's; block blk is the
  // run's chunks 4 blk .. 4 blk + 3 (past the end: the last ones)
  const uint8_t *srow[Cfg::kSU];
#pragma unroll
  for (int i = 0; i < Cfg::kSU; ++i) {
    const int t = 64 * (wave + G * i) + lane;
    srow[i] = t < Cfg::kR ? as + (int64_t)min(m0 + t, M - 1) * nb
                          : bs + (int64_t)min(n0 + min(t - Cfg::kR, Cfg::kC - 1), N - 1) * nb;
  }
  auto has_unit = [&](int i) { return Cfg::kScaleUnits % G == 0 || wave + G * i < Cfg::kScaleUnits; };
  uint8_t *const swave = ring + Cfg::kScales + wave * 1024;
  u32x4 next_scales[Cfg::kSU];
  auto issue_scales = [&](int blk, int slot) {
#pragma unroll
    for (int i = 0; i < Cfg::kSU; ++i) {
      if (!has_unit(i)) continue;
      uint8_t *const at = swave + slot * Cfg::kSlot + i * (G * 1024);
      if constexpr (SX == 16) {
        g2l16(srow[i] + 16 * min(k0 / 4 + blk, nk / 4 - 1), at);
      } else if constexpr (SX == 4) {
#pragma unroll
        for (int w = 0; w < 4; ++w) g2l4(srow[i] + 4 * min(k0 + 4 * blk + w, nk - 1), at + 256 * w);
      } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) next_scales[i][w] = scale_word_raw(srow[i], min(k0 + 4 * blk + w, nk - 1), nb);
      }
    }
  };
  auto put_scales = [&](int blk, int slot) {  // SX = 1: the registers' words; the DMAs need no such step
    if constexpr (SX == 1) {
#pragma unroll
      for (int i = 0; i < Cfg::kSU; ++i) {
        u32x4 v;
#pragma unroll
        for (int w = 0; w < 4; ++w) v[w] = scale_word_shift(next_scales[i][w], min(k0 + 4 * blk + w, nk - 1), nb);
        if (has_unit(i)) *reinterpret_cast<u32x4 *>(swave + slot * Cfg::kSlot + i * (G * 1024) + 16 * lane) = v;
      }
    }
  };

  // Raw operands.  Step t of a chunk takes activation pieces 4 t + 2 h (Af[.][0]: substeps 0, 1) and the
  // next (Af[.][1]: substeps 2, 3) and weight piece 2 t + h (Bf[t]), from their swizzled slots.  Each is
  // read again for the next step as soon as it has been widened.
  u32x4 Af[TM][2], Bf[2][TN];
  uint32_t Sa[TM], Sb[TN];
  const int ra = lr * 128 + (((2 * lh) ^ ((lr >> 1) & 7)) << 4), rb = lr * 64 + ((lh ^ ((lr >> 2) & 3)) << 4);
  auto read_act = [&](int stage, int t, int half) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
      Af[i][half] = *reinterpret_cast<const u32x4 *>(ring + stage * Cfg::kStage + (wm * TM + i) * 4096 +
                                                     (ra ^ (64 * t + 16 * half)));
  };
  auto read_weight = [&](int stage, int t) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      Bf[t][j] = *reinterpret_cast<const u32x4 *>(ring + stage * Cfg::kStage + Cfg::kA + (wn * TN + j) * 2048 +
                                                  (rb ^ (32 * t)));
  };
  auto read_scales = [&](int slot, int word, uint32_t (&sa)[TM], uint32_t (&sb)[TN]) {
    const uint8_t *sc = ring + Cfg::kScales + slot * Cfg::kSlot;
    auto at = [&](int row32) {  // row 32 row32 + lr of the slot
      return SX == 4 ? (row32 >> 1) * 1024 + word * 256 + (row32 & 1) * 128 + lr * 4 : row32 * 512 + lr * 16 + word * 4;
    };
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[i] = *reinterpret_cast<const uint32_t *>(sc + at(wm * TM + i));
#pragma unroll
    for (int j = 0; j < TN; ++j) sb[j] = *reinterpret_cast<const uint32_t *>(sc + at(Cfg::kR / 32 + wn * TN + j));
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  // All but the last n of this wave's DMAs have landed, and so have the other waves' of its ring; a wave
  // with a ring of its own waits for nobody.
  auto arrive = [&](auto n) {
    if constexpr (G == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(decltype(n)::value) : "memory");
    else wait_vmem_then_barrier<decltype(n)::value>();
  };
#pragma unroll
  for (int s = 0; s < Cfg::kSlots - 1; ++s) {
    issue_scales(s, s);
    if (s + 2 < Cfg::kSlots) put_scales(s, s);  // the registers hold one block
  }
#pragma unroll
  for (int s = 0; s < S; ++s) issue(s, s, 0, Cfg::kDmas);
  put_scales(Cfg::kSlots - 2, Cfg::kSlots - 2);
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0) alone
  arrive(std::integral_constant<int, (S - 1) * Cfg::kDmas>{});  // chunk 0 and scale block 0 are there
  read_weight(0, 0);
  read_act(0, 0, 0);
  read_act(0, 0, 1);
  read_scales(0, 0, Sa, Sb);

  // Operands of 8 k's (a quarter of a step), widened.  Step t: lane (r, h) takes block 2 t + h.
  bf16x8 wa[TM], wb[2][TN];
  const uint32_t turn[2] = {scale_turn(lh), scale_turn(2 + lh)};
  auto widen_a = [&](int t, int u, int i, uint32_t word) {
    wa[i] = widen_act(Af[i][u >> 1][2 * (u & 1)], Af[i][u >> 1][2 * (u & 1) + 1], scale_at(word, turn[t]));
  };
  auto widen_b = [&](int t, int u, int j, uint32_t word, uint32_t mask) {
    wb[u & 1][j] = widen_weight(Bf[t][j][u] & mask, scale_at(word, turn[t]));
  };
  // The products of substep u, and behind those that use it last each operand of the next (t, v)
  auto substep = [&](int u, int t, int v, const uint32_t (&sa)[TM], const uint32_t (&sb)[TN], uint32_t mask) {
#pragma unroll
    for (int j = 0; j < TN; ++j) widen_b(t, v, j, sb[j], mask);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[u & 1][j], wa[i], acc[i][j], 0, 0, 0);
      widen_a(t, v, i, sa[i]);
    }
  };
#pragma unroll
  for (int j = 0; j < TN; ++j) widen_b(0, 0, j, Sb[j], inside(0, 0));
#pragma unroll
  for (int i = 0; i < TM; ++i) widen_a(0, 0, i, Sa[i]);
  // Instruction order of a substep.  The matrix instructions run beside the vector unit only if they are
  // not issued back to back: behind each go a share of the conversions for the next substep, the operand
  // reads and the DMAs.
#define W4A8_ORDER(READS, DMAS)                                                                               \
  _Pragma("unroll") for (int i = 0; i < TM * TN; ++i) {                                                       \
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);                                     /* matrix */          \
    if (2 * i < (READS)) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);              /* LDS reads */       \
    if (i * (DMAS) / (TM * TN) != (i + 1) * (DMAS) / (TM * TN)) __builtin_amdgcn_sched_group_barrier(0x20, 1, 0); \
    __builtin_amdgcn_sched_group_barrier(0x2, (4 * (TM + TN) + TM * TN - 1) / (TM * TN), 0); /* conversions */ \
  }
  // one chunk; P = kc % 4 (compile time: the body is one basic block, which keeps the two steps'
  // products on their sides of the barrier)
  // scale DMAs that may stay in flight in phase 1; none where not every wave has them, or where they are plain
  // loads, whose number is the compiler's
  constexpr int kScaleDmas = Cfg::kScaleUnits % G == 0 && SX != 1 ? Cfg::kSU * (SX == 16 ? 1 : 4) : 0;
  int stage = 0, slot = 0;
  auto chunk = [&](int kc, auto phase) {
    constexpr int P = decltype(phase)::value;
    const int nxt = stage == S - 1 ? 0 : stage + 1;
    const int free_slot = slot == 0 ? Cfg::kSlots - 1 : slot - 1;  // of the block before this one
    const uint32_t in0 = inside(kc, 0), in1 = inside(kc, 1);
    if constexpr (P == 2) put_scales((kc >> 2) + Cfg::kSlots - 1, free_slot);
    read_weight(stage, 1);
    substep(0, 0, 1, Sa, Sb, in0);
    W4A8_ORDER(TN, 0)
    read_act(stage, 1, 0);
    substep(1, 0, 2, Sa, Sb, in0);
    W4A8_ORDER(TM, 0)
    substep(2, 0, 3, Sa, Sb, in0);
    W4A8_ORDER(0, 0)
    read_act(stage, 1, 1);
    substep(3, 1, 0, Sa, Sb, in1);
    W4A8_ORDER(TM, 0)
    // step 1's operands have arrived (so this stage is free once every wave is here), the scale
    // words are written, and the next chunk has landed: only those after it (and, in phase 1, the
    // scale loads issued behind them) are still on their way
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0) alone
    arrive(std::integral_constant<int, (S - 2) * Cfg::kDmas + (P == 1 ? kScaleDmas : 0)>{});
    __builtin_amdgcn_sched_barrier(0);
    uint32_t Na[TM], Nb[TN];
    if constexpr (P == 3) slot = slot == Cfg::kSlots - 1 ? 0 : slot + 1;
    read_scales(slot, (P + 1) & 3, Na, Nb);
    read_weight(nxt, 0);
    constexpr int D = Cfg::kDmas, D1 = (D + 3) / 4, D2 = (D + 1) / 2, D3 = (3 * D + 3) / 4;
    issue(kc + S, stage, 0, D1);
    substep(0, 1, 1, Sa, Sb, in1);
    W4A8_ORDER(TM + 2 * TN, D1)
    read_act(nxt, 0, 0);
    issue(kc + S, stage, D1, D2);
    substep(1, 1, 2, Sa, Sb, in1);
    W4A8_ORDER(TM, D2 - D1)
    issue(kc + S, stage, D2, D3);
    substep(2, 1, 3, Sa, Sb, in1);
    W4A8_ORDER(0, D3 - D2)
    read_act(nxt, 0, 1);
    issue(kc + S, stage, D3, D);
    if constexpr (P == 0) issue_scales((kc >> 2) + Cfg::kSlots - 1, free_slot);
    substep(3, 0, 0, Na, Nb, inside(kc + 1, 0));
    W4A8_ORDER(TM, D - D3)
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < TM; ++i) Sa[i] = Na[i];
#pragma unroll
    for (int j = 0; j < TN; ++j) Sb[j] = Nb[j];
    stage = nxt;
  };
  int kc = 0;
  for (; kc + 3 < run; kc += 4) {
    chunk(kc, std::integral_constant<int, 0>{});
    chunk(kc + 1, std::integral_constant<int, 1>{});
    chunk(kc + 2, std::integral_constant<int, 2>{});
    chunk(kc + 3, std::integral_constant<int, 3>{});
  }
  if (kc < run) chunk(kc, std::integral_constant<int, 0>{});
  if (kc + 1 < run) chunk(kc + 1, std::integral_constant<int, 1>{});
  if (kc + 2 < run) chunk(kc + 2, std::integral_constant<int, 2>{});

  wait_vmem();  // the last DMAs target the rings, which now stage sums and output
  __syncthreads();
  if constexpr (KG > 1) {
    auto part = [&](int g, int i, int j, int v4) {  // 4 of the 16 sums of tile (i, j)
      return reinterpret_cast<f32x4 *>(smem + ((g - 1) * G + wave) * Cfg::kPart + (i * TN + j) * 4096 + v4 * 1024 +
                                       lane * 16);
    };
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            *part(kg, i, j, v) = f32x4{acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]};
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int g = 1; g < KG; ++g)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const f32x4 q = *part(g, i, j, v);
            acc[i][j][4 * v] += q.x;
            acc[i][j][4 * v + 1] += q.y;
            acc[i][j][4 * v + 2] += q.z;
            acc[i][j][4 * v + 3] += q.w;
          }
  }
  typedef typename std::conditional<OUT == 0, float, __bf16>::type OutT;
  const bool vec = (ldc * (int64_t)sizeof(OutT)) % 16 == 0;
  constexpr int CW = Cfg::kC / WN;
  const int row0 = m0 + wm * (Cfg::kR / Cfg::WM), col0 = n0 + wn * CW;
  uint8_t *const slab = smem + Cfg::kEpi + wave * Cfg::kEpiWave;
  if (vec) store_tile<CW, TM, TN, OutT, true>(acc, 1.0f, static_cast<OutT *>(c), ldc, M, N, row0, col0, true, slab, lane);
  else store_tile_unaligned<CW, TM, TN>(acc, static_cast<OutT *>(c), ldc, M, N, row0, col0, slab, lane);
}

// ---- few rows -----------------------------------------------------------------------------------------
//
// Bound by latency: the weight is read once, 17/32 B a value, and there are few bytes to a CU (4608 x 1152
// for one row: 3.2 us, 2.0 of them the launch and 2.06 a bare read of the weight; 4096 x 4096: 4.9 us; the
// weight in the last-level cache).
// A workgroup owns 16 NT output columns and up to 16 MT rows; its W waves take every W-th run of U 128-k
// chunks and their sums are added in LDS in the order of the runs.  Operands straight from memory: lane (r, q) = (l % 16, l / 16)
// takes block q of row r, and its 32 values make four v_mfma_f32_16x16x32_bf16 of 8 k from every block.
// A weight load covers 64 contiguous bytes of 16 rows.  U chunks' loads are in flight while the U before
// them multiply.

template <int OUT, int W, int MT, int NT, int U>
__global__ __launch_bounds__(64 * W) void k_w4a8_rows(const uint8_t *__restrict__ a, const uint8_t *__restrict__ as,
                                                      const uint8_t *__restrict__ b, const uint8_t *__restrict__ bs,
                                                      int M, int N, int K, void *__restrict__ c, int64_t ldc) {
  static_assert((W & (W - 1)) == 0, "waves");
  __shared__ f32x4 part[W][MT * NT][64];
  const int lane = threadIdx.x & 63;
  // Workgroups of one XCD (every 8th) start at different runs, so that they do not all ask its L2 for
  // the same activation lines at once.
  const int wave = __builtin_amdgcn_readfirstlane(((threadIdx.x >> 6) + (blockIdx.x >> 3)) & (W - 1));
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * (16 * NT), m0 = blockIdx.y * (16 * MT);
  const int nk = (K + 127) / 128, nb = K / 32;

  const uint8_t *pa[MT], *pb[NT], *psa[MT], *psb[NT];
  bool row_in[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = min(m0 + 16 * i + r, M - 1);
    row_in[i] = m0 + 16 * i + r < M;
    pa[i] = a + row * K;
    psa[i] = as + row * nb;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t row = min(n0 + 16 * j + r, N - 1);
    pb[j] = b + row * (K / 2);
    psb[j] = bs + row * nb;
  }

  // A run of U chunks.  Past the end of K the weights are zero; the activation is then read from inside
  // the row (finite).  Rows past M are zero and not read.
  struct Run {
    u32x4 a[U][MT][2], b[U][NT];
    uint32_t sa[MT][U], sb[NT][U];
  };
  auto fetch = [&](int kc, Run &f) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = 128 * (kc + u) + 32 * q;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        f.b[u][j] = u32x4{0, 0, 0, 0};
        if (kb < K) f.b[u][j] = *reinterpret_cast<const u32x4 *>(pb[j] + kb / 2);
      }
      const int ka = min(kb, K - 32);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        f.a[u][i][0] = f.a[u][i][1] = u32x4{0, 0, 0, 0};
        if (row_in[i]) {
          f.a[u][i][0] = *reinterpret_cast<const u32x4 *>(pa[i] + ka);
          f.a[u][i][1] = *reinterpret_cast<const u32x4 *>(pa[i] + ka + 16);
        }
      }
    }
    typedef uint32_t words_t __attribute__((ext_vector_type(U), aligned(1)));
    const bool whole = 4 * (kc + U) <= nb;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (whole) {
        const words_t v = *reinterpret_cast<const words_t *>(psa[i] + 4 * kc);
#pragma unroll
        for (int u = 0; u < U; ++u) f.sa[i][u] = v[u];
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) f.sa[i][u] = scale_word(psa[i], min(kc + u, nk - 1), nb);
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (whole) {
        const words_t v = *reinterpret_cast<const words_t *>(psb[j] + 4 * kc);
#pragma unroll
        for (int u = 0; u < U; ++u) f.sb[j][u] = v[u];
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) f.sb[j][u] = scale_word(psb[j], min(kc + u, nk - 1), nb);
      }
    }
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const uint32_t turn = scale_turn(q);
  auto multiply = [&](const Run &f) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float Xa[MT], Xb[NT];
#pragma unroll
      for (int i = 0; i < MT; ++i) Xa[i] = scale_at(f.sa[i][u], turn);
#pragma unroll
      for (int j = 0; j < NT; ++j) Xb[j] = scale_at(f.sb[j][u], turn);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 wb[NT], wa[MT];
#pragma unroll
        for (int j = 0; j < NT; ++j) wb[j] = widen_weight(f.b[u][j][s], Xb[j]);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          wa[i] = widen_act(f.a[u][i][s >> 1][2 * (s & 1)], f.a[u][i][s >> 1][2 * (s & 1) + 1], Xa[i]);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], wa[i], acc[i][j], 0, 0, 0);
      }
    }
  };

  Run now, next;
  if (wave * U < nk) {
    fetch(wave * U, now);
    for (int kc = wave * U; kc < nk; kc += W * U) {
      const bool more = kc + W * U < nk;
      if (more) fetch(kc + W * U, next);
      multiply(now);
      if (more) now = next;
    }
  }

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  // element (lane l, e) of tile (i, j): row m = 16 i + l % 16, column n = 16 j + 4 (l / 16) + e
  const bool vec = ldc % 4 == 0;
  for (int t = threadIdx.x; t < MT * NT * 64; t += 64 * W) {
    const int tile = t >> 6, l = t & 63;
    const int m = m0 + 16 * (tile / NT) + (l & 15), n = n0 + 16 * (tile % NT) + 4 * (l >> 4);
    if (m >= M) continue;
    f32x4 v = part[0][tile][l];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w][tile][l];
    if (vec && n + 4 <= N) {
      if (OUT == 0) {
        *reinterpret_cast<f32x4 *>(static_cast<float *>(c) + m * ldc + n) = v;
      } else {
        const bf16x2 lo = {(__bf16)v.x, (__bf16)v.y}, hi = {(__bf16)v.z, (__bf16)v.w};
        *reinterpret_cast<u32x2 *>(static_cast<__bf16 *>(c) + m * ldc + n) =
            u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
      }
      continue;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e < N) {
        if (OUT == 0) static_cast<float *>(c)[m * ldc + n + e] = v[e];
        else static_cast<__bf16 *>(c)[m * ldc + n + e] = (__bf16)v[e];
      }
    }
  }
}

// ---- launchers ----------------------------------------------------------------------------------------

hipError_t launch_mx8_quantize(const void *x, int dtype, int64_t M, int64_t K, int64_t ld, uint8_t *codes,
                               uint8_t *scales, hipStream_t s) {
  const FastDiv bpr = make_fastdiv((uint32_t)(K / kMx8Blk));
  const uint64_t nseg = (uint64_t)M * (uint64_t)K / 8;
  const unsigned grid = (unsigned)((nseg + 511) / 512);
  const bool dense = ld == K;
  if (dtype == 0) {
    if (dense) k_mx8_quantize<0, true><<<grid, 256, 0, s>>>(x, ld, nseg, bpr, codes, scales);
    else k_mx8_quantize<0, false><<<grid, 256, 0, s>>>(x, ld, nseg, bpr, codes, scales);
  } else {
    if (dense) k_mx8_quantize<1, true><<<grid, 256, 0, s>>>(x, ld, nseg, bpr, codes, scales);
    else k_mx8_quantize<1, false><<<grid, 256, 0, s>>>(x, ld, nseg, bpr, codes, scales);
  }
  return hipGetLastError();
}

namespace {

template <int OUT, class Cfg, int SX>
hipError_t launch_tiles_sx(const W4A8Args &g, int run, hipStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];  // per instantiation and device
  auto kern = k_w4a8<OUT, Cfg, SX>;
  hipError_t e = set_dynamic_lds(reinterpret_cast<const void *>(kern), Cfg::kLds, configured);
  if (e != hipSuccess) return e;
  const int tm = (int)((g.M + Cfg::kR - 1) / Cfg::kR), tn = (int)((g.N + Cfg::kC - 1) / Cfg::kC);
  kern<<<tm * tn, Cfg::kThreads, Cfg::kLds, s>>>(g.a, g.as, g.b, g.bs, (int)g.M, (int)g.N, (int)g.K, g.c, g.ldc, tm, tn,
                                                 run);
  return hipGetLastError();
}

template <int OUT, class Cfg>
hipError_t launch_tiles(const W4A8Args &g, hipStream_t s) {
  const int nk = (int)((g.K + 127) / 128), run = (nk + Cfg::KG - 1) / Cfg::KG;
  if (g.K % 128 != 0) return launch_tiles_sx<OUT, Cfg, 1>(g, run, s);
  const uintptr_t at = reinterpret_cast<uintptr_t>(g.as) | reinterpret_cast<uintptr_t>(g.bs);
  if (g.K % 512 == 0 && at % 16 == 0 && (Cfg::KG == 1 || run % 4 == 0)) return launch_tiles_sx<OUT, Cfg, 16>(g, run, s);
  return launch_tiles_sx<OUT, Cfg, 4>(g, run, s);
}

template <int OUT, int W, int MT, int NT, int U>
hipError_t launch_rows(const W4A8Args &g, hipStream_t s) {
  const dim3 grid((unsigned)((g.N + 16 * NT - 1) / (16 * NT)), (unsigned)((g.M + 16 * MT - 1) / (16 * MT)));
  k_w4a8_rows<OUT, W, MT, NT, U><<<grid, 64 * W, 0, s>>>(g.a, g.as, g.b, g.bs, (int)g.M, (int)g.N, (int)g.K, g.c, g.ldc);
  return hipGetLastError();
}

// Which kernel.  One tile per CU (there are 256) is the aim: a workgroup alone on its CU takes, per 128 k,
// 0.14 us for 32 x 32, 0.2 for 64 x 32, 0.33 for 64 x 64, 0.48 for 128 x 64, 0.68 for 128 x 128 and 2.1 for
// 256 x 256 (8192 x 8192 weights), so the smallest tile that still needs one round is the fastest, e.g. for
// M = 64: 32 x 32 8.0 us and 64 x 32 10.0 (1152 x 4608), 21.3 and 16.5 (8192 x 8192, where 32 x 32 needs two
// rounds); M = 512 x 4608 x 1152: 128 x 64 12.2, 128 x 128 11.1; M = 2048 x 8192 x 8192: 128 x 128 209,
// 256 x 256 192.  Past one round the 128 x 128 tiles, two of which share a CU, and the 256 x 256 tiles are
// compared by what their rounds cost.  All of this was measured on weights of 1152 to 8192 columns that stay in the
// last-level cache.  Few rows of wider weights also take the tall tiles, most of whose rows are copies: N = 12288,
// K = 3072 10.2 us for one row and 28672 x 8192 51.1, where a read of the weight takes 3.4 and 21.2.
template <int OUT>
hipError_t launch_out(const W4A8Args &g, hipStream_t s) {
  auto tiles = [&](int64_t r, int64_t c) { return ((g.M + r - 1) / r) * ((g.N + c - 1) / c); };
  // the tiles' row offsets are 32 bits, and their scale rows at least a word; the few-row kernel that takes
  // shorter ones is launched over rows in y
  if (256 * g.K >= (int64_t(1) << 31) || (g.K < 128 && (g.M > 32 * 65535 || tiles(32, 16) > (1 << 22)))) {
    int64_t grid = (g.M * g.N + 255) / 256;
    if (grid > 65536) grid = 65536;
    k_w4a8_generic<OUT><<<(unsigned)grid, 256, 0, s>>>(g.a, g.as, g.b, g.bs, g.M, g.N, g.K, g.c, g.ldc);
    return hipGetLastError();
  }
  const int64_t nk = (g.K + 127) / 128;
  // Few rows: up to about 192 blocks of 32 columns the kernel without staging is faster (one row, 4096 x
  // 4096: 4.9 us and 6.9; 16 rows: 6.6 and 7.0), above it the staged tile (16 rows, 8192 x 8192: 18.3 and
  // 12.2).  Sixteen waves need K to share (1152 x 4608: 4.8 us, with eight 5.0; 4608 x 1152: 4.5 and 3.7).
  // 17 to 32 rows gain for small weights only (1152 x 1152: 4.4 us and 5.5; 1152 x 4608: 8.9 and 7.9).
  // Rows of scales below a word (K < 128) are read here.
  if (g.M <= 16 && g.N <= 6144)
    return nk > 16 ? launch_rows<OUT, 16, 1, 1, 2>(g, s) : launch_rows<OUT, 8, 1, 1, 2>(g, s);
  if ((g.M <= 32 && g.N <= 2048 && nk <= 18) || g.K < 128) return launch_rows<OUT, 8, 2, 1, 2>(g, s);
  // The 32 x 32 tile shares a CU with a second one (64 x 4608 x 1152, 288 tiles: 6.3 us and 6.5 with 64 x 32).
  if (tiles(32, 32) <= 300) return launch_tiles<OUT, TileCfg<32, 32, 1, 1, 4, 3>>(g, s);
  if (tiles(64, 32) <= 256) return launch_tiles<OUT, TileCfg<64, 32, 2, 1, 4, 3>>(g, s);
  // Long K: a wave to 64 x 64, with half the conversions per product, in four or two groups (128 x 8192 x
  // 8192: 21.7 us and 24.4; 256 x 8192 x 8192: 34.6 and 41.3); short K: more waves on the tile (256 x 4096 x
  // 4096: 13.6 us and 14.0; 512 x 4608 x 1152: 12.2 and 16.6).
  if (tiles(64, 64) <= 256)
    return nk >= 48 ? launch_tiles<OUT, TileCfg<64, 64, 1, 1, 4, 3>>(g, s) : launch_tiles<OUT, TileCfg<64, 64, 2, 2, 2, 3>>(g, s);
  if (tiles(128, 64) <= 256)
    return nk >= 24 ? launch_tiles<OUT, TileCfg<128, 64, 2, 1, 2, 3>>(g, s) : launch_tiles<OUT, TileCfg<128, 64, 2, 2, 1, 3>>(g, s);
  const double small = 0.29 / 256 * (double)tiles(128, 128), big = (double)((tiles(256, 256) + 255) / 256);
  return small <= big ? launch_tiles<OUT, TileCfg<128, 128, 2, 2, 1, 3>>(g, s)
                      : launch_tiles<OUT, TileCfg<256, 256, 2, 4, 1, 3>>(g, s);
}

}  // namespace

hipError_t launch_w4a8(const W4A8Args &g, hipStream_t s) {
  return g.out_dtype == 0 ? launch_out<0>(g, s) : launch_out<1>(g, s);
}

}  // namespace nvfp4
