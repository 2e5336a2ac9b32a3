// MXFP8 quantize, and the product of MXFP8 activations with MXFP4 weights (W4A8), for gfx950.
//
// Y[m][n] = sum_k a[m][k] Xa[m][k / 32] b[n][k] Xb[n][k / 32]: E4M3 codes times E2M1 codes under
// E8M0 scales, exact products, fp32 sums.
#include <type_traits>

#include "epilogue.hpp"
#include "launch.hpp"
#include "mx8.hpp"

namespace nvfp4 {

// A lane takes 8 consecutive elements, 4 adjacent lanes a block.
template <int DT, bool DENSE>
__global__ __launch_bounds__(256) void k_mx8_quantize(const void *__restrict__ x, int64_t ld, uint64_t nseg,
                                                      FastDiv bpr, uint8_t *__restrict__ codes,
                                                      uint8_t *__restrict__ scales) {
  for (uint64_t g = blockIdx.x * 256ull + threadIdx.x; g < nseg; g += gridDim.x * 256ull) {
    int64_t off = (int64_t)g * 8;
    if (!DENSE) {
      const uint32_t blk = (uint32_t)(g >> 2), row = fastdiv(blk, bpr);
      off = (int64_t)row * ld + (int64_t)(blk - row * bpr.d) * kMx8Blk + 8 * (int64_t)(g & 3);
    }
    Vec8<DT> v;
    v.template load<true>(x, off);
    float f[8];
    v.get(f);
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
      const float X = mx8_scale_value(as[(m * K + k) / kMx8Blk]) * mx8_scale_value(bs[(n * K + k) / kMx8Blk]);
      float part = 0.0f;
      for (int i = 0; i < kMx8Blk; i += 2) {
        const uint32_t w = b[(n * K + k + i) / 2];
        const f32x2 q = fp4_decode2_f32<0>(w);
        part = fmaf(e4m3_to_f32(a[m * K + k + i]), q.x, part);
        part = fmaf(e4m3_to_f32(a[m * K + k + i + 1]), q.y, part);
      }
      acc = fmaf(part, X, acc);
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
// the codes are widened to bf16 with their scale (exact: at most 4 significant bits; one conversion
// instruction per two values) and multiplied by v_mfma_f32_32x32x16_bf16, at half the rate.
//
// Operands of a 64-k step: lane (r, h) = (l % 32, l / 32) takes block h of row r: 32 activation bytes, 16
// weight bytes, one scale each; its 32 values make four matrix instructions of 8 k from either block.  In
// 16-byte pieces of a 128-k chunk (8 per activation row, 4 per weight row) step t takes activation
// pieces 4 t + 2 h and the next, and weight piece 2 t + h: both operands stream from their canonical
// layouts by LDS-DMA.
//
// T x T tile per workgroup of WM x WN waves; K in chunks of 128 in a ring of 3 LDS stages:
//   activation [T / 16 blocks of 16 rows][8 pieces][16 rows][16 B]   weight [T / 16][4 pieces][16][16 B]
// A DMA fills 4 pieces of 16 rows (64 contiguous bytes of each row) and every 16-lane pass of an operand
// read is one contiguous 256-byte span.  Scales: [2 slots][2 operands], blocks of 4 chunks (16 bytes of a
// row), one row per thread: a 16-byte DMA lane, four 4-byte ones ([64 rows' chunk 0][chunk 1]..), or, where
// rows of scales are not aligned, registers that are written to LDS two chunks later.
//
// A chunk is two 64-k steps.  While step 0 multiplies, step 1's operands are read; in the middle one
// barrier says that the next chunk has landed everywhere and that this one's stage is free, the DMA of
// the chunk after the next two starts into it, and while step 1 multiplies the next chunk's step 0 is read.
// Rows past M or N repeat the last one and are never stored.  Where K is no multiple of 128 (TAIL), the
// last chunk's missing pieces are fetched from a zero page: their products are 0 under any finite scale.

__device__ uint8_t zero_page[64];

namespace {

typedef uint32_t u32_any __attribute__((aligned(1)));

// A scale byte as the float the conversions take (they read its exponent field).
__device__ __forceinline__ float scale_of(uint32_t word, int byte) {
  return __uint_as_float(((word >> (8 * byte)) & 255u) << 23);
}
// 8 E4M3 codes of words lo, hi, or the 8 E2M1 codes of a word, times their scale: exact in bf16.
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

template <int T, int WM, int WN>
struct TileCfg {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kTM = T / 32 / WM, kTN = T / 32 / WN;
  static constexpr int kA = T * 128, kB = T * 64, kStage = kA + kB, kStages = 3;
  static constexpr int kScales = kStages * kStage, kScaleOp = T * 16;
  static constexpr int kLds = kScales + 4 * kScaleOp;
  static constexpr int kNA = 2 * (T / 16) / kWaves, kNB = (T / 16) / kWaves, kSlots = kNA + kNB;
  static_assert(kNA * kWaves == T / 8 && kNB * kWaves == T / 16, "even DMA split");
  static_assert(kThreads == 2 * T, "one scale row per thread");
  static_assert(kLds <= 160 * 1024, "LDS fits");
};

}  // namespace

// SX: how a row's scale bytes of 4 chunks are loaded -- 16: one 16-byte DMA lane (K % 512 == 0, 16-byte
// aligned arrays), 4: four 4-byte ones (K % 128 == 0), 1: unaligned words, bytes at the end (TAIL)
template <int OUT, int T, int WM, int WN, int SX>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_w4a8(
    const uint8_t *__restrict__ a, const uint8_t *__restrict__ as, const uint8_t *__restrict__ b,
    const uint8_t *__restrict__ bs, int M, int N, int K, void *__restrict__ c, int64_t ldc, int tiles_m, int tiles_n) {
  using Cfg = TileCfg<T, WM, WN>;
  constexpr int TM = Cfg::kTM, TN = Cfg::kTN, S = Cfg::kStages, W = Cfg::kWaves;
  constexpr bool TAIL = SX == 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
  const int m0 = tmi * T, n0 = tni * T;
  const int nk = (K + 127) / 128, nb = K / 32;

  const uint8_t *a_tile = a + (int64_t)m0 * K, *b_tile = b + (int64_t)n0 * (K / 2);
  const int piece = lane >> 4;
  uint32_t oa[Cfg::kNA], ob[Cfg::kNB];
#pragma unroll
  for (int i = 0; i < Cfg::kNA; ++i) {
    const int d = wave + W * i, row = 16 * (d >> 1) + (lane & 15);  // DMA d: rows 16 (d / 2) .., pieces 4 (d % 2) ..
    oa[i] = (uint32_t)(min(m0 + row, M - 1) - m0) * (uint32_t)K + 64 * (d & 1) + 16 * piece;
  }
#pragma unroll
  for (int i = 0; i < Cfg::kNB; ++i) {
    const int row = 16 * (wave + W * i) + (lane & 15);
    ob[i] = (uint32_t)(min(n0 + row, N - 1) - n0) * (uint32_t)(K / 2) + 16 * piece;
  }
  auto issue = [&](int kc, int stage) {
    uint8_t *st = smem + stage * Cfg::kStage;
#pragma unroll
    for (int i = 0; i < Cfg::kNA; ++i) {
      const uint8_t *p = a_tile + (int64_t)kc * 128 + oa[i];
      if (TAIL && kc * 128 + 64 * ((wave + W * i) & 1) + 16 * piece >= K) p = zero_page;
      g2l16(p, st + (wave + W * i) * 1024);
    }
#pragma unroll
    for (int i = 0; i < Cfg::kNB; ++i) {
      const uint8_t *p = b_tile + (int64_t)kc * 64 + ob[i];
      if (TAIL && kc * 128 + 32 * piece >= K) p = zero_page;
      g2l16(p, st + Cfg::kA + (wave + W * i) * 1024);
    }
  };

  // scales: this thread's row; block blk is chunks 4 blk .. 4 blk + 3 (past the end: the last ones)
  const uint8_t *srow;
  {
    const int t = threadIdx.x % T;
    srow = threadIdx.x < T ? as + (int64_t)min(m0 + t, M - 1) * nb : bs + (int64_t)min(n0 + t, N - 1) * nb;
  }
  uint8_t *const swave = smem + Cfg::kScales + wave * 1024;  // both operands' rows in thread order
  u32x4 next_scales = {0, 0, 0, 0};
  auto issue_scales = [&](int blk) {
    uint8_t *const at = swave + (blk & 1) * (2 * Cfg::kScaleOp);
    if constexpr (SX == 16) {
      g2l16(srow + 16 * min(blk, nk / 4 - 1), at);
    } else if constexpr (SX == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) g2l4(srow + 4 * min(4 * blk + i, nk - 1), at + 256 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) next_scales[i] = scale_word(srow, min(4 * blk + i, nk - 1), nb);
    }
  };
  auto put_scales = [&](int blk) {  // SX = 1: the registers' words; the DMAs need no such step
    uint8_t *const at = swave + (blk & 1) * (2 * Cfg::kScaleOp);
    if constexpr (SX == 1) *reinterpret_cast<u32x4 *>(at + 16 * lane) = next_scales;
  };

  u32x4 Af[2][TM][2], Bf[2][TN];
  uint32_t Sa[TM], Sb[TN];
  // operands of step t of the chunk in `stage`
  auto read_step = [&](int stage, int t) {
    const uint8_t *st = smem + stage * Cfg::kStage;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const uint8_t *p = st + (2 * (wm * TM + i) + (lr >> 4)) * 2048 + ((4 * t + 2 * lh) * 16 + (lr & 15)) * 16;
      Af[t][i][0] = *reinterpret_cast<const u32x4 *>(p);
      Af[t][i][1] = *reinterpret_cast<const u32x4 *>(p + 256);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j)
      Bf[t][j] = *reinterpret_cast<const u32x4 *>(st + Cfg::kA + (2 * (wn * TN + j) + (lr >> 4)) * 1024 +
                                                  ((2 * t + lh) * 16 + (lr & 15)) * 16);
  };
  auto read_scales = [&](int kc, uint32_t (&sa)[TM], uint32_t (&sb)[TN]) {
    const uint8_t *sc = smem + Cfg::kScales + ((kc >> 2) & 1) * (2 * Cfg::kScaleOp);
    auto at = [&](int grp) {  // row 32 grp + lr
      return SX == 4 ? (grp >> 1) * 1024 + (kc & 3) * 256 + (grp & 1) * 128 + lr * 4 : grp * 512 + lr * 16 + (kc & 3) * 4;
    };
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[i] = *reinterpret_cast<const uint32_t *>(sc + at(wm * TM + i));
#pragma unroll
    for (int j = 0; j < TN; ++j) sb[j] = *reinterpret_cast<const uint32_t *>(sc + Cfg::kScaleOp + at(wn * TN + j));
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  issue_scales(0);
  put_scales(0);
#pragma unroll
  for (int s = 0; s < S; ++s) issue(min(s, nk - 1), s);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  wait_vmem_then_barrier<(S - 1) * Cfg::kSlots>();  // chunk 0 and scale block 0 are there
  read_step(0, 0);
  read_scales(0, Sa, Sb);

  // step t: lane (r, h) takes block 2 t + h
  auto multiply = [&](int t) {
    float Xa[TM], Xb[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) Xa[i] = scale_of(Sa[i] >> (8 * lh), 2 * t);
#pragma unroll
    for (int j = 0; j < TN; ++j) Xb[j] = scale_of(Sb[j] >> (8 * lh), 2 * t);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8 wb[TN], wa[TM];
#pragma unroll
      for (int j = 0; j < TN; ++j) wb[j] = widen_weight(Bf[t][j][s], Xb[j]);
#pragma unroll
      for (int i = 0; i < TM; ++i) wa[i] = widen_act(Af[t][i][s >> 1][2 * (s & 1)], Af[t][i][s >> 1][2 * (s & 1) + 1], Xa[i]);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j], wa[i], acc[i][j], 0, 0, 0);
    }
  };
  // one chunk; P = kc % 4 (compile time: the body is one basic block, which keeps the two steps'
  // products on their sides of the barrier)
  int stage = 0;
  auto chunk = [&](int kc, auto phase) {
    constexpr int P = decltype(phase)::value;
    const int nxt = stage == S - 1 ? 0 : stage + 1;
    read_step(stage, 1);
    if constexpr (P == 2) put_scales((kc >> 2) + 1);
    multiply(0);
    // step 1's operands have arrived (so this stage is free once every wave is here), the scale
    // words are written, and the next chunk has landed: only the one after it (and, in phase 1, the
    // scale loads issued behind it) is still on its way
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0) alone
    wait_vmem_then_barrier<Cfg::kSlots + (P == 1 ? (SX == 16 ? 1 : 4) : 0)>();
    __builtin_amdgcn_sched_barrier(0);
    uint32_t Na[TM], Nb[TN];
    read_scales(kc + 1, Na, Nb);
    read_step(nxt, 0);
    issue(min(kc + S, nk - 1), stage);
    if constexpr (P == 0) issue_scales((kc >> 2) + 1);
    multiply(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < TM; ++i) Sa[i] = Na[i];
#pragma unroll
    for (int j = 0; j < TN; ++j) Sb[j] = Nb[j];
    stage = nxt;
  };
  int kc = 0;
  for (; kc + 3 < nk; kc += 4) {
    chunk(kc, std::integral_constant<int, 0>{});
    chunk(kc + 1, std::integral_constant<int, 1>{});
    chunk(kc + 2, std::integral_constant<int, 2>{});
    chunk(kc + 3, std::integral_constant<int, 3>{});
  }
  if (kc < nk) chunk(kc, std::integral_constant<int, 0>{});
  if (kc + 1 < nk) chunk(kc + 1, std::integral_constant<int, 1>{});
  if (kc + 2 < nk) chunk(kc + 2, std::integral_constant<int, 2>{});

  wait_vmem();  // the last DMAs target the ring, which now stages the output
  __syncthreads();
  typedef typename std::conditional<OUT == 0, float, __bf16>::type OutT;
  const bool vec = (ldc * (int64_t)sizeof(OutT)) % 16 == 0;
  constexpr int CW = T / WN;
  static_assert(W * 32 * EpiPitch<CW, 4>::kPitch <= S * Cfg::kStage, "epilogue staging fits the LDS ring");
  store_tile<CW, TM, TN, OutT, true>(acc, 1.0f, static_cast<OutT *>(c), ldc, M, N, m0 + wm * (T / WM), n0 + wn * CW, vec,
                                     smem + wave * (32 * EpiPitch<CW, 4>::kPitch), lane);
}

// ---- few rows -----------------------------------------------------------------------------------------
//
// A workgroup owns 16 NT output columns and up to 16 MT rows; its W waves take every W-th 128-k chunk and
// their sums are added in LDS in wave order.  Operands straight from memory: lane (r, q) = (l % 16, l / 16)
// takes block q of row r, and its 32 values make four v_mfma_f32_16x16x32_bf16 of 8 k from every block.
// A weight load covers 64 contiguous bytes of 16 rows.  U chunks' loads are in flight while the U before
// them multiply.

template <int OUT, int W, int MT, int NT, int U>
__global__ __launch_bounds__(64 * W) void k_w4a8_rows(const uint8_t *__restrict__ a, const uint8_t *__restrict__ as,
                                                      const uint8_t *__restrict__ b, const uint8_t *__restrict__ bs,
                                                      int M, int N, int K, void *__restrict__ c, int64_t ldc) {
  __shared__ f32x4 part[W][MT * NT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * (16 * NT), m0 = blockIdx.y * (16 * MT);
  const int nk = (K + 127) / 128, nb = K / 32;

  const uint8_t *pa[MT], *pb[NT], *psa[MT], *psb[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = min(m0 + 16 * i + r, M - 1);
    pa[i] = a + row * K;
    psa[i] = as + row * nb;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t row = min(n0 + 16 * j + r, N - 1);
    pb[j] = b + row * (K / 2);
    psb[j] = bs + row * nb;
  }

  struct Chunk {
    u32x4 a[MT][2], b[NT];
    uint32_t sa[MT], sb[NT];
  };
  // chunk kc (past the end: zero weights).  Activation pieces past K meet zero weights; they are read
  // from inside the row.
  auto fetch = [&](int kc, Chunk &f) {
    const int k = min(kc, nk - 1);
    const int kb = 128 * k + 32 * q, ka = min(kb, K - 32);
    const bool in = kc < nk && kb < K;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      f.b[j] = u32x4{0, 0, 0, 0};
      if (in) f.b[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(pb[j] + kb / 2));
      f.sb[j] = scale_word(psb[j], k, nb);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      f.a[i][0] = *reinterpret_cast<const u32x4 *>(pa[i] + ka);
      f.a[i][1] = *reinterpret_cast<const u32x4 *>(pa[i] + ka + 16);
      f.sa[i] = scale_word(psa[i], k, nb);
    }
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  auto multiply = [&](const Chunk &f) {
    float Xa[MT], Xb[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) Xa[i] = scale_of(f.sa[i] >> (8 * q), 0);
#pragma unroll
    for (int j = 0; j < NT; ++j) Xb[j] = scale_of(f.sb[j] >> (8 * q), 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8 wb[NT], wa[MT];
#pragma unroll
      for (int j = 0; j < NT; ++j) wb[j] = widen_weight(f.b[j][s], Xb[j]);
#pragma unroll
      for (int i = 0; i < MT; ++i) wa[i] = widen_act(f.a[i][s >> 1][2 * (s & 1)], f.a[i][s >> 1][2 * (s & 1) + 1], Xa[i]);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], wa[i], acc[i][j], 0, 0, 0);
    }
  };

  Chunk now[U], next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) fetch(wave + W * u, now[u]);
  for (int kc = wave; kc < nk; kc += W * U) {
    const bool more = kc + W * U < nk;
    if (more) {
#pragma unroll
      for (int u = 0; u < U; ++u) fetch(kc + W * (U + u), next[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(now[u]);
    if (more) {
#pragma unroll
      for (int u = 0; u < U; ++u) now[u] = next[u];
    }
  }

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  // element (lane l, e) of tile (i, j): row m = 16 i + l % 16, column n = 16 j + 4 (l / 16) + e
  for (int t = threadIdx.x; t < MT * NT * 64; t += 64 * W) {
    const int tile = t >> 6, l = t & 63;
    f32x4 v = part[0][tile][l];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w][tile][l];
    const int m = m0 + 16 * (tile / NT) + (l & 15), n = n0 + 16 * (tile % NT) + 4 * (l >> 4);
    if (m >= M) continue;
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
  uint64_t g = (nseg + 255) / 256;
  const unsigned grid = (unsigned)(g > 16384 ? 16384 : g);
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

template <int OUT, int T, int WM, int WN, int SX>
hipError_t launch_tiles_sx(const W4A8Args &g, hipStream_t s) {
  using Cfg = TileCfg<T, WM, WN>;
  static std::atomic<bool> configured[kMaxDevices];  // per instantiation and device
  auto kern = k_w4a8<OUT, T, WM, WN, SX>;
  hipError_t e = set_dynamic_lds(reinterpret_cast<const void *>(kern), Cfg::kLds, configured);
  if (e != hipSuccess) return e;
  const int tm = (int)((g.M + T - 1) / T), tn = (int)((g.N + T - 1) / T);
  kern<<<tm * tn, Cfg::kThreads, Cfg::kLds, s>>>(g.a, g.as, g.b, g.bs, (int)g.M, (int)g.N, (int)g.K, g.c, g.ldc, tm, tn);
  return hipGetLastError();
}

template <int OUT, int T, int WM, int WN>
hipError_t launch_tiles(const W4A8Args &g, hipStream_t s) {
  if (g.K % 128 != 0) return launch_tiles_sx<OUT, T, WM, WN, 1>(g, s);
  const uintptr_t at = reinterpret_cast<uintptr_t>(g.as) | reinterpret_cast<uintptr_t>(g.bs);
  if (g.K % 512 == 0 && at % 16 == 0) return launch_tiles_sx<OUT, T, WM, WN, 16>(g, s);
  return launch_tiles_sx<OUT, T, WM, WN, 4>(g, s);
}

template <int OUT, int W, int MT, int NT, int U>
hipError_t launch_rows(const W4A8Args &g, hipStream_t s) {
  const dim3 grid((unsigned)((g.N + 16 * NT - 1) / (16 * NT)), (unsigned)((g.M + 16 * MT - 1) / (16 * MT)));
  k_w4a8_rows<OUT, W, MT, NT, U><<<grid, 64 * W, 0, s>>>(g.a, g.as, g.b, g.bs, (int)g.M, (int)g.N, (int)g.K, g.c, g.ldc);
  return hipGetLastError();
}

template <int OUT>
hipError_t launch_out(const W4A8Args &g, hipStream_t s) {
  if (256 * g.K >= (int64_t(1) << 31)) {  // the tiles' row offsets are 32 bits
    int64_t grid = (g.M * g.N + 255) / 256;
    if (grid > 65536) grid = 65536;
    k_w4a8_generic<OUT><<<(unsigned)grid, 256, 0, s>>>(g.a, g.as, g.b, g.bs, g.M, g.N, g.K, g.c, g.ldc);
    return hipGetLastError();
  }
  if (g.M <= 16) return launch_rows<OUT, 8, 1, 2, 2>(g, s);
  if (g.M <= 32) return launch_rows<OUT, 8, 2, 2, 1>(g, s);
  if (g.M <= 64) return launch_rows<OUT, 8, 4, 2, 1>(g, s);
  const int64_t big = ((g.M + 255) / 256) * ((g.N + 255) / 256);
  return big >= 256 ? launch_tiles<OUT, 256, 2, 4>(g, s) : launch_tiles<OUT, 128, 2, 2>(g, s);
}

}  // namespace

hipError_t launch_w4a8(const W4A8Args &g, hipStream_t s) {
  return g.out_dtype == 0 ? launch_out<0>(g, s) : launch_out<1>(g, s);
}

}  // namespace nvfp4
