// Gradients of softmax attention (gfx950).  With P_ij = exp(scale q_i k_j - lse_i), delta_i = sum dO_i O_i,
// dS_ij = P_ij (dO_i v_j - delta_i):
//   dQ_i = scale sum_j dS_ij k_j     dV_j = sum_i P_ij dO_i     dK_j = scale sum_i dS_ij q_i
// with sums over the query heads that share a key head.
//
// Two kernels, one with queries as the columns of its products (as forward) for dQ, one with keys as columns
// for dK and dV: each gradient is summed in one wave's registers in a fixed order, without atomics, for
// computing scores and dO V^T twice (seven products instead of five).  P and dS are rounded to bf16 where
// they are multiplied; everything else is fp32.
//
// Measured (best of 20): 4096 tokens, 16 heads of 72: dQ 145 us, dK and dV 189 us (matrix cores busy 51 and 52 %); 4096 causal,
// 32 / 8 heads of 128: 230 and 314 us (51 and 44 %) and 13 us for the join.  Bound as the forward pass by issue, and at 128 by LDS, of
// which a block of 32 x 32 reads 56 operands of 1 KB for 32 products.
#include "attention.hpp"

namespace nvfp4 {
namespace {

constexpr int kRows = 64;  // rows per tile

template <int KS, int DB, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_attention_dq(const AttentionGradArgs g) {
  const AttentionArgs &a = g.f;
  constexpr int P = 4 * DB, BQ = 32 * NW, kTile = kRows * P * 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int head, slot, b, blk;
  block_of(a.Hq, a.slots * a.splits, a.causal, head, slot);
  if (a.causal) slot = a.slots * a.splits - 1 - slot;
  const int split = slot % a.splits;
  slot /= a.splits;
  find_block<BQ>(slot, a.cu_q, a.B, a.Tq, a.per_q, lane, b, blk);
  const SeqRows sq = seq_rows(a.cu_q, b, a.Tq, a.per_q), sk = seq_rows(a.cu_k, b, a.Tk, a.per_k);
  if (blk < 0 || blk * BQ >= sq.n) return;
  const int kv = head / a.group, q0 = blk * BQ + 32 * wave, query = q0 + c, ahead = sk.n - sq.n;

  const uint16_t *q = static_cast<const uint16_t *>(a.q) + sq.begin * a.ldq_t + head * a.ldq_h;
  const uint16_t *k = static_cast<const uint16_t *>(a.k) + sk.begin * a.ldk_t + kv * a.ldk_h;
  const uint16_t *v = static_cast<const uint16_t *>(a.v) + sk.begin * a.ldv_t + kv * a.ldv_h;
  const uint16_t *dout = static_cast<const uint16_t *>(g.dout) + sq.begin * g.lddo_t + head * g.lddo_h;
  const uint16_t *out = static_cast<const uint16_t *>(a.out) + sq.begin * a.ldo_t + head * a.ldo_h;
  bf16x8 Q[KS], dO[KS];
  float delta = 0.0f;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    Q[s] = load_column_operand(q, a.ldq_t, query, sq.n, s, a.D, lane);
    dO[s] = load_column_operand(dout, g.lddo_t, query, sq.n, s, a.D, lane);
    const bf16x8 o = load_column_operand(out, a.ldo_t, query, sq.n, s, a.D, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) delta = __builtin_fmaf((float)dO[s][e], (float)o[e], delta);
  }
  delta = add_halves(delta);
  const int64_t at = (int64_t)head * a.Tq + sq.begin + query;
  const float lse2 = query < sq.n ? a.lse[at] * kLog2e : 0.0f;
  if (query < sq.n && h == 0 && split == 0) {
    g.rows[at] = lse2;
    g.rows[(int64_t)a.Hq * a.Tq + at] = delta;
  }

  const int limit = a.causal ? min(query + ahead, sk.n - 1) : sk.n - 1;
  const int last_wg = a.causal ? min(min((blk + 1) * BQ, sq.n) - 1 + ahead, sk.n - 1) : sk.n - 1;
  const int last_wave = a.causal ? min(q0 + 31 + ahead, sk.n - 1) : sk.n - 1;
  const int first_limit = a.causal ? min(q0 + ahead, sk.n - 1) : sk.n - 1;
  const int all = last_wg >= 0 ? last_wg / kRows + 1 : 0;
  const int first = (int)((int64_t)all * split / a.splits), tiles = (int)((int64_t)all * (split + 1) / a.splits);
  TileLoad<P, kRows, NW> lk, lv;
  lk.init(wave, lane, a.ldk_t, a.D);
  lv.init(wave, lane, a.ldv_t, a.D);
  auto issue = [&](int t, uint8_t *to) __attribute__((always_inline)) {
    const int64_t row = (int64_t)t * kRows;
    const int left = sk.n - t * kRows;
    lk.issue(k + row * a.ldk_t, left, a.ldk_t, a.D, to, wave);
    lv.issue(v + row * a.ldv_t, left, a.ldv_t, a.D, to + kTile, wave);
  };
  const TileRead<P> read_(lane);
  const float scale2 = a.scale * kLog2e;
  f32x16 dQ[DB];

  auto pass = [&](const bool careful) __attribute__((always_inline)) {  // see k_attention
    bool again = false;
#pragma unroll
    for (int d = 0; d < DB; ++d) dQ[d] = zeros16();
    if (first < tiles) issue(first, smem);
    auto step = [&](const uint8_t *__restrict cur, uint8_t *__restrict next, int t) __attribute__((always_inline)) {
      if (t + 1 < tiles) issue(t + 1, next);
      const int key0 = t * kRows;
      if (key0 > last_wave) return;
      const TileRead<P> read = read_.here();
      const uint8_t *tk = cur, *tv = cur + kTile;
      const bool masked = key0 + kRows - 1 > first_limit;
      bool apart = masked && a.causal && tile_nonfinite<P, kRows>(tk, lane);
      if (!careful) {
        again |= apart;
        apart = false;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f32x16 S = zeros16(), dP = zeros16();
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          S = mfma(read.row_operand(tk, 32 * i, s), Q[s], S);
          dP = mfma(read.row_operand(tv, 32 * i, s), dO[s], dP);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r)
          S[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[r], scale2, -lse2)) * (dP[r] - delta);
        if (masked) {
#pragma unroll
          for (int r = 0; r < 16; ++r) S[r] = key0 + 32 * i + c_row(r, h) <= limit ? S[r] : 0.0f;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bf16x8 ds = as_operand(S, s);
          const int r0 = 32 * i + 16 * s;
          if (!careful || !apart) {
#pragma unroll
            for (int d = 0; d < DB; ++d) dQ[d] = mfma(read.column_operand(tk, r0, d), ds, dQ[d]);
          } else {
            add_rows_apart<P, DB>(tk, r0, ds, dQ, read, lane, [&](int row) { return key0 + row <= limit; });
          }
        }
      }
    };
    for (int t = first; t < tiles; ++t) {
      tile_barrier();
      step(smem + ((t - first) & 1) * 2 * kTile, smem + (~(t - first) & 1) * 2 * kTile, t);
    }
    return again;
  };
  if (__syncthreads_or(pass(false))) pass(true);
  if (query >= sq.n) return;
  if (a.splits > 1) {  // [splits][Tq][Hq][D]
    store_column_f32<DB>(dQ, a.scale, a.parts + (((int64_t)split * a.Tq + sq.begin + query) * a.Hq + head) * a.D, a.D, h);
    return;
  }
  store_column<DB>(dQ, a.scale, static_cast<uint16_t *>(g.dq) + (int64_t)(sq.begin + query) * g.lddq_t + head * g.lddq_h, a.D, h);
}

// dK and dV of a block of keys.
// KW waves of 32 keys (RS = 2: two such sets, which take a tile's 32-row halves and add their sums at the end: with 128
// values a head one workgroup's tiles fill the LDS of a CU, and its 4 waves would leave the SIMDs one each).  The steps (query heads of the group, times their tiles) of a block of keys are shared by a.splits workgroups,
// whose sums a second kernel adds.  VL: the value operands are read from LDS at every use (with 128 values a head
// they would be registers too many for two waves per SIMD).
template <int KS, int DB, int KW, int RS, bool VL>
__global__ __launch_bounds__(64 * KW * RS) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_attention_dkv(const AttentionGradArgs g) {
  const AttentionArgs &a = g.f;
  constexpr int P = 4 * DB, BK = 32 * KW, NW = KW * RS, kTile = kRows * P * 16, kStage = 2 * kTile + 512;  // and 64 floats twice: a DMA's
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  uint8_t *const tv = smem + 2 * kStage;  // VL: the block's values
  const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kw = wave % KW, rs = wave / KW;
  int kv, slot, b, blk;
  block_of(a.Hq / a.group, a.slots * g.splits, a.causal, kv, slot);
  const int split = slot % g.splits;
  find_block<BK>(slot / g.splits, a.cu_k, a.B, a.Tk, a.per_k, lane, b, blk);
  const SeqRows sq = seq_rows(a.cu_q, b, a.Tq, a.per_q), sk = seq_rows(a.cu_k, b, a.Tk, a.per_k);
  if (blk < 0 || blk * BK >= sk.n) return;
  const int k0 = blk * BK + 32 * kw, key = k0 + c, ahead = sk.n - sq.n;
  const uint16_t *k = static_cast<const uint16_t *>(a.k) + sk.begin * a.ldk_t + kv * a.ldk_h;
  const uint16_t *v = static_cast<const uint16_t *>(a.v) + sk.begin * a.ldv_t + kv * a.ldv_h;
  bf16x8 K[KS], V[VL ? 1 : KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    K[s] = load_column_operand(k, a.ldk_t, key, sk.n, s, a.D, lane);
    if constexpr (!VL) V[s] = load_column_operand(v, a.ldv_t, key, sk.n, s, a.D, lane);
  }
  if constexpr (VL) {  // the first step's barrier waits for it
    TileLoad<P, BK, NW> lv;
    lv.init(wave, lane, a.ldv_t, a.D);
    lv.issue(v + (int64_t)blk * BK * a.ldv_t, sk.n - blk * BK, a.ldv_t, a.D, tv, wave);
  }
  // the first query that attends a key j is j - ahead
  const int first_row = a.causal ? key - ahead : 0;
  const int last_first = a.causal ? k0 + 31 - ahead : 0, first_wave = a.causal ? max(k0 - ahead, 0) : 0;
  const int first_tile = (a.causal ? max(blk * BK - ahead, 0) : 0) / kRows, tiles = (sq.n + kRows - 1) / kRows;
  const int per_head = max(tiles - first_tile, 0), steps = per_head * a.group;
  const int begin = (int)((int64_t)steps * split / g.splits), end = (int)((int64_t)steps * (split + 1) / g.splits);

  TileLoad<P, kRows, NW> lq, lo;
  lq.init(wave, lane, a.ldq_t, a.D);
  lo.init(wave, lane, g.lddo_t, a.D);
  int ih, it;  // the next step to load: head of the group, tile
  auto issue = [&](uint8_t *to) __attribute__((always_inline)) {
    const int head = kv * a.group + ih;
    const int64_t row = sq.begin + (int64_t)it * kRows;
    const int left = sq.n - it * kRows;
    lq.issue(static_cast<const uint16_t *>(a.q) + row * a.ldq_t + head * a.ldq_h, left, a.ldq_t, a.D, to, wave);
    lo.issue(static_cast<const uint16_t *>(g.dout) + row * g.lddo_t + head * g.lddo_h, left, g.lddo_t, a.D, to + kTile, wave);
    if (wave < 2) {  // the rows' log sums, and their sums of dO O
      const float *rows = g.rows + ((int64_t)wave * a.Hq + head) * a.Tq + row;
      buffer_dma4(rows, left > 0 ? 4 * min(left, kRows) : 0, to + 2 * kTile + 256 * wave, 4 * lane);
    }
    if (++it == tiles) {
      it = first_tile;
      ++ih;
    }
  };
  const TileRead<P> read_(lane);
  const float scale2 = a.scale * kLog2e;
  f32x16 dK[DB], dV[DB];
  auto pass = [&](const bool careful) __attribute__((always_inline)) {  // see k_attention
    bool again = false;
    ih = per_head > 0 ? begin / per_head : 0;
    it = first_tile + begin - ih * per_head;
    int t = it;
#pragma unroll
    for (int d = 0; d < DB; ++d) dK[d] = dV[d] = zeros16();
    if (begin < end) issue(smem);
    auto step = [&](const uint8_t *__restrict cur, uint8_t *__restrict next, int i) __attribute__((always_inline)) {
      if (i + 1 < end) issue(next);
      const TileRead<P> read = read_.here();
      const uint8_t *tq = cur, *to = cur + kTile;
      const float *rows = reinterpret_cast<const float *>(tq + 2 * kTile);
      const int tile0 = t * kRows;
      t = t + 1 == tiles ? first_tile : t + 1;
      const bool cut = tile0 < last_first, masked = cut || (careful && tile0 + kRows > sq.n);
      if (tile0 + kRows - 1 < first_wave) return;
      bool apart = cut && (tile_nonfinite<P, kRows>(tq, lane) || tile_nonfinite<P, kRows>(to, lane));
      if (!careful) {
        again |= apart;
        apart = false;
      }
#pragma unroll 1
      for (int j = 0; j < 2 / RS; ++j) {
        const int i0 = 32 * (RS == 2 ? rs : j);
        const int row0 = tile0 + i0;
        f32x16 S = zeros16(), dP = zeros16();
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          S = mfma(read.row_operand(tq, i0, s), K[s], S);
          if constexpr (VL) dP = mfma(read.row_operand(to, i0, s), read.row_operand(tv, 32 * kw, s), dP);
          else dP = mfma(read.row_operand(to, i0, s), V[s], dP);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const f32x4 lse2 = *reinterpret_cast<const f32x4 *>(rows + i0 + 8 * u + 4 * h);
          const f32x4 delta = *reinterpret_cast<const f32x4 *>(rows + 64 + i0 + 8 * u + 4 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            S[4 * u + e] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[4 * u + e], scale2, -lse2[e]));
            dP[4 * u + e] = S[4 * u + e] * (dP[4 * u + e] - delta[e]);
          }
        }
        if (masked) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const bool in = row0 + c_row(r, h) >= first_row && (!careful || row0 + c_row(r, h) < sq.n);
            S[r] = in ? S[r] : 0.0f;
            dP[r] = in ? dP[r] : 0.0f;
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bf16x8 p = as_operand(S, s), ds = as_operand(dP, s);
          const int r0 = i0 + 16 * s;
          if (!careful || !apart) {
#pragma unroll
            for (int d = 0; d < DB; ++d) {
              dV[d] = mfma(read.column_operand(to, r0, d), p, dV[d]);
              dK[d] = mfma(read.column_operand(tq, r0, d), ds, dK[d]);
            }
          } else {
            add_rows_apart<P, DB>(to, r0, p, dV, read, lane, [&](int row) { return tile0 + row >= first_row; });
            add_rows_apart<P, DB>(tq, r0, ds, dK, read, lane, [&](int row) { return tile0 + row >= first_row; });
          }
        }
      }
    };
    for (int i = begin; i < end; ++i) {
      tile_barrier();
      step(smem + ((i - begin) & 1) * kStage, smem + (~(i - begin) & 1) * kStage, i);
    }
    // Rows past the last query are zeros, and their products too, but not with an infinity of a key: all of its sums are NaN
    // then, and the careful pass masks these rows (always masked: 129, 64, 1, 500 queries over 1600 keys 1 us more).
    if (!careful) again |= dV[0][0] != dV[0][0];
    return again;
  };
  if (__syncthreads_or(pass(false))) pass(true);
  if constexpr (VL) wait_vmem();  // the values', where there was no step to wait for them
  if constexpr (RS == 2) {
    f32x4 *const part = reinterpret_cast<f32x4 *>(smem) + kw * (DB * 4 * 64) + lane;
    auto join = [&](f32x16(&x)[DB]) __attribute__((always_inline)) {
      __syncthreads();
      if (rs == 1) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int u = 0; u < 4; ++u) part[(4 * d + u) * 64] = f32x4{x[d][4 * u], x[d][4 * u + 1], x[d][4 * u + 2], x[d][4 * u + 3]};
      }
      __syncthreads();
      if (rs == 0) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const f32x4 o = part[(4 * d + u) * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[d][4 * u + e] += o[e];
          }
      }
    };
    join(dK);
    join(dV);
    if (rs == 1) return;
  }
  if (key >= sk.n) return;
  const int64_t row = sk.begin + key;
  if (g.splits == 1) {
    store_column<DB>(dK, a.scale, static_cast<uint16_t *>(g.dk) + row * g.lddk_t + kv * g.lddk_h, a.D, h);
    store_column<DB>(dV, 1.0f, static_cast<uint16_t *>(g.dv) + row * g.lddv_t + kv * g.lddv_h, a.D, h);
  } else {  // [splits][dK, dV][Tk][Hkv][D]
    const int Hkv = a.Hq / a.group;
    const int64_t each = (int64_t)a.Tk * Hkv * a.D;
    float *to = a.parts + 2 * split * each + (row * Hkv + kv) * a.D;
    store_column_f32<DB>(dK, a.scale, to, a.D, h);
    store_column_f32<DB>(dV, 1.0f, to + each, a.D, h);
  }
}

// Adds fp32 parts [splits][outputs][T][H][D] in order: a thread has 4 values of output blockIdx.y.
struct GradJoin {
  const float *parts;
  int splits, T, D, B;
  const int32_t *cu;
  void *out[2];
  int64_t ld_t[2], ld_h[2];
  FastDiv per_row, heads;
};
__global__ __launch_bounds__(kJoinThreads) void k_gradient_join(const GradJoin g) {
  const uint32_t i = blockIdx.x * (uint32_t)kJoinThreads + threadIdx.x, j = blockIdx.y;
  const uint32_t r = fastdiv(i, g.per_row), at = 4 * (i - r * g.per_row.d), t = fastdiv(r, g.heads), head = r - t * g.heads.d;
  if (!holds(joined_rows(g.cu, g.B, g.T), t)) return;
  const int64_t each = (int64_t)g.T * g.heads.d * g.D;
  const float *from = g.parts + j * each + (int64_t)r * g.D + at;
  f32x4 sum = {0, 0, 0, 0};
  for (int s = 0; s < g.splits; ++s) {
    const f32x4 x = *reinterpret_cast<const f32x4 *>(from + gridDim.y * s * each);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += x[e];
  }
  const bf16x2 lo = {(__bf16)sum[0], (__bf16)sum[1]}, hi = {(__bf16)sum[2], (__bf16)sum[3]};
  *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(g.out[j]) + t * g.ld_t[j] + head * g.ld_h[j] + at) =
      u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}
void join(const GradJoin &g, int outputs, hipStream_t stream) {
  const int64_t threads = (int64_t)g.T * g.heads.d * (g.D / 4);  // few: the splits are for small problems
  k_gradient_join<<<dim3((unsigned)((threads + kJoinThreads - 1) / kJoinThreads), (unsigned)outputs), dim3(kJoinThreads), 0, stream>>>(g);
}

constexpr int kKeyWaves = 4;

template <int KS, int DB>
hipError_t launch(AttentionGradArgs g, hipStream_t stream) {
  constexpr int NW = 4, KW = kKeyWaves;
  constexpr bool VL = DB >= 3;
  constexpr int kTile = kRows * DB * 64, kLdsQ = 4 * kTile;
  constexpr int RS = DB == 4 ? 2 : 1;
  constexpr int kLdsK = 2 * (2 * kTile + 512) + (VL ? 32 * KW * DB * 64 : 0);
  static_assert(RS == 1 || KW * DB * 4096 <= kLdsK, "the sums pass through the tiles' memory");
  static std::atomic<bool> done_q[kMaxDevices], done_k[kMaxDevices];
  const int Hkv = g.f.Hq / g.f.group;
  const FastDiv per_row = make_fastdiv((uint32_t)(g.f.D / 4));
  if (g.f.Tq > 0) {
    const void *kern = reinterpret_cast<const void *>(&k_attention_dq<KS, DB, NW>);
    if (hipError_t e = set_dynamic_lds(kern, kLdsQ, done_q); e != hipSuccess) return e;
    g.f.slots = (int)attention_slots(g.f.Tq, g.f.B, g.f.cu_q != nullptr, 32 * NW);
    k_attention_dq<KS, DB, NW><<<dim3((unsigned)(g.f.slots * g.f.Hq * g.f.splits)), dim3(64 * NW), kLdsQ, stream>>>(g);
    if (g.f.splits > 1)
      join({g.f.parts, g.f.splits, g.f.Tq, g.f.D, g.f.B, g.f.cu_q, {g.dq, nullptr}, {g.lddq_t, 0}, {g.lddq_h, 0}, per_row,
            make_fastdiv((uint32_t)g.f.Hq)}, 1, stream);
  }
  if (g.f.Tk > 0) {
    const void *kern = reinterpret_cast<const void *>(&k_attention_dkv<KS, DB, KW, RS, VL>);
    if (hipError_t e = set_dynamic_lds(kern, kLdsK, done_k); e != hipSuccess) return e;
    g.f.slots = (int)attention_slots(g.f.Tk, g.f.B, g.f.cu_k != nullptr, 32 * KW);
    k_attention_dkv<KS, DB, KW, RS, VL><<<dim3((unsigned)(g.f.slots * Hkv * g.splits)), dim3(64 * KW * RS), kLdsK, stream>>>(g);
    if (g.splits > 1)
      join({g.f.parts, g.splits, g.f.Tk, g.f.D, g.f.B, g.f.cu_k, {g.dk, g.dv}, {g.lddk_t, g.lddv_t}, {g.lddk_h, g.lddv_h}, per_row,
            make_fastdiv((uint32_t)Hkv)}, 2, stream);
  }
  return hipGetLastError();
}

}  // namespace

// Workgroups for two rounds of 256 CUs, but none with less than about 4 steps (4096 causal, 8 key heads of 128: 256 workgroups
// of very different lengths alone, 512 halves 341 us with the join; 4 key heads of 64, 1600 keys: 49 us alone, 40 shared).
// Of several sequences the longest is taken for twice the average, it is waited for: queries 129, 64, 1, 500 over 1600 keys, 12 /
// 4 heads of 64, the whole backward 60 us against 69; eight of 1 and one of 1000 81 and 109; two equal ones of 512 45 and 42.
int attention_backward_splits(int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t B) {
  const int64_t blocks = (Tk / (32 * kKeyWaves) + B) * Hkv, want = (512 + blocks - 1) / blocks;
  const int64_t steps = ((B > 1 ? 2 * Tq : Tq) / (B > 0 ? B : 1) / kRows + 1) * (Hq / Hkv), most = steps / 4 > 1 ? steps / 4 : 1;
  return (int)(want < most ? want : most);
}

hipError_t launch_attention_backward(const AttentionGradArgs &g, hipStream_t stream) {
  const int D = g.f.D;
  if (D <= 32) return launch<2, 1>(g, stream);
  if (D <= 64) return launch<4, 2>(g, stream);
  if (D <= 80) return launch<5, 3>(g, stream);
  if (D <= 96) return launch<6, 3>(g, stream);
  if (D <= 112) return launch<7, 4>(g, stream);
  return launch<8, 4>(g, stream);
}

}  // namespace nvfp4
