// Softmax attention of whole prompts and images (gfx950):
//   O[i] = sum_j softmax_j(scale q_i k_j) v_j,   lse[i] = log sum_j exp(scale q_i k_j)
// over packed sequences, with query heads that share key heads, causal (aligned at the ends) or not.
//
// A wave has 32 queries as the columns of its products, so that a query's softmax is a lane's (and its
// partner's in the other half): S^T = K Q^T gives a lane 16 of 32 keys of its query, the exponentials are
// rounded to bf16 where they are and multiply as they lie, O^T += V^T P^T, and the running maximum and sum
// are one register each.  Keys and values pass through LDS in tiles of 64, two in turn; V^T is read from
// its rows by the transposing LDS read.
//
// Measured: 4096 tokens, 16 heads of 72: 103 us (750 TFLOP/s); 8192 causal, 32 / 8 heads of 128: 528 us (1.04 PFLOP/s).  Bound by
// issue: the products of one wave of a SIMD hide little of the other's vector instructions (each product costs these about 23
// of its 32 clocks), so that their times add up: of the prompt's 1.00 M cycles products are 0.53, vector instructions about 0.45.
#include "attention.hpp"

namespace nvfp4 {
namespace {

constexpr int kKeys = 64;  // keys per tile

// KS: 16-value steps of a head in S; DB: 32-value blocks in O; NW waves of 32 queries.
template <int KS, int DB, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_attention(const AttentionArgs a) {
  constexpr int P = 4 * DB, BQ = 32 * NW;
  constexpr int kTile = kKeys * P * 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  int head, slot;
  block_of(a.Hq, a.slots * a.splits, a.causal, head, slot);
  if (a.causal) slot = a.slots * a.splits - 1 - slot;
  const int split = slot % a.splits;
  slot /= a.splits;
  int b, blk;
  find_block<BQ>(slot, a.cu_q, a.B, a.Tq, a.per_q, lane, b, blk);
  const SeqRows sq = seq_rows(a.cu_q, b, a.Tq, a.per_q), sk = seq_rows(a.cu_k, b, a.Tk, a.per_k);
  if (blk < 0 || blk * BQ >= sq.n) return;
  const int kv = head / a.group, q0 = blk * BQ + 32 * wave, query = q0 + c, ahead = sk.n - sq.n;

  const uint16_t *q = static_cast<const uint16_t *>(a.q) + sq.begin * a.ldq_t + head * a.ldq_h;
  const uint16_t *k = static_cast<const uint16_t *>(a.k) + sk.begin * a.ldk_t + kv * a.ldk_h;
  const uint16_t *v = static_cast<const uint16_t *>(a.v) + sk.begin * a.ldv_t + kv * a.ldv_h;
  bf16x8 Q[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) Q[s] = load_column_operand(q, a.ldq_t, query, sq.n, s, a.D, lane);

  // keys 0 .. limit of this lane's query; the workgroup's tiles, and this wave's
  const int limit = a.causal ? min(query + ahead, sk.n - 1) : sk.n - 1;
  const int last_wg = a.causal ? min(min((blk + 1) * BQ, sq.n) - 1 + ahead, sk.n - 1) : sk.n - 1;
  const int last_wave = a.causal ? min(q0 + 31 + ahead, sk.n - 1) : sk.n - 1;
  const int first_limit = a.causal ? min(q0 + ahead, sk.n - 1) : sk.n - 1;
  const int all = last_wg >= 0 ? last_wg / kKeys + 1 : 0;
  const int first = (int)((int64_t)all * split / a.splits), tiles = (int)((int64_t)all * (split + 1) / a.splits);

  TileLoad<P, kKeys, NW> lk, lv;
  lk.init(wave, lane, a.ldk_t, a.D);
  lv.init(wave, lane, a.ldv_t, a.D);
  auto issue = [&](int t, uint8_t *at) __attribute__((always_inline)) {
    const int64_t row = (int64_t)t * kKeys;
    const int left = sk.n - t * kKeys;
    lk.issue(k + row * a.ldk_t, left, a.ldk_t, a.D, at, wave);
    lv.issue(v + row * a.ldv_t, left, a.ldv_t, a.D, at + kTile, wave);
  };

  const TileRead<P> read_(lane);
  const float scale2 = a.scale * kLog2e;  // exp(scale s) = 2^(scale2 s)
  float top, total;  // running maximum of s (both halves of a column), sum (this lane's)
  f32x16 O[DB];

  // A pass over the keys; the careful one, which keeps infinities and NaN from queries that do not attend
  // them, only where a masked tile holds some (as a branch inside one loop it took 40 registers from it), or where
  // a maximum is far.
  auto pass = [&](const bool careful) __attribute__((always_inline)) {
    bool again = false;
    top = -INFINITY;
    total = 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d) O[d] = zeros16();
    if (first < tiles) issue(first, smem);
    auto step = [&](const uint8_t *__restrict cur, uint8_t *__restrict next, int t) __attribute__((always_inline)) {
      if (t + 1 < tiles) issue(t + 1, next);
      const int key0 = t * kKeys;
      if (key0 > last_wave) return;
      const TileRead<P> read = read_.here();
      const uint8_t *tk = cur, *tv = cur + kTile;

      f32x16 S[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        S[i] = zeros16();
#pragma unroll
        for (int s = 0; s < KS; ++s) S[i] = mfma(read.row_operand(tk, 32 * i, s), Q[s], S[i]);
      }
      const bool masked = key0 + kKeys - 1 > first_limit;
      if (masked) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) S[i][r] = key0 + 32 * i + c_row(r, h) <= limit ? S[i][r] : -INFINITY;
      }
      float m = S[0][0];
#pragma unroll
      for (int r = 1; r < 16; ++r) m = fmaxf(m, S[0][r]);
#pragma unroll
      for (int r = 0; r < 16; ++r) m = fmaxf(m, S[1][r]);
      m = max_halves(m);
      // The sums are kept relative to a maximum that may lag by 2^8: they cannot overflow, and are as exact.
      // Only the queries that need it move theirs, so that a query's bits do not depend on its neighbours (where workgroups
      // share keys, they depend on where the keys are cut: on the call's sizes and the block's last query).
      const bool rise = (m - top) * scale2 > 8.0f;
      if (__ballot(rise)) {
        const float old = !rise ? 1.0f : top == -INFINITY ? 0.0f : joined_weight(top, m, scale2);
        top = rise ? m : top;
        if (!careful) again |= rise && fabsf(top * scale2) > kFar;
        total *= old;
#pragma unroll
        for (int d = 0; d < DB; ++d) O[d] *= old;
      }
      const float shift = top == -INFINITY ? 0.0f : top * scale2;
      const bool far = careful && fabsf(shift) > kFar;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          S[i][r] = __builtin_amdgcn_exp2f(exponent(S[i][r], scale2, top, shift, far));
          total += S[i][r];
        }
      bool apart = masked && a.causal && tile_nonfinite<P, kKeys>(tv, lane);
      if (!careful) {
        again |= apart;
        apart = false;
      }
      // rounding the exponentials to bf16 is what the matrix instruction takes: 2^-9 of each, averaged out
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bf16x8 p = as_operand(S[i], s);
          const int r0 = 32 * i + 16 * s;
          if (!careful || !apart) {
#pragma unroll
            for (int d = 0; d < DB; ++d) O[d] = mfma(read.column_operand(tv, r0, d), p, O[d]);
          } else {
            add_rows_apart<P, DB>(tv, r0, p, O, read, lane, [&](int row) { return key0 + row <= limit; });
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

  total = add_halves(total);
  if (query >= sq.n) return;
  const int64_t row = sq.begin + query;
  // A query without keys gives 0.  One whose scores are all -inf has no weights either, and gives 0 / 0.
  const bool none = limit < 0;
  if (a.splits > 1) {  // [splits][Tq][Hq][D] sums relative to top, then [splits][Tq][Hq] (top, sum of weights); top -inf: none
    const int64_t each = (int64_t)a.Tq * a.Hq, at = split * each + row * a.Hq + head;
    store_column_f32<DB>(O, 1.0f, a.parts + at * a.D, a.D, h);
    if (h == 0) reinterpret_cast<f32x2 *>(a.parts + a.splits * each * a.D)[at] = f32x2{none ? -INFINITY : fmaxf(top, kLowest), total};
    return;
  }
  const float inv = none ? 0.0f : 1.0f / total;
  store_column<DB>(O, inv, static_cast<uint16_t *>(a.out) + row * a.ldo_t + head * a.ldo_h, a.D, h);
  if (a.lse && h == 0)
    a.lse[(int64_t)head * a.Tq + row] = none ? -INFINITY : (top * scale2 + __builtin_amdgcn_logf(total)) * kLn2;
}

// Joins the splits in order: a thread has 4 values of a query's head.
__global__ __launch_bounds__(kJoinThreads) void k_attention_join(const AttentionArgs a, const FastDiv per_row, const FastDiv heads) {
  const uint32_t i = blockIdx.x * (uint32_t)kJoinThreads + threadIdx.x, r = fastdiv(i, per_row), d = 4 * (i - r * per_row.d);
  const uint32_t t = fastdiv(r, heads), head = r - t * heads.d;
  if (!holds(joined_rows(a.cu_q, a.B, a.Tq), t)) return;
  const int64_t each = (int64_t)a.Tq * a.Hq;
  const f32x2 *const st = reinterpret_cast<const f32x2 *>(a.parts + a.splits * each * a.D) + r;
  const float scale2 = a.scale * kLog2e;
  float top = -INFINITY, total = 0.0f;
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, st[s * each].x);
  f32x4 o = {0, 0, 0, 0};
  for (int s = 0; s < a.splits; ++s) {
    const f32x2 x = st[s * each];
    const float f = x.y == 0.0f ? 0.0f : joined_weight(x.x, top, scale2);
    const f32x4 v = *reinterpret_cast<const f32x4 *>(a.parts + (s * each + r) * a.D + d);
    total += x.y * f;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += v[e] * f;
  }
  const bool none = total == 0.0f && top == -INFINITY;
  const float inv = none ? 0.0f : 1.0f / total;
  const bf16x2 lo = {(__bf16)(o[0] * inv), (__bf16)(o[1] * inv)}, hi = {(__bf16)(o[2] * inv), (__bf16)(o[3] * inv)};
  *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + t * a.ldo_t + head * a.ldo_h + d) =
      u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
  if (a.lse && d == 0)
    a.lse[(int64_t)head * a.Tq + t] = none ? -INFINITY : (top * scale2 + __builtin_amdgcn_logf(total)) * kLn2;
}

constexpr int kWaves = 4;

template <int KS, int DB>
hipError_t launch(AttentionArgs a, hipStream_t stream) {
  constexpr int kLds = 4 * kKeys * DB * 64;
  static std::atomic<bool> done[kMaxDevices];
  const void *kern = reinterpret_cast<const void *>(&k_attention<KS, DB, kWaves>);
  if (hipError_t e = set_dynamic_lds(kern, kLds, done); e != hipSuccess) return e;
  a.slots = (int)attention_slots(a.Tq, a.B, a.cu_q != nullptr, 32 * kWaves);
  k_attention<KS, DB, kWaves><<<dim3((unsigned)(a.slots * a.Hq * a.splits)), dim3(64 * kWaves), kLds, stream>>>(a);
  if (a.splits > 1) {
    const int64_t threads = (int64_t)a.Tq * a.Hq * (a.D / 4);  // few: the splits are for small problems
    k_attention_join<<<dim3((unsigned)((threads + kJoinThreads - 1) / kJoinThreads)), dim3(kJoinThreads), 0, stream>>>(
        a, make_fastdiv((uint32_t)(a.D / 4)), make_fastdiv((uint32_t)a.Hq));
  }
  return hipGetLastError();
}

}  // namespace

// Workgroups that share a block of queries' keys: for one on each of 256 CUs, none with less than four tiles (256 keys).
// Alone a workgroup takes 0.95 us a tile: 17 queries x 32 heads over 4096 keys 77 us, shared by 8 22 us; 926 x 4 heads over
// 1933 36 and 21; but 1024 x 16 heads, 144 workgroups, 23 us, and 26 shared by 3: their fp32 sums go through memory.
int attention_splits(int64_t Tq, int64_t Tk, int64_t Hq, int64_t B) {
  const int64_t blocks = (Tq / (32 * kWaves) + B) * Hq, want = 256 / (blocks > 0 ? blocks : 1);
  const int64_t most = Tk / (B > 0 ? B : 1) / (4 * kKeys), n = want < most ? want : most;
  return (int)(n < 1 ? 1 : n < 32 ? n : 32);
}

hipError_t launch_attention(const AttentionArgs &a, hipStream_t stream) {
  if (a.D <= 32) return launch<2, 1>(a, stream);
  if (a.D <= 64) return launch<4, 2>(a, stream);
  if (a.D <= 80) return launch<5, 3>(a, stream);
  if (a.D <= 96) return launch<6, 3>(a, stream);
  if (a.D <= 112) return launch<7, 4>(a, stream);
  return launch<8, 4>(a, stream);
}

}  // namespace nvfp4
