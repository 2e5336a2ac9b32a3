// A paged cache of keys and values, in bf16 or MXFP8: writing new tokens into it, and the attention of one new
// token per sequence over it (gfx950).
//
// Cache: [pages][Hkv][page][D], so that a head's rows of a page are one run of memory.  Pages hold 2^s >= 16
// tokens; sequence b's token t lies in page table[b][t >> s].  Entries outside [0, pages) hold no tokens.
#include "attention.hpp"
#include "mx8.hpp"

namespace nvfp4 {
namespace {

// ---- append -------------------------------------------------------------------------------------------

// A thread takes 8 values of a row (a token's head), of the key and of the value.  Rows go by 16 tokens of a head, which lie
// side by side in the cache.  MX8: the 4 threads of a block of 32 find its scale together; blocks past D are zeros.
// Three loads follow one another before a row's place is known: the values are on their way meanwhile.  Two prompts of 8192,
// 8 heads of 128, into MXFP8: 25 us (4.1 TB/s; 28 with the heads of a token side by side); 64 tokens into bf16 2.7 us.
template <bool MX8>
__global__ __launch_bounds__(256) void k_cache_append(const CacheAppendArgs a) {
  const PagedCacheArgs &c = a.c;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t row = fastdiv(i, a.per_row), piece = i - row * a.per_row.d;
  const uint32_t group = row >> 4, block = fastdiv(group, a.heads), head = group - block * a.heads.d, t = 16 * block + (row & 15);
  if (t >= (uint32_t)a.T) return;
  const bool inside = piece < (uint32_t)c.D / 8;
  u32x4 w[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  if (inside) {
    w[0] = load16<true>(static_cast<const uint16_t *>(a.k) + t * a.ldk_t + head * a.ldk_h + 8 * piece);
    w[1] = load16<true>(static_cast<const uint16_t *>(a.v) + t * a.ldv_t + head * a.ldv_h + 8 * piece);
  }
  const TokenPlace place = token_place(a.cu, c.lengths, c.B, (int)t);
  const int page = page_of(c.table + place.b * c.ld_table, place.pos, c.page_shift, c.max_pages, c.pages);
  if (page < 0) return;
  const int64_t at = cache_row(page, (int)head, c.Hkv, place.pos, c.page_shift);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    void *const to = j ? c.v : c.k;
    if constexpr (!MX8) {
      store16<false>(static_cast<uint16_t *>(to) + at * c.D + 8 * piece, w[j]);
    } else {
      float f[8];
      SegIn<1>::unpack(w[j], f);
      const uint32_t x = mx8_scale_byte(mx8_amax_bits(f));
      if (inside) *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(to) + at * c.D + 8 * piece) = mx8_encode8(f, x);
      if ((piece & 3) == 0) (j ? c.vs : c.ks)[at * ((c.D + 31) / 32) + piece / 4] = (uint8_t)x;
    }
  }
}

// ---- one new token --------------------------------------------------------------------------------------
//
// Products are v_mfma_f32_16x16x32_bf16: C[16][16] += A[16][32] B[32][16].  Lane l = 16 g + c holds row (of A) or
// column (of B) c and k = 8 g .. 8 g + 7, and of C column c, rows 4 g .. 4 g + 3.  With query heads as columns and 32
// keys as two C's, a lane's 8 scores are its B operand over the k order key(g, e) = 16 (e / 4) + 4 g + e % 4.

constexpr int kTileKeys = 32, kWaves = 4, kStep = kTileKeys * kWaves, kMaxSplits = 256;

__device__ __forceinline__ f32x4 mfma16(const bf16x8 &a, const bf16x8 &b, const f32x4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// Over the four lanes that share a column.
__device__ __forceinline__ float max_quarters(float v) {
  const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max_halves(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)));
}
__device__ __forceinline__ float add_quarters(float v) {
  const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return add_halves(__uint_as_float(r.x) + __uint_as_float(r.y));
}

// Piece p of row r of a tile lies in place p ^ swizzle16(r): 16 rows' same piece, and 8 rows' same 32 bytes, pass over
// all banks.
template <int P>
__device__ __forceinline__ int swizzle16(int r) {
  if constexpr (P == 16) return ((r & 7) << 1) | ((r >> 3) & 1);
  else if constexpr (P == 8) return (((r >> 1) & 3) << 1) | ((r >> 3) & 1);
  else return (((r >> 2) & 1) << 1) | ((r >> 3) & 1);
}
// A operand: rows r0 .. r0 + 15, values 32 s .. 32 s + 31.
template <int P>
__device__ __forceinline__ bf16x8 rows16(const uint8_t *tile, int r0, int s, int lane) {
  const int r = lane & 15, p = (4 * s + (lane >> 4)) ^ swizzle16<P>(r);
  return *reinterpret_cast<const bf16x8 *>(tile + (r0 + r) * (P * 16) + (p << 4));
}
// A operand of the transposed tile: values 16 d .. 16 d + 15, keys in the order above.
template <int P>
__device__ __forceinline__ bf16x8 columns16(const uint8_t *tile, int d, int lane) {
  const int i = lane & 15, r = 4 * (lane >> 4) + (i >> 2), p = (2 * d + ((i >> 1) & 1)) ^ swizzle16<P>(r);
  const uint8_t *at = tile + r * (P * 16) + (p << 4) + 8 * (i & 1);  // rows r and r + 16 are swizzled alike
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(at + 16 * (P * 16)));
  return __builtin_bit_cast(bf16x8, s16x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
}

// The 8 values of a piece as bf16: codes times their scale (exact down to bf16's least number, 2^-133).  The conversion reads the
// scale's exponent: 0 stands for 2^-127 (E8M0's least), 255 for NaN.
__device__ __forceinline__ u32x4 widen_piece(const u32x2 &codes, uint32_t x) {
  const float X = __uint_as_float(x << 23);
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.x, X, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.x, X, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.y, X, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.y, X, true);
  return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
}

// A sequence's keys are split over up to `splits` workgroups, evenly by its own length, in whole steps of 128
// keys: keys per workgroup.
__device__ __forceinline__ int split_keys(int len, int splits) {
  const int steps = (len + kStep - 1) / kStep;
  return (steps + splits - 1) / splits * kStep;
}
// What a lane brings of a tile, kN runs of W values (W = 8: 16 bytes of bf16, 8 of MXFP8; W = 16: 16 bytes of MXFP8,
// half the loads, where D is whole 16 values and a half of the tile whole loads): offsets in the cache, from the first
// row of their half, of the scales, and places in LDS.
template <int P, bool MX8, int W>
struct Pieces {
  static constexpr int kRun = W / 8, kRow = P / kRun, kN = kTileKeys * kRow / 64;
  static_assert(kN % 2 == 0, "halves of the tile in whole loads");
  uint32_t off[kN], soff[MX8 ? kN : 1], place[kN];
  __device__ __forceinline__ void find(int lane, int D, int nb) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int n = 64 * i + lane, r = P == 12 ? n / kRow : i * (64 / kRow) + lane / kRow;
      const int p = kRun * (P == 12 ? n - r * kRow : lane % kRow);
      place[i] = r * (P * 16) + ((p ^ swizzle16<P>(r)) << 4);
      off[i] = p < D / 8 ? (uint32_t)((r & 15) * D + 8 * p) * (MX8 ? 1 : 2) : kOutside;
      if constexpr (MX8) soff[i] = p < D / 8 ? (uint32_t)((r & 15) * nb + p / 4) : kOutside;
    }
  }
};

// A wave's next tile of keys or of values on its way through registers.  Half of a lane's pieces belong to the
// tile's first 16 rows, the others to the last 16: one page each.
template <int P, bool MX8, int W>
struct TileInFlight {
  using At = Pieces<P, MX8, W>;
  static constexpr int kN = At::kN;
  u32x4 w[MX8 && W == 8 ? 1 : kN];
  u32x2 codes[MX8 && W == 8 ? kN : 1];
  uint32_t scale[MX8 ? kN : 1];
  // `left` rows from row `at` of the cache on, for the pieces of half `half`
  __device__ __forceinline__ void load(int half, const void *cache, const uint8_t *scales, int64_t at, int left, int D, int nb,
                                       const At &x) {
    const uint32_t n = left > 16 ? 16 : left > 0 ? left : 0;
    const auto rows = byte_buffer(static_cast<const uint8_t *>(cache) + at * D * (MX8 ? 1 : 2), n * D * (MX8 ? 1 : 2));
    const auto bytes = byte_buffer(scales + (MX8 ? at * nb : 0), MX8 ? n * nb : 0);
#pragma unroll
    for (int i = half * kN / 2; i < (half + 1) * kN / 2; ++i) {
      if constexpr (MX8 && W == 8) codes[i] = __builtin_amdgcn_raw_buffer_load_b64(rows, x.off[i], 0, 0);
      else w[i] = __builtin_amdgcn_raw_buffer_load_b128(rows, x.off[i], 0, 0);
      if constexpr (MX8) scale[i] = __builtin_amdgcn_raw_buffer_load_b8(bytes, x.soff[i], 0, 0);
    }
  }
  __device__ __forceinline__ void put(uint8_t *tile, const At &x) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      u32x4 *const to = reinterpret_cast<u32x4 *>(tile + x.place[i]);
      if constexpr (!MX8) {
        *to = w[i];
      } else if constexpr (W == 8) {
        *to = widen_piece(codes[i], scale[i]);
      } else {
        *to = widen_piece(u32x2{w[i].x, w[i].y}, scale[i]);
        *reinterpret_cast<u32x4 *>(tile + (x.place[i] ^ 16)) = widen_piece(u32x2{w[i].z, w[i].w}, scale[i]);
      }
    }
  }
};

// A workgroup has a key head of a sequence, 16 NC of its query heads as columns, and a run of keys, of which each
// wave takes every fourth 32.  A wave brings a tile from its pages to registers while the one before multiplies, and
// from there to its own part of LDS (keys first, then values in their place), without barriers; MXFP8 is widened on
// that way.  Few registers and little LDS, so that 3 waves per SIMD keep loads in flight.
// Bound by memory in bf16: two sequences of 131072, 8 heads of 128, 134 us (5.5 of the 6.1 TB/s that a large reduction reads;
// with 32 columns and 2 waves 132); in MXFP8 by issue and LDS beside it: 64 sequences to 8192 119 us (4.7 TB/s; 166 with 32
// columns, 130 with 8 bytes a load).
template <int DB, bool MX8, int W, int NC>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(NC == 2 ? 2 : 3))) void k_paged_attention(
    const PagedAttentionArgs a) {
  constexpr int P = 4 * DB, kTile = kTileKeys * P * 16, kPart = kTile * NC;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kWaves * kPart];
  __shared__ float tops[kWaves][16 * NC], totals[kWaves][16 * NC];
  const PagedCacheArgs &c = a.c;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x, kv = blockIdx.y % c.Hkv, first = blockIdx.y / c.Hkv * (16 * NC), b = blockIdx.z;
  const int len = tokens_of(c.lengths[b], c.page_shift, c.max_pages), run = split_keys(len, a.splits), lo = split * run, hi = min(lo + run, len);
  if (lo >= len && split > 0) return;
  const int heads = min(a.group - first, 16 * NC);

  const int32_t *table = c.table + b * c.ld_table;
  const int nb = (c.D + 31) / 32;
  uint8_t *const tile = smem + wave * kPart;
  Pieces<P, MX8, W> pieces;
  pieces.find(lane, c.D, nb);
  // where the two halves of a tile lie, and how many keys each has there (0: none, or no page)
  struct Where {
    int64_t at[2];
    int left[2];
  };
  auto find = [&](int key0) {
    Where w;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int pos = key0 + 16 * half;
      const int page = pos < hi ? __builtin_amdgcn_readfirstlane(page_of(table, pos, c.page_shift, c.max_pages, c.pages)) : -1;
      w.at[half] = page >= 0 ? cache_row(page, kv, c.Hkv, pos, c.page_shift) : 0;
      w.left[half] = page >= 0 ? min(hi - pos, 16) : 0;
    }
    return w;
  };
  TileInFlight<P, MX8, W> keys, values;
  auto load = [&](TileInFlight<P, MX8, W> &t, const void *cache, const uint8_t *scales, const Where &w) __attribute__((always_inline)) {
    t.load(0, cache, scales, w.at[0], w.left[0], c.D, nb, pieces);
    t.load(1, cache, scales, w.at[1], w.left[1], c.D, nb, pieces);
  };
  const int start = lo + wave * kTileKeys;
  Where now = find(start);
  load(keys, c.k, c.ks, now);
  load(values, c.v, c.vs, now);

  const uint16_t *q = static_cast<const uint16_t *>(a.q) + b * a.ldq_t;
  bf16x8 Q[NC][DB];
#pragma unroll
  for (int n = 0; n < NC; ++n)
#pragma unroll
    for (int s = 0; s < DB; ++s) {
      const int h = 16 * n + col, d = 32 * s + 8 * g;
      u32x4 w = {0, 0, 0, 0};
      if (h < heads && d < c.D) w = *reinterpret_cast<const u32x4 *>(q + (kv * a.group + first + h) * a.ldq_h + d);
      Q[n][s] = __builtin_bit_cast(bf16x8, w);
    }
  const float scale2 = a.scale * kLog2e;
  bool some = false;  // whether this wave met a token
  float top[NC], total[NC];
  f32x4 O[NC][2 * DB];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    top[n] = -INFINITY;
    total[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < 2 * DB; ++d) O[n][d] = f32x4{0, 0, 0, 0};
  }

  for (int key0 = start; key0 < hi; key0 += kStep) {
    const Where next = find(key0 + kStep);
    if constexpr (P != 12) {  // a few instructions here instead of registers kept around the loop
      int l = lane;
      asm volatile("" : "+v"(l));
      pieces.find(l, c.D, nb);
    }
    keys.put(tile, pieces);
    load(keys, c.k, c.ks, next);
    asm volatile("" ::: "memory");
    f32x4 S[NC][2];
#pragma unroll
    for (int n = 0; n < NC; ++n) S[n][0] = S[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < DB; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bf16x8 A = rows16<P>(tile, 16 * i, s, lane);
#pragma unroll
        for (int n = 0; n < NC; ++n) S[n][i] = mfma16(A, Q[n][s], S[n][i]);
      }
    asm volatile("" ::: "memory");
    values.put(tile, pieces);
    load(values, c.v, c.vs, next);
    asm volatile("" ::: "memory");
    some |= (now.left[0] | now.left[1]) > 0;
    bf16x8 p[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      if (now.left[0] < 16 || now.left[1] < 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[n][i][e] = 4 * g + e < now.left[i] ? S[n][i][e] : -INFINITY;
      }
      float m = fmaxf(S[n][0][0], S[n][1][0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) m = fmaxf(fmaxf(m, S[n][0][e]), S[n][1][e]);
      m = max_quarters(m);
      const bool rise = (m - top[n]) * scale2 > 8.0f;  // see k_attention
      if (__ballot(rise)) {
        const float old = !rise ? 1.0f : top[n] == -INFINITY ? 0.0f : joined_weight(top[n], m, scale2);
        top[n] = rise ? m : top[n];
        total[n] *= old;
#pragma unroll
        for (int d = 0; d < 2 * DB; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[n][d][e] *= old;
      }
      const float shift = top[n] == -INFINITY ? 0.0f : top[n] * scale2;
      const bool far = fabsf(shift) > kFar;
      if (__builtin_expect(__ballot(far) != 0, 0)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[n][i][e] = exponent(S[n][i][e], scale2, top[n], shift, far);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[n][i][e] = exponent(S[n][i][e], scale2, top[n], shift, false);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = __builtin_amdgcn_exp2f(S[n][i][e]);
          total[n] += x;
          p[n][4 * i + e] = (__bf16)x;
        }
    }
#pragma unroll
    for (int d = 0; d < 2 * DB; ++d) {
      const bf16x8 A = columns16<P>(tile, d, lane);
#pragma unroll
      for (int n = 0; n < NC; ++n) O[n][d] = mfma16(A, p[n], O[n][d]);
    }
    asm volatile("" ::: "memory");
    now = next;
  }

  // The waves' sums meet in LDS, each as [16 NC columns][32 DB values] in its wave's part, column c's piece of 4 values
  // p in place p ^ (c & 7).
  constexpr int kW = 32 * DB;
  float *const part = reinterpret_cast<float *>(tile);
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int h = 16 * n + col;
    total[n] = add_quarters(total[n]);
    if (g == 0) {
      tops[wave][h] = some ? fmaxf(top[n], kLowest) : -INFINITY;
      totals[wave][h] = total[n];
    }
#pragma unroll
    for (int d = 0; d < 2 * DB; ++d) *reinterpret_cast<f32x4 *>(part + h * kW + 4 * ((4 * d + g) ^ (h & 7))) = O[n][d];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < heads * (kW / 4); i += 64 * kWaves) {
    const int h = i / (kW / 4), p = i - h * (kW / 4);
    if (4 * p >= c.D) continue;
    float t = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) t = fmaxf(t, tops[w][h]);
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float l = totals[w][h], f = l == 0.0f ? 0.0f : joined_weight(tops[w][h], t, scale2);
      const f32x4 x = *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(smem + w * kPart) + h * kW + 4 * (p ^ (h & 7)));
      sum += l * f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += x[e] * f;
    }
    const int head = kv * a.group + first + h;
    const int64_t who = (int64_t)b * a.Hq + head;
    if (a.splits == 1) {
      const float inv = sum == 0.0f && t == -INFINITY ? 0.0f : 1.0f / sum;  // no tokens: 0; scores all -inf: 0 / 0
      const bf16x2 x = {(__bf16)(o[0] * inv), (__bf16)(o[1] * inv)}, y = {(__bf16)(o[2] * inv), (__bf16)(o[3] * inv)};
      *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + b * a.ldo_t + head * a.ldo_h + 4 * p) =
          u32x2{__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)};
    } else {
      *reinterpret_cast<f32x4 *>(a.partial + (who * a.splits + split) * c.D + 4 * p) = o;
      if (p == 0) {
        float *const st = a.partial + (int64_t)c.B * a.Hq * a.splits * c.D + 2 * (who * a.splits + split);
        st[0] = t;
        st[1] = sum;
      }
    }
  }
}

// One workgroup per query head of a sequence: its splits' sums, weighted by their maxima, in a fixed order.
__global__ __launch_bounds__(256) void k_paged_join(const PagedAttentionArgs a) {
  const PagedCacheArgs &c = a.c;
  const int head = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int len = tokens_of(c.lengths[b], c.page_shift, c.max_pages), run = split_keys(len, a.splits), n = run > 0 ? (len + run - 1) / run : 0;
  const int64_t who = (int64_t)b * a.Hq + head;
  const float *const part = a.partial + who * a.splits * c.D;
  const float *const st = a.partial + (int64_t)c.B * a.Hq * a.splits * c.D + 2 * who * a.splits;
  const float scale2 = a.scale * kLog2e;
  __shared__ float weights[kMaxSplits], tops[4], sums[8][32][5];
  static_assert(kMaxSplits <= 256, "a thread per split");
  float t = -INFINITY, l = 0.0f;
  if ((int)threadIdx.x < n) {
    t = st[2 * threadIdx.x];
    l = st[2 * threadIdx.x + 1];
  }
  float top = t;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  const float f = l == 0.0f ? 0.0f : joined_weight(t, top, scale2);
  weights[threadIdx.x] = f;
  l *= f;
  __syncthreads();
  // 32 lanes hold the D values, 4 each; 8 such groups take every eighth split
  const int p = threadIdx.x & 31, g = threadIdx.x >> 5;
  f32x4 o = {0, 0, 0, 0};
  if (4 * p < c.D) {
#pragma unroll 4
    for (int s = g; s < n; s += 8) {
      const f32x4 x = *reinterpret_cast<const f32x4 *>(part + (int64_t)s * c.D + 4 * p);
      const float w = weights[s];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += x[e] * w;
    }
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) l += __shfl_xor(l, x);
  __syncthreads();
  if (lane == 0) tops[wave] = l;
#pragma unroll
  for (int e = 0; e < 4; ++e) sums[g][p][e] = o[e];
  __syncthreads();
  if (g != 0 || 4 * p >= c.D) return;
  const float sum = (tops[0] + tops[1]) + (tops[2] + tops[3]), inv = sum == 0.0f && top == -INFINITY ? 0.0f : 1.0f / sum;
  float r[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] += sums[i][p][e];
  const bf16x2 x = {(__bf16)(r[0] * inv), (__bf16)(r[1] * inv)}, y = {(__bf16)(r[2] * inv), (__bf16)(r[3] * inv)};
  *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + b * a.ldo_t + head * a.ldo_h + 4 * p) =
      u32x2{__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)};
}

// query heads per workgroup
int columns_of(int64_t group) { return group <= 16 ? 16 : 32; }

template <int DB, bool MX8, int W>
void launch(const PagedAttentionArgs &a, const dim3 &grid, hipStream_t stream) {
  if (a.group <= 16) k_paged_attention<DB, MX8, W, 1><<<grid, dim3(64 * kWaves), 0, stream>>>(a);
  else k_paged_attention<DB, MX8, W, 2><<<grid, dim3(64 * kWaves), 0, stream>>>(a);
}
template <int DB>
void launch_kind(const PagedAttentionArgs &a, const dim3 &grid, hipStream_t stream) {
  constexpr int kWide = DB == 2 || DB == 4 ? 16 : 8;
  if (!a.c.ks) launch<DB, false, 8>(a, grid, stream);
  else if (a.c.D % kWide == 0) launch<DB, true, kWide>(a, grid, stream);
  else launch<DB, true, 8>(a, grid, stream);
}

}  // namespace

hipError_t launch_cache_append(CacheAppendArgs a, hipStream_t stream) {
  const int per_row = a.c.ks ? (a.c.D + 31) / 32 * 4 : a.c.D / 8;
  a.per_row = make_fastdiv((uint32_t)per_row);
  a.heads = make_fastdiv((uint32_t)a.c.Hkv);
  const int64_t threads = ((int64_t)a.T + 15) / 16 * 16 * a.c.Hkv * per_row;  // below 2^32, the call checked
  const dim3 grid((unsigned)((threads + 255) / 256));
  if (a.c.ks) k_cache_append<true><<<grid, dim3(256), 0, stream>>>(a);
  else k_cache_append<false><<<grid, dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

// Workgroups for about 6 on each of 256 CUs (64 sequences of all lengths to 8192, MXFP8: 4 a CU 121 us, 8 116 us; two of
// 131072, bf16: 134, 136), but none with less than a step of keys.
// Short sequences are not split: a second launch costs what four steps take.
int paged_attention_splits(int64_t B, int64_t Hq, int64_t Hkv, int64_t capacity) {
  if (capacity <= 4 * kStep) return 1;
  const int64_t group = Hq / Hkv, blocks = B * Hkv * ((group + columns_of(group) - 1) / columns_of(group));
  int64_t n = (1536 + blocks - 1) / blocks;
  n = n < kMaxSplits ? n : kMaxSplits;
  const int64_t most = (capacity + kStep - 1) / kStep;
  return (int)(n < most ? n : most);
}

hipError_t launch_paged_attention(const PagedAttentionArgs &a, hipStream_t stream) {
  const int columns = columns_of(a.group);
  const dim3 grid((unsigned)a.splits, (unsigned)(a.c.Hkv * ((a.group + columns - 1) / columns)), (unsigned)a.c.B);
  const int D = a.c.D;
  if (D <= 32) launch_kind<1>(a, grid, stream);
  else if (D <= 64) launch_kind<2>(a, grid, stream);
  else if (D <= 96) launch_kind<3>(a, grid, stream);
  else launch_kind<4>(a, grid, stream);
  if (a.splits > 1) k_paged_join<<<dim3((unsigned)a.Hq, (unsigned)a.c.B), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
