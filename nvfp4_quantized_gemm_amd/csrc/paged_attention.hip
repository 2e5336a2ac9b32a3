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

// A thread takes 8 values of a row (a token's head); blockIdx.y: keys, values.  MX8: the 4 threads of a block
// of 32 find its scale together; blocks past D are zeros.
template <bool MX8>
__global__ __launch_bounds__(256) void k_cache_append(const CacheAppendArgs a) {
  const PagedCacheArgs &c = a.c;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t row = fastdiv(i, a.per_row), piece = i - row * a.per_row.d;
  const uint32_t t = fastdiv(row, a.heads), head = row - t * a.heads.d;
  if (t >= (uint32_t)a.T) return;
  int b = (int)t;
  int64_t behind = 1;  // tokens of the sequence from this one on
  if (a.cu) {
    int lo = 0, hi = c.B;  // the last b with cu[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= (int)t) lo = mid;
      else hi = mid;
    }
    b = lo;
    behind = (int64_t)a.cu[b + 1] - t;
    if (behind <= 0) return;
  }
  const int64_t pos = c.lengths[b] - behind;
  if (pos < 0 || (pos >> c.page_shift) >= c.max_pages) return;
  const int page = c.table[b * c.ld_table + (pos >> c.page_shift)];
  if (page < 0 || page >= c.pages) return;
  const bool values = blockIdx.y != 0;
  const uint16_t *src = values ? static_cast<const uint16_t *>(a.v) + t * a.ldv_t + head * a.ldv_h
                               : static_cast<const uint16_t *>(a.k) + t * a.ldk_t + head * a.ldk_h;
  const int64_t at = (((int64_t)page * c.Hkv + head) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
  const bool inside = piece < (uint32_t)c.D / 8;
  u32x4 w = {0, 0, 0, 0};
  if (inside) w = load16<false>(src + 8 * piece);
  if constexpr (!MX8) {
    store16<false>(static_cast<uint16_t *>(values ? c.v : c.k) + at * c.D + 8 * piece, w);
  } else {
    float f[8];
    SegIn<1>::unpack(w, f);
    const uint32_t x = mx8_scale_byte(mx8_amax_bits(f));
    if (inside) *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(values ? c.v : c.k) + at * c.D + 8 * piece) = mx8_encode8(f, x);
    if ((piece & 3) == 0) (values ? c.vs : c.ks)[at * ((c.D + 31) / 32) + piece / 4] = (uint8_t)x;
  }
}

// ---- one new token --------------------------------------------------------------------------------------

constexpr int kTileKeys = 32, kWaves = 4, kStep = kTileKeys * kWaves;

// The 8 values of a piece as bf16: codes times their scale (exact, as in the W4A8 product).
__device__ __forceinline__ u32x4 widen_piece(const u32x2 &codes, uint32_t x) {
  // The conversion reads the scale's exponent: 2^0 stands for 2^-127 (E8M0's least) and NaN for 255.
  const float X = __uint_as_float(x << 23);
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.x, X, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.x, X, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.y, X, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.y, X, true);
  return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
}

// A sequence's keys are split over up to `splits` workgroups, evenly by its own length, in whole steps of 128
// keys; this workgroup's first key and the one past its last.
__device__ __forceinline__ int split_keys(int len, int splits) {  // keys per workgroup
  const int steps = (len + kStep - 1) / kStep;
  return (steps + splits - 1) / splits * kStep;
}

// A workgroup has a key head of a sequence, 32 of its query heads as columns, and a run of keys, of which each
// wave takes every fourth 32.  A wave brings a tile from its pages to registers while the one before
// multiplies, and from there to its own part of LDS, without barriers; MXFP8 is widened on that way.
template <int KS, int DB, bool MX8>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_paged_attention(const PagedAttentionArgs a) {
  constexpr int P = 4 * DB, kN = kTileKeys * P / 64, kTile = kTileKeys * P * 16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kWaves * 2 * kTile];
  __shared__ float tops[kWaves][32], totals[kWaves][32];
  const PagedCacheArgs &c = a.c;
  const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x, kv = blockIdx.y % c.Hkv, first = blockIdx.y / c.Hkv * 32, b = blockIdx.z;
  const int len = (int)min((int64_t)max(c.lengths[b], 0), (int64_t)c.max_pages << c.page_shift);
  const int run = split_keys(len, a.splits), lo = split * run, hi = min(lo + run, len);
  if (lo >= len && split > 0) return;
  const int heads = min(a.group - first, 32), head = kv * a.group + first + col;

  const uint16_t *q = static_cast<const uint16_t *>(a.q) + b * a.ldq_t;
  bf16x8 Q[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int d = 16 * s + 8 * h;
    u32x4 w = {0, 0, 0, 0};
    if (col < heads && d < c.D) w = *reinterpret_cast<const u32x4 *>(q + head * a.ldq_h + d);
    Q[s] = __builtin_bit_cast(bf16x8, w);
  }

  uint8_t *const tk = smem + wave * 2 * kTile, *const tv = tk + kTile;
  const int32_t *table = c.table + b * c.ld_table;
  constexpr int ES = MX8 ? 1 : 2;
  const int nb = (c.D + 31) / 32, mask = (1 << c.page_shift) - 1;
  uint32_t off[kN], soff[kN];  // of this lane's pieces, in bytes, rows counted from a half of the tile
  int row[kN], place[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int n = 64 * i + lane, r = n / P, p = n - r * P;
    row[i] = r;
    place[i] = r * (P * 16) + ((p ^ swizzle<P>(r)) << 4);
    off[i] = p < c.D / 8 ? (uint32_t)((r & 15) * c.D + 8 * p) * ES : kOutside;
    soff[i] = p < c.D / 8 ? (uint32_t)((r & 15) * nb + p / 4) : kOutside;
  }
  u32x4 wk[kN], wv[kN];
  uint32_t xk[kN], xv[kN];
  bool ok[2] = {false, false}, next_ok[2] = {false, false};
  // Half i < kN / 2 of a tile's pieces are its first 16 rows, the others the last 16: one page each.
  auto load = [&](int key0) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int pos = key0 + 16 * half;
      const int page = pos < hi ? __builtin_amdgcn_readfirstlane(table[pos >> c.page_shift]) : -1;
      next_ok[half] = page >= 0 && page < c.pages;
      const int64_t at = next_ok[half] ? (((int64_t)page * c.Hkv + kv) << c.page_shift) + (pos & mask) : 0;
      const int left = next_ok[half] ? hi - pos : 0;
      const __amdgpu_buffer_rsrc_t bk = byte_buffer(static_cast<const uint8_t *>(c.k) + at * c.D * ES, 0x7fffffffu),
                                   bv = byte_buffer(static_cast<const uint8_t *>(c.v) + at * c.D * ES, 0x7fffffffu);
#pragma unroll
      for (int i = half * kN / 2; i < (half + 1) * kN / 2; ++i) {
        const uint32_t o = (row[i] & 15) < left ? off[i] : kOutside;
        if constexpr (!MX8) {
          wk[i] = __builtin_amdgcn_raw_buffer_load_b128(bk, o, 0, 0);
          wv[i] = __builtin_amdgcn_raw_buffer_load_b128(bv, o, 0, 0);
        } else {
          const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(bk, o, 0, 0), v = __builtin_amdgcn_raw_buffer_load_b64(bv, o, 0, 0);
          wk[i] = u32x4{u.x, u.y, 0, 0};
          wv[i] = u32x4{v.x, v.y, 0, 0};
        }
      }
      if constexpr (MX8) {
        const __amdgpu_buffer_rsrc_t sk = byte_buffer(c.ks + at * nb, 0x7fffffffu), sv = byte_buffer(c.vs + at * nb, 0x7fffffffu);
#pragma unroll
        for (int i = half * kN / 2; i < (half + 1) * kN / 2; ++i) {
          const uint32_t o = (row[i] & 15) < left ? soff[i] : kOutside;
          xk[i] = __builtin_amdgcn_raw_buffer_load_b8(sk, o, 0, 0);
          xv[i] = __builtin_amdgcn_raw_buffer_load_b8(sv, o, 0, 0);
        }
      }
    }
  };
  auto put = [&]() {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      *reinterpret_cast<u32x4 *>(tk + place[i]) = MX8 ? widen_piece(u32x2{wk[i].x, wk[i].y}, xk[i]) : wk[i];
      *reinterpret_cast<u32x4 *>(tv + place[i]) = MX8 ? widen_piece(u32x2{wv[i].x, wv[i].y}, xv[i]) : wv[i];
    }
    ok[0] = next_ok[0];
    ok[1] = next_ok[1];
  };

  const TileRead<P> read(lane);
  const float scale2 = a.scale * kLog2e;
  float top = -INFINITY, total = 0.0f;
  f32x16 O[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) O[d] = zeros16();
  const int start = lo + wave * kTileKeys;
  if (start < hi) load(start);
  for (int key0 = start; key0 < hi; key0 += kStep) {
    put();
    if (key0 + kStep < hi) load(key0 + kStep);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    f32x16 S = zeros16();
#pragma unroll
    for (int s = 0; s < KS; ++s) S = mfma(read.row_operand(tk, 0, s), Q[s], S);
    if (key0 + kTileKeys > hi || !ok[0] || !ok[1]) {
#pragma unroll
      for (int r = 0; r < 16; ++r) S[r] = key0 + c_row(r, h) < hi && ok[r >> 3] ? S[r] : -INFINITY;
    }
    float m = S[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) m = fmaxf(m, S[r]);
    m = max_halves(m);
    const bool rise = (m - top) * scale2 > 8.0f;  // see k_attention
    if (__ballot(rise)) {
      const float old = !rise ? 1.0f : top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((top - m) * scale2);
      top = rise ? m : top;
      total *= old;
#pragma unroll
      for (int d = 0; d < DB; ++d) O[d] *= old;
    }
    const float shift = top == -INFINITY ? 0.0f : top * scale2;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      S[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[r], scale2, -shift));
      total += S[r];
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bf16x8 p = as_operand(S, s);
#pragma unroll
      for (int d = 0; d < DB; ++d) O[d] = mfma(read.column_operand(tv, 16 * s, d), p, O[d]);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  // The waves' sums meet in LDS, each as [32 columns][32 DB values] in its wave's part.
  total = add_halves(total);
  if (h == 0) {
    tops[wave][col] = top;
    totals[wave][col] = total;
  }
  constexpr int kW = 32 * DB;  // a column's values; piece p of column c lies in place p ^ (c & 7)
  float *const part = reinterpret_cast<float *>(tk);
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<f32x4 *>(part + col * kW + 4 * ((8 * d + 2 * g + h) ^ (col & 7))) =
          f32x4{O[d][4 * g], O[d][4 * g + 1], O[d][4 * g + 2], O[d][4 * g + 3]};
  __syncthreads();
  for (int i = threadIdx.x; i < heads * (kW / 4); i += 64 * kWaves) {
    const int cc = i / (kW / 4), p = i - cc * (kW / 4);
    if (4 * p >= c.D) continue;
    float t = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) t = fmaxf(t, tops[w][cc]);
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = tops[w][cc] == -INFINITY && !(totals[w][cc] != totals[w][cc]) ? 0.0f : __builtin_amdgcn_exp2f((tops[w][cc] - t) * scale2);
      const f32x4 x = *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(smem + w * 2 * kTile) + cc * kW + 4 * (p ^ (cc & 7)));
      sum += totals[w][cc] * f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += x[e] * f;
    }
    const int64_t who = (int64_t)b * a.Hq + kv * a.group + first + cc;
    if (a.splits == 1) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const bf16x2 x = {(__bf16)(o[0] * inv), (__bf16)(o[1] * inv)}, y = {(__bf16)(o[2] * inv), (__bf16)(o[3] * inv)};
      *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + b * a.ldo_t + (kv * a.group + first + cc) * a.ldo_h + 4 * p) =
          u32x2{__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)};
    } else {
      float *const to = a.partial + (who * a.splits + split) * c.D;
      *reinterpret_cast<f32x4 *>(to + 4 * p) = o;
      if (p == 0) {
        float *const st = a.partial + (int64_t)c.B * a.Hq * a.splits * c.D + 2 * (who * a.splits + split);
        st[0] = t;
        st[1] = sum;
      }
    }
  }
}

// One workgroup per query head of a sequence: its splits' sums, weighted by their maxima, in order.
__global__ __launch_bounds__(256) void k_paged_join(const PagedAttentionArgs a) {
  const PagedCacheArgs &c = a.c;
  const int head = blockIdx.x, b = blockIdx.y;
  const int len = (int)min((int64_t)max(c.lengths[b], 0), (int64_t)c.max_pages << c.page_shift);
  const int run = split_keys(len, a.splits), n = run > 0 ? (len + run - 1) / run : 0;
  const int64_t who = (int64_t)b * a.Hq + head;
  const float *const part = a.partial + who * a.splits * c.D;
  const float *const st = a.partial + (int64_t)c.B * a.Hq * a.splits * c.D + 2 * who * a.splits;
  const float scale2 = a.scale * kLog2e;
  __shared__ float sums[8][32][5];
  // 32 lanes hold the D values, 4 each; 8 such groups take every eighth split
  const int p = threadIdx.x & 31, g = threadIdx.x >> 5;
  float top = -INFINITY;
  for (int s = 0; s < n; ++s) top = fmaxf(top, st[2 * s]);
  f32x4 o = {0, 0, 0, 0};
  float sum = 0.0f;
  for (int s = g; s < n; s += 8) {
    const float t = st[2 * s], l = st[2 * s + 1];
    const float f = t == -INFINITY && l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f((t - top) * scale2);
    sum += l * f;
    if (4 * p < c.D) {
      const f32x4 x = *reinterpret_cast<const f32x4 *>(part + (int64_t)s * c.D + 4 * p);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += x[e] * f;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sums[g][p][e] = o[e];
  sums[g][p][4] = sum;
  __syncthreads();
  if (g != 0 || 4 * p >= c.D) return;
  float r[5] = {0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 5; ++e) r[e] += sums[i][p][e];
  const float inv = r[4] == 0.0f ? 0.0f : 1.0f / r[4];
  const bf16x2 x = {(__bf16)(r[0] * inv), (__bf16)(r[1] * inv)}, y = {(__bf16)(r[2] * inv), (__bf16)(r[3] * inv)};
  *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + b * a.ldo_t + head * a.ldo_h + 4 * p) =
      u32x2{__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)};
}

template <int KS, int DB>
void launch(const PagedAttentionArgs &a, const dim3 &grid, hipStream_t stream) {
  if (a.c.ks) k_paged_attention<KS, DB, true><<<grid, dim3(64 * kWaves), 0, stream>>>(a);
  else k_paged_attention<KS, DB, false><<<grid, dim3(64 * kWaves), 0, stream>>>(a);
}

}  // namespace

hipError_t launch_cache_append(CacheAppendArgs a, hipStream_t stream) {
  const int per_row = a.c.ks ? (a.c.D + 31) / 32 * 4 : a.c.D / 8;
  a.per_row = make_fastdiv((uint32_t)per_row);
  a.heads = make_fastdiv((uint32_t)a.c.Hkv);
  const int64_t threads = (int64_t)a.T * a.c.Hkv * per_row;  // below 2^31, the call checked
  const dim3 grid((unsigned)((threads + 255) / 256), 2);
  if (a.c.ks) k_cache_append<true><<<grid, dim3(256), 0, stream>>>(a);
  else k_cache_append<false><<<grid, dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

// Workgroups for about 4 on each of 256 CUs (two at a time), but none with less than a step of keys.
int paged_attention_splits(int64_t B, int64_t Hq, int64_t Hkv, int64_t capacity) {
  const int64_t blocks = B * Hkv * ((Hq / Hkv + 31) / 32), most = (capacity + kStep - 1) / kStep;
  const int64_t want = (1024 + blocks - 1) / blocks;
  return (int)(want < most ? want : most > 1 ? most : 1);
}

hipError_t launch_paged_attention(const PagedAttentionArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)a.splits, (unsigned)(a.c.Hkv * ((a.group + 31) / 32)), (unsigned)a.c.B);
  const int D = a.c.D;
  if (D <= 32) launch<2, 1>(a, grid, stream);
  else if (D <= 64) launch<4, 2>(a, grid, stream);
  else if (D <= 80) launch<5, 3>(a, grid, stream);
  else if (D <= 96) launch<6, 3>(a, grid, stream);
  else if (D <= 112) launch<7, 4>(a, grid, stream);
  else launch<8, 4>(a, grid, stream);
  if (a.splits > 1) k_paged_join<<<dim3((unsigned)a.Hq, (unsigned)a.c.B), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
