// What the attention kernels share (gfx950): sequences, tiles of head rows in LDS, matrix operands.
//
// All products are v_mfma_f32_32x32x16_bf16: C[32][32] += A[32][16] B[16][32].  Lane l = 32 h + c holds
//   A   row c,     k = 8 h .. 8 h + 7        B   column c,  k = 8 h .. 8 h + 7
//   C   column c,  rows 8 g + 4 h + i        (register 4 g + i; g, i = 0 .. 3)
// So a lane's C registers 8 s .. 8 s + 7 are 8 rows of its column, and rounded to bf16 they are a B operand
// over the k order  kappa(s, h, e) = 16 s + 8 (e / 4) + 4 h + e % 4:  the result of one product is the
// operand of the next without a move between lanes, as long as its A operand lists k in the same order.
#pragma once
#include "launch.hpp"
#include "sequence_index.hpp"

namespace nvfp4 {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A maximum of scores that are all -inf, where -inf itself says that there is no score.
constexpr float kLowest = -3.402823466e38f;
// Exponents are scale2 s - shift in one instruction, with shift the rounded product of scale2 and the maximum: all weights of a
// query share the factor 2^(what was rounded), which leaves them when they are normed.  From this shift on (where the rounding is
// 2^-4 at most) they are (s - maximum) scale2, or that factor would leave fp32 from a shift of 2^31 on.
constexpr float kFar = 1048576.0f;
__device__ __forceinline__ float exponent(float s, float scale2, float top, float shift, bool far) {
  return far ? (s - top) * scale2 : __builtin_fmaf(s, scale2, -shift);
}
// The weight of sums relative to maximum t beside those relative to top: by the shifts that they were summed with, whose
// roundings differ (by the maxima themselves it was off by 2^-5 at shifts of 2^19).
__device__ __forceinline__ float joined_weight(float t, float top, float scale2) {
  const float a = t * scale2, b = top * scale2;
  return __builtin_amdgcn_exp2f(fabsf(a) > kFar || fabsf(b) > kFar ? (t - top) * scale2 : a - b);
}

// ---- sequences ----------------------------------------------------------------------------------------

// The sequence of a slot, and which of its blocks that is (none of them where blk is negative or past its end).
template <int BLK>
__device__ __forceinline__ void find_block(int slot, const int32_t *cu, int B, int T, int per, int lane, int &b, int &blk) {
  if (!cu) {
    const int each = (per + BLK - 1) / BLK;
    b = slot / each;
    blk = slot - b * each;
    return;
  }
  int lo = 0, len = B;  // the last b with cu[b] / BLK + b <= slot: 64 candidates at a time
  while (len > 1) {
    const int step = (len + 63) >> 6, at = lane * step;
    const bool here = at < len && first_slot(cu, lo + min(at, len - 1), T, BLK) <= slot;
    const int n = max((int)__popcll(__ballot(here)), 1);
    lo += (n - 1) * step;
    len = min(step, len - (n - 1) * step);
  }
  b = __builtin_amdgcn_readfirstlane(lo);
  blk = slot - first_slot(cu, b, T, BLK);
}

// Rows that sequences hold, for a kernel of kJoinThreads threads that joins what several workgroups summed: no row else was
// computed, and the workspace holds anything there.  None where the offsets descend: which rows have blocks is not known
// then.  (Calls whose sums are joined have at most 512 sequences, see attention_splits and attention_backward_splits.)
constexpr int kJoinThreads = 256;
__device__ __forceinline__ SeqRows joined_rows(const int32_t *cu, int B, int T) {
  if (cu) {
    bool down = false;
    for (int b = threadIdx.x; b < B; b += kJoinThreads) down |= descends(cu, b, T);
    if (__syncthreads_or(down)) return {0, 0};
  }
  const int begin = rows_before(cu, T);
  return {begin, rows_in_use(cu, B, T) - begin};
}
__device__ __forceinline__ bool holds(const SeqRows &s, uint32_t row) { return row - (uint32_t)s.begin < (uint32_t)s.n; }

// Which block of which head: neighbouring workgroups lie on different XCDs, so where the heads divide evenly
// each XCD takes its own, and all blocks that read a key head's rows share an L2.  slots_first: block by block
// over the heads, else head by head.  (Causal calls go from the last slot on: of one sequence
// the blocks with many tiles go first; of several, the last sequence does, whatever its length.)
__device__ __forceinline__ void block_of(int heads, int slots, bool slots_first, int &head, int &slot) {
  const bool own = heads % 8 == 0;
  const int w = blockIdx.x, per = own ? heads / 8 : heads, i = own ? w >> 3 : w, x = own ? (w & 7) * per : 0;
  if (slots_first) {
    slot = i / per;
    head = x + i % per;
  } else {
    head = x + i / slots;
    slot = i % slots;
  }
}

// This wave's loads have landed and its reads of LDS are back, and every other wave's too.
__device__ __forceinline__ void tile_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---- tiles of head rows in LDS ------------------------------------------------------------------------
//
// A tile is ROWS rows of P 16-byte pieces, P = 4 DB (DB blocks of 32 values).  Piece p of row r lies in
// place p ^ swizzle(r), so that both ways of reading it pass over all banks:
//   by row       32 lanes the same piece of 32 rows (16 bytes each)
//   transposed   16 lanes 4 rows of 32 bytes, two such groups side by side
// P = 16: rows are 256 bytes, and r's low two bits have to move 64 bytes.  P = 8: rows 2 i and 2 i + 1
// share 256 bytes.  P = 4, 12: four rows begin at four different 64 bytes already.
template <int P>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (P == 16) return ((r & 3) << 2) | ((r >> 2) & 3);
  else if constexpr (P == 8) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  else return (r >> 2) & 3;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t byte_buffer(const void *base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (int)bytes, 0x00027000);
}
// 16 bytes a lane from `bytes` bytes at base to LDS: lane i's to lds + 16 i; zeros past the end.
__device__ __forceinline__ void buffer_dma16(const void *base, uint32_t bytes, uint8_t *lds, uint32_t lane_off, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(byte_buffer(base, bytes), (lds_void_t *)lds, 16, lane_off, off, 0, 0);
}
__device__ __forceinline__ void buffer_dma4(const void *base, uint32_t bytes, uint8_t *lds, uint32_t lane_off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(byte_buffer(base, bytes), (lds_void_t *)lds, 4, lane_off, 0, 0, 0);
}
constexpr uint32_t kOutside = 0x80000000u;  // an offset past every buffer: loads give zeros

// This lane's part of loading a tile: wave-wide 16-byte LDS-DMAs, number j filling the places 64 j .. 64 j + 63.
// A wave's DMAs are kN of them, chosen so that what a lane loads repeats (every kPeriod of them, further down).
template <int P, int ROWS, int NW>
struct TileLoad {
  static constexpr int kAll = ROWS * P / 64, kBytes = ROWS * P * 16;
  static constexpr bool kThree = P == 12;  // 3 DMAs are 16 rows
  static constexpr int kUnit = kThree ? 3 : 1, kUnits = kAll / kUnit, kN = (kUnits + NW - 1) / NW;
  static constexpr int kUnitRows = 64 * kUnit / P;
  static_assert(kUnits * kUnit == kAll && (kThree || P == 4 || NW * kUnitRows % 16 == 0), "the swizzle repeats");
  uint32_t off[kUnit], step;
  __device__ __forceinline__ void init(int wave, int lane, int64_t ld, int D) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      const int n = 64 * i + lane, r = wave * kUnitRows + n / P, p = (n - n / P * P) ^ swizzle<P>(r);
      off[i] = p < D / 8 ? (uint32_t)r * (uint32_t)ld * 2u + 16u * p : kOutside;
    }
    step = NW * kUnitRows * (uint32_t)ld * 2u;
  }
  // The first `left` rows from base on; what lies past their last value is loaded as zeros (pitch >= D).
  __device__ __forceinline__ void issue(const uint16_t *base, int left, int64_t ld, int D, uint8_t *lds, int wave) const {
    const uint32_t bytes = left > 0 ? (uint32_t)(min(left, ROWS) - 1) * (uint32_t)ld * 2u + 2u * D : 0u;
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      if (kUnits % NW != 0 && wave + NW * u >= kUnits) break;
#pragma unroll
      for (int i = 0; i < kUnit; ++i)
        buffer_dma16(base, bytes, lds + 1024 * (kUnit * (wave + NW * u) + i), off[i], u * step);
    }
  }
};

// Where this lane reads a tile, so that the places of other steps, blocks and rows are an exclusive or with a
// constant and the instruction's offset.
template <int P>
struct TileRead {
  static constexpr bool kXor = P == 8 || P == 16;
  uint32_t rows, columns;
  __device__ __forceinline__ explicit TileRead(int lane) {
    const int r = lane & 31, h = lane >> 5, i = lane & 15, k = 4 * h + (i >> 2);
    rows = r * (P * 16) + ((h ^ swizzle<P>(r)) << 4);
    columns = k * (P * 16) + (((2 * ((lane >> 4) & 1) + ((i >> 1) & 1)) ^ swizzle<P>(k)) << 4) + 8 * (i & 1);
  }
  // The same, for use inside a loop: the places of its reads are computed there (one instruction each) instead of
  // being kept in registers around it.
  __device__ __forceinline__ TileRead here() const {
    TileRead r = *this;
    asm volatile("" : "+v"(r.rows), "+v"(r.columns));
    return r;
  }
  // A operand: rows r0 .. r0 + 31 (r0 a multiple of 16), values 16 s .. 16 s + 15.
  __device__ __forceinline__ bf16x8 row_operand(const uint8_t *tile, int r0, int s) const {
    const uint32_t at = kXor ? rows ^ (s << 5) : (rows ^ ((s & 1) << 5)) + ((s >> 1) << 6);
    return *reinterpret_cast<const bf16x8 *>(tile + at + r0 * (P * 16));
  }
  // A operand of the transposed tile: rows are values 32 d .. 32 d + 31, k rows r0 + kappa(0, h, 0 .. 7) (r0 a
  // multiple of 16).  Each of the two reads turns 4 rows of 16 values per 16 lanes.
  __device__ __forceinline__ bf16x8 column_operand(const uint8_t *tile, int r0, int d) const {
    const uint32_t at = kXor ? columns ^ (d << 6) : columns + (d << 6);
    const uint8_t *p = tile + at + r0 * (P * 16), *q = tile + (at ^ 32) + (r0 + 8) * (P * 16);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p), b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)q);
    return __builtin_bit_cast(bf16x8, s16x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
  }
};

// B operand from global memory: column c is row c of [n][ld], zeros past row n - 1 and past D.
__device__ __forceinline__ bf16x8 load_column_operand(const uint16_t *base, int64_t ld, int row, int n, int s, int D,
                                                      int lane) {
  const int d = 16 * s + 8 * (lane >> 5);
  u32x4 w = {0, 0, 0, 0};
  if (row < n && d < D) w = *reinterpret_cast<const u32x4 *>(base + (int64_t)row * ld + d);
  return __builtin_bit_cast(bf16x8, w);
}

__device__ __forceinline__ f32x16 mfma(const bf16x8 &a, const bf16x8 &b, const f32x16 &c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zeros16() { return f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0}; }

// C registers 8 s .. 8 s + 7 as a B operand, rounded to bf16.
__device__ __forceinline__ bf16x8 as_operand(const f32x16 &c, int s) {
  bf16x8 o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = (__bf16)c[8 * s + e];
  return o;
}
// Row of C register r (kappa: the same as 16 s + .. for r = 8 s + e).
__device__ __forceinline__ int c_row(int r, int h) { return (r & 3) + 8 * (r >> 2) + 4 * h; }

// Column c of a result C^T (rows are the D values of a head) to row `out` of a bf16 tensor, times f.
template <int DB>
__device__ __forceinline__ void store_column(const f32x16 (&c)[DB], float f, uint16_t *out, int D, int h) {
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int at = 32 * d + 8 * g + 4 * h;
      if (at >= D) continue;
      const bf16x2 lo = {(__bf16)(c[d][4 * g] * f), (__bf16)(c[d][4 * g + 1] * f)};
      const bf16x2 hi = {(__bf16)(c[d][4 * g + 2] * f), (__bf16)(c[d][4 * g + 3] * f)};
      *reinterpret_cast<u32x2 *>(out + at) = u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    }
}

template <int DB>
__device__ __forceinline__ void store_column_f32(const f32x16 (&c)[DB], float f, float *out, int D, int h) {
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int at = 32 * d + 8 * g + 4 * h;
      if (at >= D) continue;
      *reinterpret_cast<f32x4 *>(out + at) = f32x4{c[d][4 * g] * f, c[d][4 * g + 1] * f, c[d][4 * g + 2] * f, c[d][4 * g + 3] * f};
    }
}

// Over the two lanes that share a column.
__device__ __forceinline__ float max_halves(float v) {
  const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}
__device__ __forceinline__ float add_halves(float v) {
  const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// Whether a tile holds an infinity or a NaN (every lane of the wave gets the answer).
template <int P, int ROWS>
__device__ __forceinline__ bool tile_nonfinite(const uint8_t *tile, int lane) {
  bool bad = false;
#pragma unroll 4
  for (int i = 0; i < ROWS * P / 64; ++i) {
    const u32x4 w = *reinterpret_cast<const u32x4 *>(tile + 16 * (64 * i + lane));
#pragma unroll
    for (int j = 0; j < 4; ++j) bad |= (w[j] & 0x7f80u) == 0x7f80u || (w[j] & 0x7f800000u) == 0x7f800000u;
  }
  return __ballot(bad) != 0;
}

// c[d] += (rows r0 .. r0 + 15 of a tile)^T b where b is 0 at masked (row, column) places and the tile holds
// infinities or NaN: one at a masked place must not reach the column (0 times it is NaN).  The finite values
// are multiplied as always, so what no other value touches has the same bits; then the others, each row
// alone, added only to the columns that see it.  sees(row): whether this lane's column does.
template <int P, int DB, typename Sees>
__device__ __forceinline__ void add_rows_apart(const uint8_t *tile, int r0, const bf16x8 &b, f32x16 (&c)[DB],
                                               const TileRead<P> &at, int lane, Sees sees) {
  auto split = [](uint32_t w, bool finite) {  // the halves of w that are finite, or those that are not
    const uint32_t bad = ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
    return finite ? w & ~bad : w & bad;
  };
#pragma unroll
  for (int d = 0; d < DB; ++d) {
    u32x4 w = __builtin_bit_cast(u32x4, at.column_operand(tile, r0, d));
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = split(w[i], true);
    c[d] = mfma(__builtin_bit_cast(bf16x8, w), b, c[d]);
  }
#pragma unroll 1
  for (int row = 0; row < 16; ++row) {
    const int h = (row >> 2) & 1, e = 4 * (row >> 3) + (row & 3);  // kappa(0, h, e) = row
    const bool add = sees(r0 + row);
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      u32x4 w = __builtin_bit_cast(u32x4, at.column_operand(tile, r0, d));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (lane >> 5) == h && e >> 1 == i ? split(w[i], false) & (e & 1 ? 0xffff0000u : 0xffffu) : 0u;
      const f32x16 t = mfma(__builtin_bit_cast(bf16x8, w), b, zeros16());
#pragma unroll
      for (int r = 0; r < 16; ++r) c[d][r] = (int)add & (int)(t[r] != 0.0f) ? c[d][r] + t[r] : c[d][r];
    }
  }
}

}  // namespace nvfp4
