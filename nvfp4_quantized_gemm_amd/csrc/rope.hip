// Rotary positions with several axes (gfx950): the first axis_dims[0] elements of every head turn by
// the token's first coordinate, the next axis_dims[1] by the second, and so on; elements past the
// sections pass through.
//
// Pair p of axis a (pairs are numbered through the sections in order) turns by
//   angle = RN32(positions[t][a] * inv_freq[p]):   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin),
// the inverse by -angle: the transpose of the rotation, which is its gradient.  Layout pairs: x1, x2
// are neighbours; layout halves: they lie half a section apart.
//
// cos and sin are taken once per token and pair, into LDS, for all heads.  The angle is brought to
// turns with 1/(2 pi) held in two floats, so the reduction is exact to 2^-48 of the angle and
// large positions lose nothing beyond the angle's own fp32 rounding.
//
// Bound by memory: every element is read and written once.  10240 x 64 x 128 bf16 out of a QKV row (pairs): 56.6
// us, 5.9 TB/s, the rate of a large copy; halves of 22 and 21: 59 us; 4097 x 32 x 72 (38 MB): pairs 10.0 us,
// halves of 18 11.4 us, one token 2.9 us, where the launch and one round of latency count.
#include <algorithm>
#include <type_traits>

#include "launch.hpp"
#include "mx8.hpp"

namespace nvfp4 {

namespace {

__device__ __forceinline__ f32x2 turn(float angle) {
  constexpr float kHi = 0x1.45f306p-3f, kLo = 0x1.b9391p-28f;  // 1 / (2 pi) = kHi + kLo
  const float p = angle * kHi;
  const float e = fmaf(angle, kLo, fmaf(angle, kHi, -p));
  const float r = (p - rintf(p)) + e;
  f32x2 cs;
  float s, c;
  sincospif(2.0f * r, &s, &c);
  cs.x = c;
  cs.y = s;
  return cs;
}

constexpr int kUnits = 1024;  // pieces of 8 elements that a workgroup takes at a time

// The block's table of cosines and sines, cs[token][pair], in two parts: each thread's first entry's
// operands are loaded before the tensor's (loads come back in order), the table is filled behind them.
struct TableEntry {
  float position, freq;
};
__device__ __forceinline__ TableEntry load_entry(const RopeArgs &a, int64_t t0, int i) {
  const int t = (int)fastdiv((uint32_t)i, a.div_p), p = i - t * a.pairs;
  int ax = 0;
  for (int k = 0; k < kRopeMaxAxes - 1; ++k) ax += k < a.n_axes - 1 && p >= a.pair_end[k];
  return {a.positions[(t0 + t) * a.n_axes + ax], a.inv_freq[p]};
}
__device__ __forceinline__ void fill_table(const RopeArgs &a, int64_t t0, int entries, TableEntry e, f32x2 *cs) {
  for (int i = threadIdx.x; i < entries; i += 256) {
    if (i >= 256) e = load_entry(a, t0, i);
    f32x2 v = turn(e.position * e.freq);
    if (a.inverse) v.y = -v.y;
    cs[i] = v;
  }
}

// V consecutive elements, fp32 or bf16 (2 to 32 bytes; 16-byte accesses at most).
template <int DT, int V>
struct Elems {
  static constexpr int kBytes = V * (DT == 0 ? 4 : 2);
  typedef typename std::conditional<kBytes == 2, uint16_t, typename std::conditional<kBytes == 4, uint32_t, typename std::conditional<
      kBytes == 8, u32x2, u32x4>::type>::type>::type Word;
  static constexpr int kWords = kBytes > 16 ? kBytes / 16 : 1;
  Word w[kWords];
  __device__ __forceinline__ void load(const void *base, int64_t elem) {
    const Word *p = reinterpret_cast<const Word *>(static_cast<const uint8_t *>(base) + elem * (DT == 0 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __builtin_nontemporal_load(p + i);
  }
  template <bool NT>
  __device__ __forceinline__ void store(void *base, int64_t elem) const {
    Word *p = reinterpret_cast<Word *>(static_cast<uint8_t *>(base) + elem * (DT == 0 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (NT) __builtin_nontemporal_store(w[i], p + i);
      else p[i] = w[i];
    }
  }
  __device__ __forceinline__ void load_lds(const uint8_t *p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const Word *>(p)[i];
  }
  __device__ __forceinline__ void store_lds(uint8_t *p) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<Word *>(p)[i] = w[i];
  }
  __device__ __forceinline__ uint32_t word(int i) const {  // 32 bits
    if constexpr (kBytes <= 4) return w[0];
    else if constexpr (kBytes == 8) return w[0][i];
    else return w[i / 4][i % 4];
  }
  __device__ __forceinline__ void set_word(int i, uint32_t v) {
    if constexpr (kBytes <= 4) w[0] = (Word)v;
    else if constexpr (kBytes == 8) w[0][i] = v;
    else w[i / 4][i % 4] = v;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == 0) return __uint_as_float(word(i));
    else return (i & 1) ? bf16hi(word(i / 2)) : bf16lo(word(i / 2));
  }
  __device__ __forceinline__ void set(const float (&v)[V]) {
    if constexpr (DT == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) set_word(i, __float_as_uint(v[i]));
    } else if constexpr (V == 1) {
      w[0] = __builtin_bit_cast(uint16_t, (__bf16)v[0]);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const bf16x2 h = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
        set_word(i, __builtin_bit_cast(uint32_t, h));
      }
    }
  }
};

}  // namespace

// One workgroup turns `tokens` consecutive tokens, 256 x B units at a time.  Layout pairs: a unit is 8
// elements (4 pairs).
template <int DT, bool NT>
__global__ __launch_bounds__(256) void k_rope_pairs(RopeArgs a) {
  constexpr int B = 4;
  extern __shared__ f32x2 cs[];
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)min((int64_t)a.tokens, a.T - t0);
  const int C = a.D / 8, n = nt * a.H * C, entries = nt * a.pairs;
  TableEntry e = {0.0f, 0.0f};
  if ((int)threadIdx.x < entries) e = load_entry(a, t0, threadIdx.x);
  for (int base = 0; base < n; base += 256 * B) {
    Elems<DT, 8> v[B];
    int tt[B], cc[B], hh[B];
#pragma unroll
    for (int q = 0; q < B; ++q) {
      const int i = base + 256 * q + threadIdx.x;
      const int row = (int)fastdiv((uint32_t)i, a.div_c);
      cc[q] = i - row * C;
      tt[q] = (int)fastdiv((uint32_t)row, a.div_h);
      hh[q] = row - tt[q] * a.H;
      if (i < n) v[q].load(a.x, (t0 + tt[q]) * a.ld_t + hh[q] * a.ld_h + 8 * cc[q]);
    }
    if (base == 0) {
      fill_table(a, t0, entries, e, cs);
      __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < B; ++q) {
      if (base + 256 * q + (int)threadIdx.x >= n) break;
      float y[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int p = 4 * cc[q] + k;
        const float x1 = v[q].get(2 * k), x2 = v[q].get(2 * k + 1);
        y[2 * k] = x1;  // past the sections: as it is
        y[2 * k + 1] = x2;
        if (p < a.pairs) {
          const f32x2 r = cs[tt[q] * a.pairs + p];
          y[2 * k] = x1 * r.x - x2 * r.y;
          y[2 * k + 1] = x2 * r.x + x1 * r.y;
        }
      }
      v[q].set(y);
      v[q].template store<NT>(a.y, (t0 + tt[q]) * a.ldy_t + hh[q] * a.ldy_h + 8 * cc[q]);
    }
  }
}

// Layout halves where 8 divides every half section, and half of what lies past the sections (which is copied
// as pairs of its own): a unit is 8 consecutive pairs, i.e. 8 elements and the 8 half a section on.  Two units a
// thread, as many as a workgroup has (with room for four: 2048 x 8 x 128 3.8 us and 4.1, 4096 x 32 x 128 fp32
// 28.7 and 30.5).
template <int DT, bool NT>
__global__ __launch_bounds__(256) void k_rope_halves(RopeArgs a) {
  constexpr int B = 2, V = 8;
  extern __shared__ f32x2 cs[];
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)min((int64_t)a.tokens, a.T - t0);
  const int C = a.D / (2 * V), n = nt * a.H * C, entries = nt * a.pairs;
  TableEntry e = {0.0f, 0.0f};
  if ((int)threadIdx.x < entries) e = load_entry(a, t0, threadIdx.x);
  for (int base = 0; base < n; base += 256 * B) {
    Elems<DT, V> v[B][2];
    int tt[B], pp[B], hh[B], e1[B], e2[B];
#pragma unroll
    for (int q = 0; q < B; ++q) {
      const int i = base + 256 * q + threadIdx.x;
      const int row = (int)fastdiv((uint32_t)i, a.div_c);
      const int p = (i - row * C) * V;
      int p0 = 0, end = a.pair_end[0];  // the section's pairs; past the sections: the rest of the head's
#pragma unroll
      for (int k = 0; k < kRopeMaxAxes; ++k) {
        if (k < a.n_axes && p >= a.pair_end[k]) {
          p0 = a.pair_end[k];
          end = k + 1 < a.n_axes ? a.pair_end[k + 1 < kRopeMaxAxes ? k + 1 : k] : a.D / 2;
        }
      }
      pp[q] = p;
      e1[q] = p + p0;  // the section starts at element 2 p0
      e2[q] = p + end;
      tt[q] = (int)fastdiv((uint32_t)row, a.div_h);
      hh[q] = row - tt[q] * a.H;
      if (i < n) {
        const int64_t src = (t0 + tt[q]) * a.ld_t + hh[q] * a.ld_h;
        v[q][0].load(a.x, src + e1[q]);
        v[q][1].load(a.x, src + e2[q]);
      }
    }
    if (base == 0) {
      fill_table(a, t0, entries, e, cs);
      __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < B; ++q) {
      if (base + 256 * q + (int)threadIdx.x >= n) break;
      if (pp[q] < a.pairs) {
        float y1[V], y2[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const f32x2 r = cs[tt[q] * a.pairs + pp[q] + k];
          const float x1 = v[q][0].get(k), x2 = v[q][1].get(k);
          y1[k] = x1 * r.x - x2 * r.y;
          y2[k] = x2 * r.x + x1 * r.y;
        }
        v[q][0].set(y1);
        v[q][1].set(y2);
      }
      const int64_t dst = (t0 + tt[q]) * a.ldy_t + hh[q] * a.ldy_h;
      v[q][0].template store<NT>(a.y, dst + e1[q]);
      v[q][1].template store<NT>(a.y, dst + e2[q]);
    }
  }
}

// Layout halves of other lengths: elements and their partners share no alignment past V elements (the largest
// of 4, 2, 1 that divides every half section), and accesses of so few bytes bound the kernel above (10240 x 64
// x 128 bf16, sections of 44, 42, 42: 104 us by elements of 2 bytes, 59 here; 4097 x 32 x 72, halves of 18:
// 12.9 and 11.4; halves of 12: 13.9 and 11.5).  So units of 8 elements go through LDS whole, and each takes its
// partners from there, V at a time.  A workgroup has the heads `heads` of its tokens, in chunks where a
// token has more.  The table holds an entry per element, (cos, -+sin), in the units' order, so that lanes
// read neighbouring words; `other` has every piece's partner.
template <int DT, int V, bool NT>
__global__ __launch_bounds__(256, DT == 0 ? 6 : 8) void k_rope_staged(RopeArgs a) {
  constexpr int B = kUnits / 256, ES = DT == 0 ? 4 : 2, NP = 8 / V;
  extern __shared__ f32x4 lds[];
  const int C = a.D / 8;
  uint8_t *const data = reinterpret_cast<uint8_t *>(lds);                       // [heads][D]
  f32x4 *const tab = reinterpret_cast<f32x4 *>(data + kUnits * 8 * ES);         // [token][4][C]: 2 x (cos, +-sin)
  uint16_t *const other = reinterpret_cast<uint16_t *>(tab + a.tokens * 4 * C);  // [D / V]
  const int64_t group = blockIdx.x / a.chunks;
  const int h0 = (int)(blockIdx.x % a.chunks) * a.heads, nh = min(a.heads, a.H - h0);
  const int64_t t0 = group * a.tokens;
  const int nt = (int)min((int64_t)a.tokens, a.T - t0);
  const int n = nt * nh * C, entries = nt * a.pairs;
  TableEntry e = {0.0f, 0.0f};
  if ((int)threadIdx.x < entries) e = load_entry(a, t0, threadIdx.x);
  Elems<DT, 8> v[B];
#pragma unroll
  for (int q = 0; q < B; ++q) {
    const int i = 256 * q + threadIdx.x;
    const int row = (int)fastdiv((uint32_t)i, a.div_c), c = i - row * C;
    const int tk = (int)fastdiv((uint32_t)row, a.div_h), h = h0 + row - tk * a.heads;
    if (i < n) v[q].load(a.x, (t0 + tk) * a.ld_t + h * a.ld_h + 8 * c);
  }
  for (int i = 255 - (int)threadIdx.x; i < a.D / V; i += 256) {
    const int el = i * V;
    int o = el, p0 = 0;
#pragma unroll
    for (int k = 0; k < kRopeMaxAxes; ++k) {
      if (k < a.n_axes) {
        const int end = a.pair_end[k];
        if (el >= 2 * p0 && el < 2 * end) o = el < p0 + end ? el + (end - p0) : el - (end - p0);
        p0 = end;
      }
    }
    other[i] = (uint16_t)o;
  }
  for (int i = threadIdx.x; i < entries; i += 256) {
    if (i >= 256) e = load_entry(a, t0, i);
    const int t = (int)fastdiv((uint32_t)i, a.div_p), p = i - t * a.pairs;
    int p0 = 0, end = a.pair_end[0];
#pragma unroll
    for (int k = 0; k < kRopeMaxAxes - 1; ++k)
      if (k < a.n_axes - 1 && p >= a.pair_end[k]) p0 = a.pair_end[k], end = a.pair_end[k + 1];
    f32x2 r = turn(e.position * e.freq);
    if (a.inverse) r.y = -r.y;
    f32x2 *const row = reinterpret_cast<f32x2 *>(tab + t * 4 * C);
    const int e1 = p + p0, e2 = p + end;
    row[(((e2 >> 1) & 3) * C + (e2 >> 3)) * 2 + (e2 & 1)] = r;
    r.y = -r.y;
    row[(((e1 >> 1) & 3) * C + (e1 >> 3)) * 2 + (e1 & 1)] = r;
  }
#pragma unroll
  for (int q = 0; q < B; ++q) {
    const int i = 256 * q + threadIdx.x;
    if (i < n) v[q].store_lds(data + i * 8 * ES);
  }
  __syncthreads();
#pragma unroll 2
  for (int q = 0; q < B; ++q) {
    const int i = 256 * q + (int)threadIdx.x;
    if (i >= n) break;
    const int row = (int)fastdiv((uint32_t)i, a.div_c), c = i - row * C;
    const int tk = (int)fastdiv((uint32_t)row, a.div_h), h = h0 + row - tk * a.heads;
    const uint8_t *const head = data + (i - c) * 8 * ES;
    Elems<DT, 8> x;
    x.load_lds(data + i * 8 * ES);
    float y[8];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const f32x4 r = tab[(tk * 4 + m) * C + c];
      y[2 * m] = x.get(2 * m) * r.x;
      y[2 * m + 1] = x.get(2 * m + 1) * r.z;
      Elems<DT, (V < 2 ? 1 : 2)> w[V < 2 ? 2 : 1];
      if constexpr (V == 1) {
        w[0].load_lds(head + other[8 * c + 2 * m] * ES);
        w[1].load_lds(head + other[8 * c + 2 * m + 1] * ES);
        y[2 * m] += w[0].get(0) * r.y;
        y[2 * m + 1] += w[1].get(0) * r.w;
      } else {
        w[0].load_lds(head + (other[NP * c + 2 * m / V] + 2 * m % V) * ES);
        y[2 * m] += w[0].get(0) * r.y;
        y[2 * m + 1] += w[0].get(1) * r.w;
      }
    }
    const int in = 2 * a.pairs - 8 * c;  // past the sections: as it is
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k >= in) y[k] = x.get(k);
    x.set(y);
    x.template store<NT>(a.y, (t0 + tk) * a.ldy_t + h * a.ldy_h + 8 * c);
  }
}

namespace {

template <int DT, bool NT>
hipError_t launch_layout(const RopeArgs &a, int V, unsigned grid, size_t lds, hipStream_t s) {
  if (!a.halves) k_rope_pairs<DT, NT><<<grid, 256, lds, s>>>(a);
  else if (V == 8) k_rope_halves<DT, NT><<<grid, 256, lds, s>>>(a);
  else if (V == 4) k_rope_staged<DT, 4, NT><<<grid, 256, lds, s>>>(a);
  else if (V == 2) k_rope_staged<DT, 2, NT><<<grid, 256, lds, s>>>(a);
  else k_rope_staged<DT, 1, NT><<<grid, 256, lds, s>>>(a);
  return hipGetLastError();
}

// Streaming stores above 128 MB, half the last-level cache, where the result would not be there for its
// reader anyway (10240 x 64 x 128 bf16, 168 MB: 56.9 us and 60.4); below they cost time (4097 x 32 x 72
// fp32, 38 MB: 20.1 us and 18.9).
template <int DT>
hipError_t launch_dtype(const RopeArgs &a, int V, unsigned grid, size_t lds, hipStream_t s) {
  const bool stream = a.T * a.H * a.D * (DT == 0 ? 4 : 2) > (int64_t(128) << 20);
  return stream ? launch_layout<DT, true>(a, V, grid, lds, s) : launch_layout<DT, false>(a, V, grid, lds, s);
}

}  // namespace

hipError_t launch_rope(RopeArgs a, hipStream_t s) {
  // About kUnits pieces per workgroup, at least one token; fewer where that leaves CUs idle: down to 512
  // workgroups, and to 256 of less than 256 pieces (halves of 64 bf16: 2048 x 8 x 128 at 256, 512, 1024
  // workgroups 4.4, 4.1 and 4.6 us; 1000 x 8 x 80 at 84, 334, 1000: 4.4, 3.6 and 4.0).
  const int64_t per = (int64_t)a.H * (a.D / 8);
  int64_t tokens = std::min<int64_t>(per >= kUnits ? 1 : kUnits / per, 16);
  tokens = std::min(tokens, std::max<int64_t>({1, a.T / 512, std::min<int64_t>(256 / per, a.T / 256)}));
  int bits = 8 | (a.D / 2 - a.pairs);  // with half of what lies past the sections
  for (int i = 0, p0 = 0; i < a.n_axes; p0 = a.pair_end[i++]) bits |= a.pair_end[i] - p0;
  const int V = bits & -bits;
  const bool staged = a.halves && V < 8;
  a.heads = a.H;
  a.chunks = 1;
  if (staged) {  // whole heads in LDS: kUnits at most, and a table of 2048 elements' angles
    const int most = kUnits / (a.D / 8);
    a.chunks = (a.H + most - 1) / most;
    a.heads = (a.H + a.chunks - 1) / a.chunks;
    a.chunks = (a.H + a.heads - 1) / a.heads;
    tokens = std::min<int64_t>(tokens, 2048 / a.D);
  }
  a.tokens = (int)tokens;
  a.div_c = make_fastdiv((uint32_t)(a.halves && !staged ? a.D / 16 : a.D / 8));
  a.div_h = make_fastdiv((uint32_t)a.heads);
  a.div_p = make_fastdiv((uint32_t)(a.pairs > 0 ? a.pairs : 1));
  const int64_t es = a.dtype == 0 ? 4 : 2, most = tokens * ((1 << 22) / a.chunks);  // tokens of one launch's grid
  const size_t lds = staged ? 8 * kUnits * es + tokens * a.D * sizeof(f32x2) + a.D / V * sizeof(uint16_t)
                            : tokens * a.pairs * sizeof(f32x2);
  for (int64_t left = a.T; left > 0; left -= most) {
    a.T = left < most ? left : most;
    const unsigned grid = (unsigned)((a.T + tokens - 1) / tokens * a.chunks);
    const hipError_t e = a.dtype == 0 ? launch_dtype<0>(a, V, grid, lds, s) : launch_dtype<1>(a, V, grid, lds, s);
    if (e != hipSuccess) return e;
    a.x = static_cast<const uint8_t *>(a.x) + a.T * a.ld_t * es;
    a.y = static_cast<uint8_t *>(a.y) + a.T * a.ldy_t * es;
    a.positions += a.T * a.n_axes;
  }
  return hipSuccess;
}

}  // namespace nvfp4
