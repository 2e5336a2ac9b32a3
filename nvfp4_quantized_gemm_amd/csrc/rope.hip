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

template <int DT>
__device__ __forceinline__ float get1(const void *p, int64_t e) {
  return DT == 0 ? static_cast<const float *>(p)[e] : bf16lo(static_cast<const uint16_t *>(p)[e]);
}

}  // namespace

// One workgroup turns `tokens` consecutive tokens.  cs[token][pair] in LDS.  Layout pairs: a lane
// takes 8 elements (4 pairs) at a time.
template <int DT>
__global__ __launch_bounds__(256) void k_rope_pairs(RopeArgs a) {
  extern __shared__ f32x2 cs[];
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)min((int64_t)a.tokens, a.T - t0);
  for (int i = threadIdx.x; i < nt * a.pairs; i += 256) {
    const int t = i / a.pairs, p = i - t * a.pairs;
    int ax = 0;
    while (p >= a.pair_end[ax]) ++ax;
    f32x2 v = turn(a.positions[(t0 + t) * a.n_axes + ax] * a.inv_freq[p]);
    if (a.inverse) v.y = -v.y;
    cs[i] = v;
  }
  __syncthreads();
  const int C = a.D / 8, n = nt * a.H * C;
  for (int i = threadIdx.x; i < n; i += 256) {
    const int row = (int)fastdiv((uint32_t)i, a.div_c), c = i - row * C;
    const int t = (int)fastdiv((uint32_t)row, a.div_h), h = row - t * a.H;
    Vec8<DT> v;
    v.template load<true>(a.x, (t0 + t) * a.ld_t + h * a.ld_h + 8 * c);
    float x[8];
    v.get(x);
    float y[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int p = 4 * c + q;
      if (p < a.pairs) {
        const f32x2 r = cs[t * a.pairs + p];
        y[2 * q] = x[2 * q] * r.x - x[2 * q + 1] * r.y;
        y[2 * q + 1] = x[2 * q + 1] * r.x + x[2 * q] * r.y;
      } else {
        y[2 * q] = x[2 * q];
        y[2 * q + 1] = x[2 * q + 1];
      }
    }
    v.set(y);
    v.template store<false>(a.y, (t0 + t) * a.ldy_t + h * a.ldy_h + 8 * c);
  }
}

// Layout halves: a lane takes one pair; the elements past the sections are copied as pairs of their own.
template <int DT>
__global__ __launch_bounds__(256) void k_rope_halves(RopeArgs a) {
  extern __shared__ f32x2 cs[];
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)min((int64_t)a.tokens, a.T - t0);
  for (int i = threadIdx.x; i < nt * a.pairs; i += 256) {
    const int t = i / a.pairs, p = i - t * a.pairs;
    int ax = 0;
    while (p >= a.pair_end[ax]) ++ax;
    f32x2 v = turn(a.positions[(t0 + t) * a.n_axes + ax] * a.inv_freq[p]);
    if (a.inverse) v.y = -v.y;
    cs[i] = v;
  }
  __syncthreads();
  const int C = a.D / 2, n = nt * a.H * C;
  for (int i = threadIdx.x; i < n; i += 256) {
    const int row = i / C, p = i - row * C;
    const int t = (int)fastdiv((uint32_t)row, a.div_h), h = row - t * a.H;
    const int64_t src = (t0 + t) * a.ld_t + h * a.ld_h, dst = (t0 + t) * a.ldy_t + h * a.ldy_h;
    int e1, e2;
    float c = 1.0f, s = 0.0f;
    if (p < a.pairs) {
      int ax = 0;
      while (p >= a.pair_end[ax]) ++ax;
      const int p0 = ax ? a.pair_end[ax - 1] : 0;
      e1 = p + p0;  // the section starts at element 2 p0
      e2 = e1 + a.pair_end[ax] - p0;
      c = cs[t * a.pairs + p].x;
      s = cs[t * a.pairs + p].y;
    } else {
      e1 = 2 * p;
      e2 = e1 + 1;
    }
    const float x1 = get1<DT>(a.x, src + e1), x2 = get1<DT>(a.x, src + e2);
    const bool pass = p >= a.pairs;
    const float y1 = pass ? x1 : x1 * c - x2 * s, y2 = pass ? x2 : x2 * c + x1 * s;
    if (DT == 0) {
      static_cast<float *>(a.y)[dst + e1] = y1;
      static_cast<float *>(a.y)[dst + e2] = y2;
    } else {
      static_cast<__bf16 *>(a.y)[dst + e1] = (__bf16)y1;
      static_cast<__bf16 *>(a.y)[dst + e2] = (__bf16)y2;
    }
  }
}

hipError_t launch_rope(RopeArgs a, hipStream_t s) {
  // about 1024 vectors of 8 elements per workgroup, at least one token
  const int64_t per = (int64_t)a.H * (a.D / 8);
  int64_t tokens = per >= 1024 ? 1 : 1024 / per;
  if (tokens > 16) tokens = 16;
  a.tokens = (int)tokens;
  a.div_c = make_fastdiv((uint32_t)(a.D / 8));
  a.div_h = make_fastdiv((uint32_t)a.H);
  const unsigned grid = (unsigned)((a.T + tokens - 1) / tokens);
  const size_t lds = (size_t)tokens * a.pairs * sizeof(f32x2);
  if (a.halves) {
    if (a.dtype == 0) k_rope_halves<0><<<grid, 256, lds, s>>>(a);
    else k_rope_halves<1><<<grid, 256, lds, s>>>(a);
  } else {
    if (a.dtype == 0) k_rope_pairs<0><<<grid, 256, lds, s>>>(a);
    else k_rope_pairs<1><<<grid, 256, lds, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
