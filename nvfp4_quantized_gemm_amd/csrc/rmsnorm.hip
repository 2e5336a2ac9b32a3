// Root-mean-square norm with the residual's addition and MXFP8 output, and its backward pass (gfx950).
//
//   s = x + residual           (fp32)              h = s rounded to x's type
//   inv_rms = 1 / sqrt(mean_k s^2 + eps)           y = s inv_rms weight
//   codes, scales = MXFP8(y)                       (mx8.hpp)
// The norm is of the fp32 sum, not of the rounded h: h is rounded once, for the next layer, and y
// once, to its 8 bits.  Sums of squares and everything before the encoding are fp32; a row whose sum of
// squares leaves fp32 is summed again times 2^-80 (overflowing_rms).  A row with a non-finite value has no norm:
// inv_rms, y, codes and scales are NaN.
//
// Bound by memory.  One pass: the row stays in registers between the sum of squares and the output, so x and
// residual are read and h and the codes written once (7.03 B per bf16 element): 16384 x 8192 in 158 to 164 us,
// 5.8 TB/s, where a large copy moves 5.9; 4096 x 1152 in 7.9 us; one row of 4608 in 3.7 us, 2.0 of them the
// launch.
//
// Backward, with n = h inv_rms, g = dy weight, c = mean_k(g n):
//   dx = inv_rms (g - n c) + dh  (x's gradient and the residual's)      dweight = sum_m dy n
#include <cfloat>
#include <cmath>

#include "launch.hpp"
#include "mx8.hpp"

namespace nvfp4 {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
  v += swap_lane1(v);
  v += swap_lane2(v);
  v += swap_lane4(v);
  v += swap_lane8(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Sum over the TPR threads of a row; every one of them gets it.  TPR == 64: the row is one wave's
// and no other wave is waited for.  Otherwise the row is the whole workgroup's, and `red` holds two
// sets of partials used in turn, so one barrier per row is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *red, int set) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float *r = red + set * W;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += r[i];
  }
  return v;
}

// A weight vector: 1 where there is no weight, else 8 values of either type.
__device__ __forceinline__ void load_weight(const void *w, int w_dtype, int64_t k, float (&v)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.0f;
  } else if (w_dtype == 0) {
    Vec8<0> t;
    t.load<false>(w, k);
    t.get(v);
  } else {
    Vec8<1> t;
    t.load<false>(w, k);
    t.get(v);
  }
}

// inv_rms of a row s whose mean square + eps is past fp32: both times 2^-160, where no finite row overflows
// (2^96 a square) and what underflows is below 2^-100 of the sum.  NaN where a value is not finite.  A third set
// of partials: the rows before and after this one use the other two.
template <int TPR, int NV>
__device__ __forceinline__ float overflowing_rms(const float (&s)[NV][8], float *red, const NormArgs &a) {
  constexpr float kDown = 0x1p-80f;
  float sq = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = s[j][i] * kDown;
      sq = fmaf(v, v, sq);
    }
  const float square = row_sum<TPR>(sq, red, 2) * a.inv_k + a.eps * kDown * kDown;
  return square <= FLT_MAX ? kDown / sqrtf(square) : NAN;
}

}  // namespace

// TPR threads (64, 256 or 1024) hold a row in registers, NV vectors of 8 elements each; workgroups
// of 256 threads take 4 rows at TPR = 64.  A workgroup walks over rows with the weight in registers
// and the next row's loads in flight while it works on one.
template <int DT, int TPR, int NV, bool NT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm(NormArgs a) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  constexpr bool kAhead = TPR < 1024 || NV <= 2;  // 16 waves leave 128 registers: none to look ahead
  __shared__ float red[TPR > 64 ? 3 * TPR / 64 : 1];  // two sets in turn, and one of overflowing_rms
  const int t = threadIdx.x % TPR;
  const int nseg = (int)(a.K / 8);
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t m = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  Vec8<DT> x[NV], r[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int seg = j * TPR + t;
      x[j].zero();
      r[j].zero();
      if (seg < nseg) {
        x[j].template load<true>(a.x, row * a.ld_x + 8 * seg);
        if (a.residual) r[j].template load<true>(a.residual, row * a.ld_r + 8 * seg);
      }
    }
  };
  if (kAhead && m < a.M) fetch(m);
  float w[kAhead ? NV : 1][8];
  if constexpr (kAhead) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int seg = j * TPR + t;
      load_weight(a.weight, a.w_dtype, 8 * (seg < nseg ? seg : 0), w[j]);
    }
  }
  for (int phase = 0; m < a.M; m += step, ++phase) {
    if constexpr (!kAhead) fetch(m);
    float s[NV][8];
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int seg = j * TPR + t;
      float v[8];
      x[j].get(s[j]);
      r[j].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[j][i] += v[i];
        sq = fmaf(s[j][i], s[j][i], sq);
      }
      if (a.h && seg < nseg) {
        Vec8<DT> h;
        h.set(s[j]);
        h.template store<NT>(a.h, m * a.ld_h + 8 * seg);
      }
    }
    if (kAhead && m + step < a.M) fetch(m + step);
    const float square = row_sum<TPR>(sq, red, phase & 1) * a.inv_k + a.eps;
    // the same for all of a row's threads, so they go together to the barrier inside
    const float inv_rms = square <= FLT_MAX ? 1.0f / sqrtf(square) : overflowing_rms<TPR, NV>(s, red, a);
    if (a.inv_rms && t == 0) a.inv_rms[m] = inv_rms;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int seg = j * TPR + t;
      if (seg >= nseg) break;  // whole blocks: K % 32 == 0 keeps 4 adjacent lanes together
      float y[8];
      float(&wj)[8] = w[kAhead ? j : 0];
      if constexpr (!kAhead) load_weight(a.weight, a.w_dtype, 8 * seg, wj);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = s[j][i] * inv_rms * wj[i];
      if (a.codes || a.fake) {
        const uint32_t b = mx8_scale_byte(mx8_amax_bits(y));
        const u32x2 c = mx8_encode8(y, b);
        if (a.codes) {
          u32x2 *const to = reinterpret_cast<u32x2 *>(a.codes + m * a.K + 8 * seg);
          if constexpr (NT) __builtin_nontemporal_store(c, to);
          else *to = c;
          if ((seg & 3) == 0) a.scales[m * (a.K / kMx8Blk) + (seg >> 2)] = (uint8_t)b;
        }
        if (a.fake) mx8_decode8(c, b, y);
      }
      if (a.y) {
        if (a.y_dtype == 0) {
          Vec8<0> o;
          o.set(y);
          o.store<NT>(a.y, m * a.ld_y + 8 * seg);
        } else {
          Vec8<1> o;
          o.set(y);
          o.store<NT>(a.y, m * a.ld_y + 8 * seg);
        }
      }
    }
  }
}

// Backward: the rows as above; every thread adds its columns' dy n over the rows it sees, and the
// workgroup writes one partial row of dweight, [gridDim.x][K] fp32, which k_sum_rows adds in order (no
// atomics: equal inputs give equal bits).  4096 x 1152 bf16 with dh: 13.3 us for both launches, 8 B per
// element at 2.8 TB/s; 10240 x 4608: 70 us, 5.4 TB/s.  Above K = 16384 a thread's rows and
// sums spill to scratch.
template <int DT, int TPR, int NV, bool NT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm_backward(NormGradArgs a) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  constexpr bool kAhead = TPR < 1024;
  __shared__ float red[TPR > 64 ? 2 * TPR / 64 : 1];
  __shared__ float fold[kRows > 1 ? (kRows - 1) * TPR * 8 : 1];
  const int t = threadIdx.x % TPR;
  const int nseg = (int)(a.K / 8);
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t m = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  Vec8<DT> vh[NV], vy[NV], vd[NV];
  float next_rms = 0.0f;
  auto fetch = [&](int64_t row) {
    next_rms = a.inv_rms[row];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int seg = j * TPR + t;
      vh[j].zero();
      vy[j].zero();
      vd[j].zero();
      if (seg < nseg) {
        vh[j].template load<true>(a.h, row * a.ld_h + 8 * seg);
        vy[j].template load<true>(a.dy, row * a.ld_dy + 8 * seg);
        if (a.dh) vd[j].template load<true>(a.dh, row * a.ld_dh + 8 * seg);
      }
    }
  };
  if (kAhead && m < a.M) fetch(m);
  float w[kAhead ? NV : 1][8], dw[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int seg = j * TPR + t;
    if constexpr (kAhead) load_weight(a.weight, a.w_dtype, 8 * (seg < nseg ? seg : 0), w[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
  }
  for (int phase = 0; m < a.M; m += step, ++phase) {
    if constexpr (!kAhead) fetch(m);
    const float inv_rms = next_rms;
    float n[NV][8], g[NV][8];
    Vec8<DT> d[NV];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int seg = j * TPR + t;
      float(&wj)[8] = w[kAhead ? j : 0];
      if constexpr (!kAhead) load_weight(a.weight, a.w_dtype, 8 * (seg < nseg ? seg : 0), wj);
      vh[j].get(n[j]);
      vy[j].get(g[j]);
      d[j] = vd[j];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[j][i] *= inv_rms;
        dw[j][i] = fmaf(g[j][i], n[j][i], dw[j][i]);
        g[j][i] *= wj[i];
        dot = fmaf(g[j][i], n[j][i], dot);
      }
    }
    if (kAhead && m + step < a.M) fetch(m + step);
    const float c = row_sum<TPR>(dot, red, phase & 1) * a.inv_k;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int seg = j * TPR + t;
      if (seg >= nseg) break;
      float o[8];
      d[j].get(o);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fmaf(inv_rms, fmaf(-n[j][i], c, g[j][i]), o[i]);
      Vec8<DT> q;
      q.set(o);
      q.template store<NT>(a.dx, m * a.ld_dx + 8 * seg);
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int seg = j * TPR + t;
    if constexpr (kRows > 1) {  // the workgroup's waves, in order
      const int r = threadIdx.x / TPR;
      __syncthreads();
      if (r > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) fold[(r - 1) * TPR * 8 + i * TPR + t] = dw[j][i];
      }
      __syncthreads();
      if (r > 0) continue;
#pragma unroll
      for (int q = 0; q < kRows - 1; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] += fold[q * TPR * 8 + i * TPR + t];
    }
    if (seg < nseg) {
      Vec8<0> o;
      o.set(dw[j]);
      o.store<false>(a.partial, (int64_t)blockIdx.x * a.K + 8 * seg);
    }
  }
}

// out[k] = sum over r of partial[r][k]: 8 lanes x 4 columns by 128 row groups per workgroup, whose
// sums are added in order.
__global__ __launch_bounds__(1024) void k_sum_rows(const float *__restrict__ partial, int rows, int64_t K,
                                                   float *__restrict__ out) {
  __shared__ f32x4 part[128][8];
  const int q = threadIdx.x & 7, r0 = threadIdx.x >> 3;
  const int64_t k = (int64_t)blockIdx.x * 32 + 4 * q;
  f32x4 v = {0, 0, 0, 0};
#pragma unroll 4
  for (int r = r0; r < rows; r += 128) v += *reinterpret_cast<const f32x4 *>(partial + (int64_t)r * K + k);
  part[r0][q] = v;
  __syncthreads();
  if (r0 < 8) {
    v = part[r0][q];
#pragma unroll
    for (int i = 1; i < 16; ++i) v += part[r0 + 8 * i][q];
    part[r0][q] = v;
  }
  __syncthreads();
  if (r0 == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += part[i][q];
    *reinterpret_cast<f32x4 *>(out + k) = v;
  }
}

// ---- launchers --------------------------------------------------------------------------------------

namespace {

int norm_grid(int64_t M, int rows, int cap) {
  const int64_t g = (M + rows - 1) / rows;
  return (int)(g < cap ? g : cap);
}

// Streaming stores from 8 MB of results on (4096 x 1152 bf16: 7.8 us and 10.2; 16384 x 8192: 163 and 180);
// below they cost time (512 x 4096: 5.5 us and 5.2).
bool streams(int64_t bytes) { return bytes > (int64_t(8) << 20); }

template <int DT, int TPR, int NV>
hipError_t norm_nv(const NormArgs &a, hipStream_t s) {
  constexpr int B = TPR < 256 ? 256 : TPR;
  const int grid = norm_grid(a.M, B / TPR, 2048);
  const int64_t per = (a.h ? (DT == 0 ? 4 : 2) : 0) + (a.codes ? 1 : 0) + (a.y ? (a.y_dtype == 0 ? 4 : 2) : 0);
  if (streams(per * a.M * a.K)) k_rmsnorm<DT, TPR, NV, true><<<grid, B, 0, s>>>(a);
  else k_rmsnorm<DT, TPR, NV, false><<<grid, B, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT, int TPR>
hipError_t norm_tpr(const NormArgs &a, hipStream_t s) {
  switch ((a.K / 8 + TPR - 1) / TPR) {
    case 1: return norm_nv<DT, TPR, 1>(a, s);
    case 2: return norm_nv<DT, TPR, 2>(a, s);
    case 3: return norm_nv<DT, TPR, 3>(a, s);
    default: return norm_nv<DT, TPR, 4>(a, s);
  }
}

template <int DT, int TPR, int NV>
hipError_t norm_grad_nv(const NormGradArgs &a, int grid, hipStream_t s) {
  constexpr int B = TPR < 256 ? 256 : TPR;
  if (streams(a.M * a.K * (DT == 0 ? 4 : 2))) k_rmsnorm_backward<DT, TPR, NV, true><<<grid, B, 0, s>>>(a);
  else k_rmsnorm_backward<DT, TPR, NV, false><<<grid, B, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT, int TPR>
hipError_t norm_grad_tpr(const NormGradArgs &a, int grid, hipStream_t s) {
  switch ((a.K / 8 + TPR - 1) / TPR) {
    case 1: return norm_grad_nv<DT, TPR, 1>(a, grid, s);
    case 2: return norm_grad_nv<DT, TPR, 2>(a, grid, s);
    case 3: return norm_grad_nv<DT, TPR, 3>(a, grid, s);
    default: return norm_grad_nv<DT, TPR, 4>(a, grid, s);
  }
}

// A wave to a row where the row fits its registers; else a workgroup of 256, or, where K is larger or the
// rows are too few to fill the chip, of 1024 (one row of 4608: 3.7 us and 3.9).
int threads_per_row(int64_t M, int64_t K) { return K <= 2048 ? 64 : K <= 8192 && M > 256 ? 256 : 1024; }

}  // namespace

int norm_grad_rows(int64_t M, int64_t K) {
  // One workgroup per CU, two where each then still has eight turns: fewer leave CUs idle, more write and
  // add more partial rows (4096 x 1152: 128, 256, 512, 1024 workgroups 15.9, 13.2, 13.7, 17.6 us; 10240 x
  // 4608: 102, 71.8, 70.2, 74.6; 512 x 4096: 10.9, 10.5, 13.7).
  const int64_t turns = threads_per_row(M, K) == 64 ? (M + 3) / 4 : M;
  return (int)(turns < 256 ? turns : turns < 8 * 256 ? 256 : turns < 8 * 512 ? turns / 8 : 512);
}

hipError_t launch_rmsnorm(const NormArgs &a, hipStream_t s) {
  const int tpr = threads_per_row(a.M, a.K);
  if (a.dtype == 0)
    return tpr == 64 ? norm_tpr<0, 64>(a, s) : tpr == 256 ? norm_tpr<0, 256>(a, s) : norm_tpr<0, 1024>(a, s);
  return tpr == 64 ? norm_tpr<1, 64>(a, s) : tpr == 256 ? norm_tpr<1, 256>(a, s) : norm_tpr<1, 1024>(a, s);
}

hipError_t launch_rmsnorm_backward(const NormGradArgs &a, float *dweight, hipStream_t s) {
  const int tpr = threads_per_row(a.M, a.K), grid = norm_grad_rows(a.M, a.K);
  if (grid > 0) {
    hipError_t e;
    if (a.dtype == 0)
      e = tpr == 64 ? norm_grad_tpr<0, 64>(a, grid, s) : tpr == 256 ? norm_grad_tpr<0, 256>(a, grid, s)
                                                                    : norm_grad_tpr<0, 1024>(a, grid, s);
    else
      e = tpr == 64 ? norm_grad_tpr<1, 64>(a, grid, s) : tpr == 256 ? norm_grad_tpr<1, 256>(a, grid, s)
                                                                    : norm_grad_tpr<1, 1024>(a, grid, s);
    if (e != hipSuccess) return e;
  }
  if (!dweight) return hipSuccess;
  k_sum_rows<<<(unsigned)(a.K / 32), 1024, 0, s>>>(a.partial, grid, a.K, dweight);
  return hipGetLastError();
}

}  // namespace nvfp4
