// MXFP8 quantize, and the product of MXFP8 activations with MXFP4 weights (W4A8), for gfx950.
//
// Y[m][n] = sum_k a[m][k] Xa[m][k / 32] b[n][k] Xb[n][k / 32]: E4M3 codes times E2M1 codes under
// E8M0 scales, exact products, fp32 sums.
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

hipError_t launch_w4a8(const W4A8Args &g, hipStream_t s) {
  int64_t grid = (g.M * g.N + 255) / 256;
  if (grid > 65536) grid = 65536;
  if (g.out_dtype == 0)
    k_w4a8_generic<0><<<(unsigned)grid, 256, 0, s>>>(g.a, g.as, g.b, g.bs, g.M, g.N, g.K, g.c, g.ldc);
  else
    k_w4a8_generic<1><<<(unsigned)grid, 256, 0, s>>>(g.a, g.as, g.b, g.bs, g.M, g.N, g.K, g.c, g.ldc);
  return hipGetLastError();
}

}  // namespace nvfp4
