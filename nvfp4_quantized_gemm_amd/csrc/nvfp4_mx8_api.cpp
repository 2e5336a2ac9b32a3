// libnvfp4 C ABI, the 8-bit activation path: MXFP8 quantize, RMS norm, W4A8 product, rotary positions.
// Semantics and layouts are documented in include/nvfp4.h.
#include "../../include/nvfp4.h"

#include "api_checks.hpp"
#include "launch.hpp"

using namespace nvfp4;

extern "C" {

nvfp4_status_t nvfp4_mx8_quantize(const void *x, nvfp4_dtype_t x_dtype, int64_t M, int64_t K, int64_t ld_x,
                                  uint8_t *codes, uint8_t *scales, void *stream) {
  if (!valid_dtype(x_dtype)) return NVFP4_ERR_DTYPE;
  nvfp4_status_t st = check_mx_mk(M, K);
  if (st != NVFP4_OK) return st;
  if (M == 0) return NVFP4_OK;
  if (!x || !codes || !scales) return NVFP4_ERR_NULL;
  if ((st = check_pitch(ld_x, M, K)) != NVFP4_OK) return st;
  if (!aligned(x, 16) || ((ld_x * elem_size(x_dtype)) % 16) != 0 || !aligned(codes, 16)) return NVFP4_ERR_ALIGN;
  if ((st = check_device()) != NVFP4_OK) return st;
  st = debug_scan(stream, {finite_values(x, x_dtype, M, K, ld_x)});
  if (st != NVFP4_OK) return st;
  return hip_status(launch_mx8_quantize(x, (int)x_dtype, M, K, ld_x, codes, scales, static_cast<hipStream_t>(stream)));
}

nvfp4_status_t nvfp4_rmsnorm(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual,
                             nvfp4_dtype_t dtype, int64_t M, int64_t K, const void *weight,
                             nvfp4_dtype_t weight_dtype, float eps, void *h, int64_t ld_h, uint8_t *codes,
                             uint8_t *scales, void *y, nvfp4_dtype_t y_dtype, int64_t ld_y, int fake_quantize,
                             float *inv_rms, void *stream) {
  if (!valid_dtype(dtype) || (weight && !valid_dtype(weight_dtype)) || (y && !valid_dtype(y_dtype)))
    return NVFP4_ERR_DTYPE;
  nvfp4_status_t st = check_mx_mk(M, K);
  if (st != NVFP4_OK) return st;
  if (K > kNormMaxK) return NVFP4_ERR_SHAPE;
  if (!(eps > 0.0f) || !(eps <= 3.0e38f)) return NVFP4_ERR_MODE;
  if ((codes == nullptr) != (scales == nullptr)) return NVFP4_ERR_NULL;
  if (M == 0) return NVFP4_OK;
  if (!x || (!codes && !y)) return NVFP4_ERR_NULL;
  if ((st = check_pitch(ld_x, M, K)) != NVFP4_OK || (residual && (st = check_pitch(ld_residual, M, K)) != NVFP4_OK) ||
      (h && (st = check_pitch(ld_h, M, K)) != NVFP4_OK) || (y && (st = check_pitch(ld_y, M, K)) != NVFP4_OK))
    return st;
  if (!rows_aligned(x, ld_x, dtype) || !rows_aligned(residual, ld_residual, dtype) || !rows_aligned(h, ld_h, dtype) ||
      !rows_aligned(y, ld_y, y_dtype) || !aligned(weight, 16) || !aligned(codes, 16) || !aligned(inv_rms, 4))
    return NVFP4_ERR_ALIGN;
  if (!in_place_fits(h, ld_h, dtype, x, ld_x, dtype, M) || !in_place_fits(h, ld_h, dtype, residual, ld_residual, dtype, M) ||
      !in_place_fits(y, ld_y, y_dtype, x, ld_x, dtype, M) ||
      !in_place_fits(y, ld_y, y_dtype, residual, ld_residual, dtype, M))
    return NVFP4_ERR_STRIDE;
  if ((st = check_device()) != NVFP4_OK) return st;
  st = debug_scan(stream, {finite_values(x, dtype, M, K, ld_x), finite_values(residual, dtype, M, K, ld_residual),
                           finite_values(weight, weight_dtype, 1, K, K)});
  if (st != NVFP4_OK) return st;
  const NormArgs a{x, residual, (int)dtype, M, K, ld_x, ld_residual, weight, (int)weight_dtype, eps, 1.0f / (float)K,
                   h, ld_h, codes, scales, y, (int)y_dtype, ld_y, fake_quantize != 0 && y, inv_rms};
  return hip_status(launch_rmsnorm(a, static_cast<hipStream_t>(stream)));
}

size_t nvfp4_rmsnorm_backward_workspace_bytes(int64_t M, int64_t K) {
  if (check_mx_mk(M, K) != NVFP4_OK || K > kNormMaxK) return 0;
  return (size_t)norm_grad_rows(M, K) * (size_t)K * sizeof(float);
}

nvfp4_status_t nvfp4_rmsnorm_backward(const void *dy, int64_t ld_dy, const void *h, int64_t ld_h, const void *dh,
                                      int64_t ld_dh, nvfp4_dtype_t dtype, int64_t M, int64_t K, const void *weight,
                                      nvfp4_dtype_t weight_dtype, const float *inv_rms, void *dx, int64_t ld_dx,
                                      float *dweight, void *workspace, size_t workspace_bytes, void *stream) {
  if (!valid_dtype(dtype) || (weight && !valid_dtype(weight_dtype))) return NVFP4_ERR_DTYPE;
  nvfp4_status_t st = check_mx_mk(M, K);
  if (st != NVFP4_OK) return st;
  if (K > kNormMaxK) return NVFP4_ERR_SHAPE;
  if (M == 0 && !dweight) return NVFP4_OK;
  if (M > 0) {
    if (!dy || !h || !inv_rms || !dx) return NVFP4_ERR_NULL;
    if ((st = check_pitch(ld_dy, M, K)) != NVFP4_OK || (st = check_pitch(ld_h, M, K)) != NVFP4_OK ||
        (st = check_pitch(ld_dx, M, K)) != NVFP4_OK || (dh && (st = check_pitch(ld_dh, M, K)) != NVFP4_OK))
      return st;
    if (!rows_aligned(dy, ld_dy, dtype) || !rows_aligned(h, ld_h, dtype) || !rows_aligned(dh, ld_dh, dtype) ||
        !rows_aligned(dx, ld_dx, dtype) || !aligned(weight, 16) || !aligned(inv_rms, 4))
      return NVFP4_ERR_ALIGN;
    if (!in_place_fits(dx, ld_dx, dtype, dy, ld_dy, dtype, M) || !in_place_fits(dx, ld_dx, dtype, h, ld_h, dtype, M) ||
        !in_place_fits(dx, ld_dx, dtype, dh, ld_dh, dtype, M))
      return NVFP4_ERR_STRIDE;
  }
  if (dweight) {
    if (M > 0 && (!workspace || workspace_bytes < nvfp4_rmsnorm_backward_workspace_bytes(M, K)))
      return NVFP4_ERR_WORKSPACE;
    if (!aligned(dweight, 16) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  }
  if ((st = check_device()) != NVFP4_OK) return st;
  st = debug_scan(stream, {finite_values(dy, dtype, M, K, ld_dy), finite_values(h, dtype, M, K, ld_h),
                           finite_values(dh, dtype, M, K, ld_dh), finite_values(weight, weight_dtype, 1, K, K),
                           finite_values(inv_rms, NVFP4_F32, 1, M, M)});
  if (st != NVFP4_OK) return st;
  const NormGradArgs a{dy, h, dh, (int)dtype, M, K, ld_dy, ld_h, ld_dh, weight, (int)weight_dtype, inv_rms,
                       1.0f / (float)K, dx, ld_dx, dweight ? static_cast<float *>(workspace) : nullptr};
  return hip_status(launch_rmsnorm_backward(a, dweight, static_cast<hipStream_t>(stream)));
}

nvfp4_status_t nvfp4_mx_gemm_w4a8(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b, const uint8_t *b_scales,
                                  int64_t M, int64_t N, int64_t K, void *c, nvfp4_dtype_t c_dtype, int64_t ldc,
                                  void *stream) {
  if (!valid_dtype(c_dtype)) return NVFP4_ERR_DTYPE;
  if (N < 0) return NVFP4_ERR_SHAPE;
  nvfp4_status_t st = check_mx_mk(M, K);
  if (st != NVFP4_OK) return st;
  st = check_mx_mk(N, K);
  if (st != NVFP4_OK) return st;
  if (M >= (1 << 30) || N >= (1 << 30) || K >= (1 << 30) || (N > 0 && M > kMaxElems / N)) return NVFP4_ERR_SHAPE;
  if (M == 0 || N == 0) return NVFP4_OK;
  if (!a || !a_scales || !b || !b_scales || !c) return NVFP4_ERR_NULL;
  if ((st = check_pitch(ldc, M, N)) != NVFP4_OK) return st;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4) || !aligned(c, 16))
    return NVFP4_ERR_ALIGN;
  if ((st = check_device()) != NVFP4_OK) return st;
  st = debug_scan(stream, {scale_bytes(a, kCheckE4M3, M, K, K), scale_bytes(a_scales, kCheckE8M0, M, K / 32, K / 32),
                           scale_bytes(b_scales, kCheckE8M0, N, K / 32, K / 32)});
  if (st != NVFP4_OK) return st;
  return hip_status(launch_w4a8({a, a_scales, b, b_scales, M, N, K, c, (int)c_dtype, ldc},
                                static_cast<hipStream_t>(stream)));
}

nvfp4_status_t nvfp4_rope_axes(const void *x, nvfp4_dtype_t dtype, int64_t T, int64_t H, int64_t D, int64_t ld_token,
                               int64_t ld_head, const float *positions, int n_axes, const int32_t *axis_dims,
                               const float *inv_freq, nvfp4_rope_layout_t layout, int inverse, void *y,
                               int64_t ldy_token, int64_t ldy_head, void *stream) {
  if (!valid_dtype(dtype)) return NVFP4_ERR_DTYPE;
  if (layout != NVFP4_ROPE_PAIRS && layout != NVFP4_ROPE_HALVES) return NVFP4_ERR_MODE;
  if (T < 0 || H < 0 || D < 8 || D % 8 != 0 || D > kRopeMaxD || H > (1 << 20) || T >= ((int64_t)1 << 31) ||
      n_axes < 1 || n_axes > kRopeMaxAxes)
    return NVFP4_ERR_SHAPE;
  if (!axis_dims) return NVFP4_ERR_NULL;
  RopeArgs a{};
  int64_t dims = 0;
  for (int i = 0; i < n_axes; ++i) {
    if (axis_dims[i] < 0 || axis_dims[i] % 2 != 0 || axis_dims[i] > D) return NVFP4_ERR_SHAPE;
    dims += axis_dims[i];
    a.pair_end[i] = (int)(dims / 2);
  }
  if (dims > D) return NVFP4_ERR_SHAPE;
  if (T == 0 || H == 0) return NVFP4_OK;
  if (!x || !y || !positions || (dims > 0 && !inv_freq)) return NVFP4_ERR_NULL;
  if (!head_rows_fit(T, H, D, ld_token, ld_head, false) || !head_rows_fit(T, H, D, ldy_token, ldy_head, true))
    return NVFP4_ERR_STRIDE;
  if (x == y && (ld_token != ldy_token || ld_head != ldy_head)) return NVFP4_ERR_STRIDE;
  if (!rows_aligned(x, ld_token, dtype) || !rows_aligned(x, ld_head, dtype) || !rows_aligned(y, ldy_token, dtype) ||
      !rows_aligned(y, ldy_head, dtype) || !aligned(positions, 4) || !aligned(inv_freq, 4))
    return NVFP4_ERR_ALIGN;
  nvfp4_status_t st = check_device();
  if (st != NVFP4_OK) return st;
  st = debug_scan(stream, {finite_values(positions, NVFP4_F32, 1, T * n_axes, T * n_axes),
                           finite_values(inv_freq, NVFP4_F32, 1, dims / 2, dims / 2)});
  if (st != NVFP4_OK) return st;
  a.x = x;
  a.y = y;
  a.dtype = (int)dtype;
  a.T = T;
  a.ld_t = ld_token;
  a.ld_h = ld_head;
  a.ldy_t = ldy_token;
  a.ldy_h = ldy_head;
  a.H = (int)H;
  a.D = (int)D;
  a.n_axes = n_axes;
  a.pairs = (int)(dims / 2);
  a.halves = layout == NVFP4_ROPE_HALVES;
  a.inverse = inverse != 0;
  a.positions = positions;
  a.inv_freq = inv_freq;
  return hip_status(launch_rope(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
