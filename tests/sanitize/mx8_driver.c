/* Host-side checks of the C ABI's 8-bit activation path under AddressSanitizer and
 * UndefinedBehaviorSanitizer, as abi_driver.c does for the rest: fake, never dereferenced device
 * pointers and extreme sizes; without a GPU every call ends at validation or at the device check. */
#include <stdint.h>
#include <stdio.h>

#include "nvfp4.h"

static int failures = 0;
#define EXPECT(cond)                                              \
  do {                                                            \
    if (!(cond)) {                                                \
      fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #cond); \
      ++failures;                                                 \
    }                                                             \
  } while (0)

#define P ((void *)0x10000)
#define Q ((void *)0x90000000)
#define U8(p) ((uint8_t *)(p))
#define F(p) ((float *)(p))

static int stops(nvfp4_status_t s) { return s == NVFP4_ERR_HIP || s == NVFP4_ERR_DEVICE; }
static int refused(nvfp4_status_t s) { return s != NVFP4_OK && !stops(s); }

int main(void) {
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 31, 32, 33, 4096, (int64_t)1 << 31, (int64_t)1 << 40, (int64_t)1 << 62, INT64_MAX};
  const int n = (int)(sizeof(sizes) / sizeof(sizes[0]));
  const int32_t dims[4] = {32, 16, 8, 8}, odd[1] = {31}, most[2] = {INT32_MAX, INT32_MAX}, least[1] = {INT32_MIN};
  int valid = 0;
  for (int i = 0; i < n; ++i) {
    for (int j = 0; j < n; ++j) {
      const int64_t M = sizes[i], K = sizes[j];
      (void)nvfp4_rmsnorm_backward_workspace_bytes(M, K);
      for (int k = 0; k < n; ++k) {
        const int64_t ld = sizes[k];
        valid += stops(nvfp4_mx8_quantize(P, NVFP4_BF16, M, K, ld, U8(P), U8(P), NULL));
        valid += stops(nvfp4_rmsnorm(P, ld, P, K, NVFP4_F32, M, K, P, NVFP4_BF16, 1e-6f, P, ld, U8(P), U8(P), P, NVFP4_F32,
                                     ld, 1, F(P), NULL));
        valid += stops(nvfp4_rmsnorm_backward(P, ld, P, ld, P, K, NVFP4_F32, M, K, P, NVFP4_F32, F(P), P, ld, F(P), P,
                                              SIZE_MAX, NULL));
        valid += stops(nvfp4_mx_gemm_w4a8(U8(P), U8(P), U8(P), U8(P), M, ld, K, P, NVFP4_BF16, ld, NULL));
        valid += stops(nvfp4_rope_axes(P, NVFP4_BF16, M, K, 64, ld, 64, F(P), 3, dims, F(P), NVFP4_ROPE_PAIRS, 0, Q, ld, 64,
                                       NULL));
        valid += stops(nvfp4_rope_axes(P, NVFP4_F32, M, 3, K, ld, K, F(P), 4, dims, F(P), NVFP4_ROPE_HALVES, 1, Q, ld, K,
                                       NULL));
      }
    }
  }
  EXPECT(valid > 0);
  EXPECT(refused(nvfp4_rope_axes(P, NVFP4_F32, 4, 3, 64, 192, 64, F(P), 1, odd, F(P), NVFP4_ROPE_PAIRS, 0, Q, 192, 64, NULL)));
  EXPECT(refused(nvfp4_rope_axes(P, NVFP4_F32, 4, 3, 64, 192, 64, F(P), 2, most, F(P), NVFP4_ROPE_PAIRS, 0, Q, 192, 64, NULL)));
  EXPECT(refused(nvfp4_rope_axes(P, NVFP4_F32, 4, 3, 64, 192, 64, F(P), 1, least, F(P), NVFP4_ROPE_PAIRS, 0, Q, 192, 64, NULL)));
  EXPECT(refused(nvfp4_rope_axes(P, NVFP4_F32, 4, 3, 64, 192, 64, F(P), 1, dims, F(P), (nvfp4_rope_layout_t)7, 0, Q, 192, 64,
                                 NULL)));
  EXPECT(refused(nvfp4_mx8_quantize(P, (nvfp4_dtype_t)-5, 4, 64, 64, U8(P), U8(P), NULL)));
  EXPECT(nvfp4_rmsnorm_backward_workspace_bytes(INT64_MAX, 64) == 0);
  EXPECT(nvfp4_rmsnorm_backward_workspace_bytes(4096, 1152) > 0);
  if (failures) return 1;
  printf("mx8 driver ok\n");
  return 0;
}
