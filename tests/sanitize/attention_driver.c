/* Host-side checks of the C ABI's attention calls under AddressSanitizer and UndefinedBehaviorSanitizer, as
 * mx8_driver.c does for the 8-bit path: fake, never dereferenced device pointers and extreme sizes; without a GPU every
 * call ends at validation or at the device check. */
#include <stdint.h>
#include <stdio.h>

#include "nvfp4.h"

#define P(i) ((void *)(uintptr_t)(0x1000000ull * (i)))
#define I(i) ((const int32_t *)P(i))
#define U8(i) ((uint8_t *)P(i))
#define F(i) ((float *)P(i))

static int stops(nvfp4_status_t s) { return s == NVFP4_ERR_HIP || s == NVFP4_ERR_DEVICE; }

int main(void) {
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 2, 8, 16, 64, 4096, (int64_t)1 << 20, (int64_t)1 << 31, (int64_t)1 << 40,
                           (int64_t)1 << 62, INT64_MAX};
  const int n = (int)(sizeof(sizes) / sizeof(sizes[0]));
  long valid = 0;
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      for (int k = 0; k < n; ++k) {
        const int64_t a = sizes[i], b = sizes[j], c = sizes[k];
        for (int u = 0; u < n; ++u) {
          const int64_t d = sizes[u];
          (void)nvfp4_attention_workspace_bytes(a, b, c, d, 64, 1);
          (void)nvfp4_attention_backward_workspace_bytes(a, b, c, d, 64, 3);
          (void)nvfp4_attention_workspace_bytes(a, 64, 4, 2, b, c);
          (void)nvfp4_paged_attention_workspace_bytes(a, b, c, 64, d);
          (void)nvfp4_paged_attention_workspace_bytes(2, a, b, c, d);
          /* sizes, heads; pitches; sequences */
          valid += stops(nvfp4_attention(P(1), 4096, 64, P(2), 4096, 64, P(3), 4096, 64, a, b, c, d, 64, I(4), I(5), 3, 1, 0.1f,
                                         P(6), 4096, 64, F(7), P(8), SIZE_MAX, NULL));
          valid += stops(nvfp4_attention(P(1), a, b, P(2), c, d, P(3), d, c, 100, 100, 4, 2, 64, NULL, NULL, 4, 0, 0.1f, P(6), b,
                                         a, NULL, P(8), SIZE_MAX, NULL));
          valid += stops(nvfp4_attention(P(1), 4096, 64, P(2), 4096, 64, P(3), 4096, 64, a, b, 4, 2, c, NULL, NULL, d, 1, 0.1f,
                                         P(6), 4096, 64, F(7), P(8), SIZE_MAX, NULL));
          valid += stops(nvfp4_attention_backward(P(9), 4096, 64, P(1), 4096, 64, P(2), 4096, 64, P(3), 4096, 64, P(6), 4096, 64,
                                                  F(7), a, b, c, d, 64, I(4), I(5), 3, 1, 0.1f, P(10), 4096, 64, P(11), 4096, 64,
                                                  P(12), 4096, 64, P(8), SIZE_MAX, NULL));
          valid += stops(nvfp4_cache_append(P(1), a, 64, P(2), b, 64, c, d, 64, I(3), I(4), 5, P(5), U8(6), P(7), U8(8), 100, 64, I(9),
                                            20, 20, NULL));
          valid += stops(nvfp4_cache_append(P(1), 4096, 64, P(2), 4096, 64, 5, 2, 64, NULL, I(4), 5, P(5), NULL, P(7), NULL, a, b,
                                            I(9), c, d, NULL));
          valid += stops(nvfp4_paged_attention(P(1), a, 64, 5, b, c, 64, P(5), U8(6), P(7), U8(8), 100, 64, I(9), 20, 20, I(4), 0.1f,
                                               P(10), d, 64, P(11), SIZE_MAX, NULL));
          valid += stops(nvfp4_paged_attention(P(1), 4096, 64, 5, 8, 2, 64, P(5), NULL, P(7), NULL, a, b, I(9), c, d, I(4), 0.1f,
                                               P(10), 4096, 64, P(11), SIZE_MAX, NULL));
        }
      }
  if (valid == 0) return 1;
  printf("attention driver ok\n");
  return 0;
}
