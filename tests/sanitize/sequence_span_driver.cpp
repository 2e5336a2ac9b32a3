// Which rows the kernels that join several workgroups' sums may take (csrc/sequence_index.hpp), on the CPU under
// AddressSanitizer and UndefinedBehaviorSanitizer: with offsets that ascend, from any first one on, those that a block of some
// sequence holds and no other; with offsets that descend somewhere, none.
#include <stdio.h>

#include <vector>

#include "sequence_index.hpp"

using namespace nvfp4;

static int failures = 0;
#define EXPECT(cond)                                              \
  do {                                                            \
    if (!(cond)) {                                                \
      fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #cond); \
      ++failures;                                                 \
    }                                                             \
  } while (0)

static uint32_t seed = 2468;
static uint32_t next() { return seed = seed * 1664525u + 1013904223u; }

int main() {
  const int blk = 128;
  for (int round = 0; round < 3000; ++round) {
    const int B = 1 + next() % 60, T = (int)(next() % 3000);
    std::vector<int32_t> cu(B + 1);
    cu[0] = (int)(next() % 900) - 100;
    for (int b = 0; b < B; ++b) cu[b + 1] = cu[b] + (next() % 3 ? (int)(next() % 60) : (int)(next() % 600));
    if (round % 3 == 0) cu[next() % (B + 1)] = (int)(next() % 6000) - 1500;
    bool down = false;
    for (int b = 0; b < B; ++b) {
      down |= descends(cu.data(), b, T);
      EXPECT(descends(cu.data(), b, T) == (clamp_row(cu[b], T) > clamp_row(cu[b + 1], T)));
    }
    if (down) continue;
    std::vector<int> held(T, 0);  // by the block of the last sequence whose first slot is not past it
    for (int slot = 0; slot < (int)attention_slots(T, B, true, blk); ++slot) {
      int b = 0;
      while (b + 1 < B && first_slot(cu.data(), b + 1, T, blk) <= slot) ++b;
      const int i = slot - first_slot(cu.data(), b, T, blk);
      const SeqRows s = seq_rows(cu.data(), b, T, 0);
      for (int r = i * blk; i >= 0 && r < (i + 1) * blk && r < s.n; ++r) ++held[s.begin + r];
    }
    const int from = rows_before(cu.data(), T), to = rows_in_use(cu.data(), B, T);
    for (int t = 0; t < T; ++t) EXPECT(held[t] == (t >= from && t < to));
  }
  EXPECT(rows_before(nullptr, 7) == 0 && rows_in_use(nullptr, 3, 7) == 7);
  if (failures) return 1;
  printf("sequence span driver ok\n");
  return 0;
}
