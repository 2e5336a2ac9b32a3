// The index arithmetic that the attention kernels take device data through (csrc/sequence_index.hpp), on the CPU under
// AddressSanitizer and UndefinedBehaviorSanitizer: with any offsets, lengths and tables the rows stay inside their arrays,
// and with sensible ones every row has one block and every token its place.
#include <stdio.h>
#include <stdlib.h>

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

static uint32_t seed = 12345;
static uint32_t next() { return seed = seed * 1664525u + 1013904223u; }
static const int32_t odd[] = {INT32_MIN, INT32_MIN + 1, -7, -1, 0, 1, 5, 63, 100, 127, 128, 1 << 20, INT32_MAX - 1, INT32_MAX};
static int32_t any() { return next() % 3 ? odd[next() % 14] : (int32_t)next(); }

// what the kernels' search finds: the last b whose first slot is not past `slot`
static int find(const int32_t *cu, int B, int T, int blk, int slot) {
  int lo = 0, len = B;
  while (len > 1) {
    const int step = (len + 63) >> 6;
    int n = 0;
    for (int lane = 0; lane < 64; ++lane)
      if (lane * step < len) n += first_slot(cu, lo + lane * step, T, blk) <= slot;
    n = n < 1 ? 1 : n;
    lo += (n - 1) * step;
    len = step < len - (n - 1) * step ? step : len - (n - 1) * step;
  }
  return lo;
}

int main() {
  for (int round = 0; round < 4000; ++round) {  // anything
    const int B = 1 + next() % 200, T = (int)(next() % 1000);
    std::vector<int32_t> cu(B + 1), lengths(B);
    for (auto &x : cu) x = any();
    for (auto &x : lengths) x = any();
    for (int b = 0; b < B; ++b) {
      const SeqRows s = seq_rows(cu.data(), b, T, 0);
      EXPECT(s.begin >= 0 && s.n >= 0 && s.begin <= T && s.n <= T - s.begin);
    }
    EXPECT(rows_in_use(cu.data(), B, T) >= 0 && rows_in_use(cu.data(), B, T) <= T);
    for (int slot = 0; slot < (int)attention_slots(T, B, true, 128); ++slot) {
      const int b = find(cu.data(), B, T, 128, slot);
      EXPECT(b >= 0 && b < B);
    }
    const int shift = 4 + next() % 5, most = (int)(next() % 6), pages = (int)(next() % 9), Hkv = 1 + next() % 4;
    std::vector<int32_t> table(most + 1);
    for (auto &x : table) x = next() % 2 ? (int32_t)(next() % 9) : any();
    for (int t = 0; t < T; t += 1 + T / 50) {
      const TokenPlace p = token_place(cu.data(), lengths.data(), B, t);
      EXPECT(p.b >= 0 && p.b < B);
      const int page = page_of(table.data(), p.pos, shift, most, pages);
      EXPECT(page == -1 || (page >= 0 && page < pages));
      if (page >= 0) EXPECT(cache_row(page, Hkv - 1, Hkv, p.pos, shift) < ((int64_t)pages * Hkv << shift));
    }
    for (int b = 0; b < B; ++b) {
      const int n = tokens_of(lengths[b], shift, most);
      EXPECT(n >= 0 && n <= most << shift);
      for (int pos = 0; pos < n; pos += 16) page_of(table.data(), pos, shift, most, pages);
    }
  }
  for (int round = 0; round < 2000; ++round) {  // ascending offsets: every row of every sequence in one block
    const int B = 1 + next() % 150, blk = 128;
    std::vector<int32_t> cu(B + 1, 0), lengths(B);
    for (int b = 0; b < B; ++b) cu[b + 1] = cu[b] + (next() % 3 ? (int)(next() % 40) : (int)(next() % 700) * (next() % 2));
    const int T = cu[B] + (int)(next() % 50);
    std::vector<char> seen(T, 0);
    for (int slot = 0; slot < (int)attention_slots(T, B, true, blk); ++slot) {
      const int b = find(cu.data(), B, T, blk, slot), i = slot - first_slot(cu.data(), b, T, blk);
      const SeqRows s = seq_rows(cu.data(), b, T, 0);
      EXPECT(i >= 0);
      for (int r = i * blk; r < (i + 1) * blk && r < s.n; ++r) EXPECT(!seen[s.begin + r]++);
    }
    for (int t = 0; t < T; ++t) EXPECT(seen[t] == (t < cu[B]));
    for (int b = 0; b < B; ++b) lengths[b] = cu[b + 1] - cu[b] + (int)(next() % 100);
    for (int b = 0; b < B; ++b)
      for (int t = cu[b]; t < cu[b + 1]; ++t) {
        const TokenPlace p = token_place(cu.data(), lengths.data(), B, t);
        EXPECT(p.b == b && p.pos == lengths[b] - (cu[b + 1] - t));
      }
    for (int t = cu[B]; t < T; ++t) EXPECT(token_place(cu.data(), lengths.data(), B, t).pos < 0);
  }
  if (failures) return 1;
  printf("sequence index driver ok\n");
  return 0;
}
