// Index arithmetic of packed sequences and of the paged cache, for host and device: where device data (offsets,
// lengths, page tables) becomes rows, it is taken into the arrays here, whatever it holds.
#pragma once
#include <stdint.h>

#ifdef __HIPCC__
#define NVFP4_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define NVFP4_HOST_DEVICE inline
#endif

namespace nvfp4 {

// Rows of a sequence.
struct SeqRows {
  int begin, n;
};
NVFP4_HOST_DEVICE int clamp_row(int row, int T) { return row < 0 ? 0 : row > T ? T : row; }
// Sequence b of offsets cu [B + 1] (null: equal sequences of `per` rows): inside [0, T], n >= 0.
NVFP4_HOST_DEVICE SeqRows seq_rows(const int32_t *cu, int b, int T, int per) {
  if (!cu) return {b * per, per};
  const int lo = clamp_row(cu[b], T), hi = clamp_row(cu[b + 1], T);
  return {lo, hi > lo ? hi - lo : 0};
}
// Rows before the first sequence, and up to the last one's end: where the offsets ascend, the sequences hold the rows
// between, each row once, and blocks find every one.
NVFP4_HOST_DEVICE int rows_before(const int32_t *cu, int T) { return cu ? clamp_row(cu[0], T) : 0; }
NVFP4_HOST_DEVICE int rows_in_use(const int32_t *cu, int B, int T) { return cu ? clamp_row(cu[B], T) : T; }
// Whether they descend at sequence b.
NVFP4_HOST_DEVICE bool descends(const int32_t *cu, int b, int T) { return clamp_row(cu[b], T) > clamp_row(cu[b + 1], T); }

// Blocks of blk rows of packed sequences are numbered by slots: sequence b's begin at cu[b] / blk + b, which
// leaves it at least ceil(n / blk) of them, so a block finds its sequence by a search, and nobody has to
// know the lengths on the host.  (Equal sequences: per / blk rounded up for each.)
NVFP4_HOST_DEVICE int first_slot(const int32_t *cu, int b, int T, int blk) { return clamp_row(cu[b], T) / blk + b; }
inline int64_t attention_slots(int64_t T, int64_t B, bool packed, int blk) {
  return packed ? T / blk + B : B * ((T / (B > 0 ? B : 1) + blk - 1) / blk);
}

// Position of token t in its sequence, as appending counts it: the sequence ends with the call's last token of it.
// -1: no sequence's.  cu null: token t is sequence t's last one.
struct TokenPlace {
  int b;
  int64_t pos;
};
NVFP4_HOST_DEVICE TokenPlace token_place(const int32_t *cu, const int32_t *lengths, int B, int t) {
  if (!cu) return {t, (int64_t)lengths[t] - 1};
  int lo = 0, hi = B;  // the last b with cu[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int64_t behind = (int64_t)cu[lo + 1] - t;  // tokens of the sequence from this one on
  if (behind <= 0 || cu[lo] > t) return {lo, -1};
  return {lo, (int64_t)lengths[lo] - behind};
}
// Page of position pos of a sequence's table row, or -1.
NVFP4_HOST_DEVICE int page_of(const int32_t *row, int64_t pos, int shift, int max_pages, int pages) {
  if (pos < 0 || (pos >> shift) >= max_pages) return -1;
  const int page = row[pos >> shift];
  return page >= 0 && page < pages ? page : -1;
}
// Row (of a head's D values) of the cache at position pos on that page.
NVFP4_HOST_DEVICE int64_t cache_row(int page, int head, int Hkv, int64_t pos, int shift) {
  return (((int64_t)page * Hkv + head) << shift) + (pos & (((int64_t)1 << shift) - 1));
}
// Tokens of a sequence, inside its table's room.
NVFP4_HOST_DEVICE int tokens_of(int length, int shift, int max_pages) {
  const int64_t room = (int64_t)max_pages << shift;
  return length < 0 ? 0 : (int64_t)length < room ? length : (int)room;
}

}  // namespace nvfp4
