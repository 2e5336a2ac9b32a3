// libnvfp4 C ABI, attention: whole prompts and their gradients, a paged cache and single tokens over it.
// Semantics and layouts are documented in include/nvfp4.h.
#include "../../include/nvfp4.h"

#include <cmath>

#include "api_checks.hpp"
#include "launch.hpp"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxCapacity = (int64_t)1 << 30;  // a sequence's positions, and a step past them, fit 32 bits
constexpr int64_t kMaxPitch = (int64_t)1 << 23;  // offsets inside a tile (128 rows at most) fit 31 bits

struct Heads {  // [T][H][D] bf16 at token and head pitches
  const void *p;
  int64_t T, H, ld_t, ld_h;
};

nvfp4_status_t check_heads(const Heads &x, int64_t D, bool written) {
  if (x.T == 0 || x.H == 0) return NVFP4_OK;
  if (!x.p) return NVFP4_ERR_NULL;
  if ((x.T > 1 && x.ld_t < D) || x.ld_t >= kMaxPitch || !head_rows_fit(x.T, x.H, D, x.ld_t, x.ld_h, written)) return NVFP4_ERR_STRIDE;
  if (!rows_aligned(x.p, x.ld_t, NVFP4_BF16) || !rows_aligned(x.p, x.ld_h, NVFP4_BF16)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}
// the token pitch that the kernels bound their rows by; a single token's is never used, whatever it is
int64_t row_pitch(const Heads &x, int64_t D) { return x.T > 1 ? x.ld_t : D; }
// two arrays that begin at one address
bool same_place(const Heads &a, const Heads &b) { return a.T > 0 && b.T > 0 && a.p == b.p; }
// a written array at an input's address has its pitches
bool same_place_fits(const Heads &out, const Heads &in) {
  return out.p != in.p || ((out.T <= 1 || out.ld_t == in.ld_t) && (out.H <= 1 || out.ld_h == in.ld_h));
}

nvfp4_status_t check_attention_shape(int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D, const int32_t *cu_q,
                                     const int32_t *cu_k, int64_t B, float scale) {
  constexpr int64_t kRows = (int64_t)1 << 31;
  if (Tq < 0 || Tk < 0 || Tq >= kRows || Tk >= kRows || Hq < 0 || Hkv < 0 || Hq > (1 << 16) || Hkv > Hq || D < 8 ||
      D > kAttentionMaxD || D % 8 != 0 || B < 0 || B > (1 << 20) || (Hq > 0 && (Hkv == 0 || Hq % Hkv != 0)))
    return NVFP4_ERR_SHAPE;
  if ((cu_q == nullptr) != (cu_k == nullptr)) return NVFP4_ERR_NULL;
  if (!cu_q && (B > 0 ? Tq % B != 0 || Tk % B != 0 : Tq > 0 || Tk > 0)) return NVFP4_ERR_SHAPE;
  // at most a workgroup of 512 threads per head and 32 rows, and 2^32 threads
  if (((Tq > Tk ? Tq : Tk) / 32 + B + 1) * Hq >= ((int64_t)1 << 23)) return NVFP4_ERR_SHAPE;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return NVFP4_ERR_MODE;
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// the backward pass' two values per query, and whole 16 bytes
size_t backward_rows_bytes(int64_t Tq, int64_t Hq) { return (2 * sizeof(float) * (size_t)Tq * (size_t)Hq + 15) / 16 * 16; }
const int32_t *const kAnyOffsets = reinterpret_cast<const int32_t *>(16);  // a packed batch, for size queries

// The shape of a paged cache, and its arrays' extents and alignment.
nvfp4_status_t check_cache(const void *k, const uint8_t *ks, const void *v, const uint8_t *vs, int64_t pages,
                           int64_t page_size, const int32_t *table, int64_t ld_table, int64_t max_pages,
                           const int32_t *lengths, int64_t B, int64_t Hkv, int64_t D) {
  constexpr int64_t kInt = (int64_t)1 << 31;
  if (D < 8 || D > kAttentionMaxD || D % 8 != 0 || Hkv < 0 || Hkv > (1 << 16) || B < 0 || B >= (1 << 16) || pages < 0 ||
      pages >= kInt || page_size < 16 || page_size > (1 << 20) || (page_size & (page_size - 1)) != 0 || max_pages < 0 ||
      max_pages >= kMaxCapacity / page_size || (Hkv > 0 && pages > kMaxElems / (Hkv * page_size * D)))
    return NVFP4_ERR_SHAPE;
  if ((ks == nullptr) != (vs == nullptr)) return NVFP4_ERR_NULL;
  if (B == 0 || Hkv == 0) return NVFP4_OK;
  if (!lengths || (max_pages > 0 && !table) || (pages > 0 && (!k || !v))) return NVFP4_ERR_NULL;
  if (ld_table < max_pages || ld_table > kMaxElems / B) return NVFP4_ERR_STRIDE;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(table, 4) || !aligned(lengths, 4)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}
PagedCacheArgs cache_args(const void *k, const uint8_t *ks, const void *v, const uint8_t *vs, int64_t pages,
                          int64_t page_size, const int32_t *table, int64_t ld_table, int64_t max_pages,
                          const int32_t *lengths, int64_t B, int64_t Hkv, int64_t D) {
  int shift = 0;
  while (((int64_t)1 << shift) < page_size) ++shift;
  return {const_cast<void *>(k), const_cast<void *>(v), const_cast<uint8_t *>(ks), const_cast<uint8_t *>(vs), (int)pages,
          shift, (int)Hkv, (int)D, table, ld_table, (int)max_pages, lengths, (int)B};
}

}  // namespace

extern "C" {

size_t nvfp4_attention_workspace_bytes(int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D, int64_t B) {
  if (check_attention_shape(Tq, Tk, Hq, Hkv, D, kAnyOffsets, kAnyOffsets, B, 1.0f) != NVFP4_OK || Hq == 0 || B == 0) return 0;
  const int splits = attention_splits(Tq, Tk, Hq, B);
  return splits > 1 ? sizeof(float) * (size_t)splits * (size_t)Tq * (size_t)Hq * (size_t)(D + 2) : 0;
}

nvfp4_status_t nvfp4_attention(const void *q, int64_t ldq_token, int64_t ldq_head, const void *k, int64_t ldk_token,
                               int64_t ldk_head, const void *v, int64_t ldv_token, int64_t ldv_head, int64_t Tq,
                               int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D, const int32_t *cu_q,
                               const int32_t *cu_k, int64_t B, int causal, float scale, void *out, int64_t ldo_token,
                               int64_t ldo_head, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  nvfp4_status_t st = check_attention_shape(Tq, Tk, Hq, Hkv, D, cu_q, cu_k, B, scale);
  if (st != NVFP4_OK) return st;
  if (Tq == 0 || Hq == 0 || B == 0) return NVFP4_OK;
  const Heads hq{q, Tq, Hq, ldq_token, ldq_head}, hk{k, Tk, Hkv, ldk_token, ldk_head}, hv{v, Tk, Hkv, ldv_token, ldv_head},
      ho{out, Tq, Hq, ldo_token, ldo_head};
  if ((st = check_heads(hq, D, false)) != NVFP4_OK || (st = check_heads(hk, D, false)) != NVFP4_OK ||
      (st = check_heads(hv, D, false)) != NVFP4_OK || (st = check_heads(ho, D, true)) != NVFP4_OK)
    return st;
  if (!same_place_fits(ho, hq) || same_place(ho, hk) || same_place(ho, hv)) return NVFP4_ERR_STRIDE;
  const size_t need = nvfp4_attention_workspace_bytes(Tq, Tk, Hq, Hkv, D, B);
  if (need > 0 && (!workspace || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
  if (!aligned(lse, 4) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  if ((st = check_device()) != NVFP4_OK) return st;
  const AttentionArgs a{q, k, v, row_pitch(hq, D), ldq_head, row_pitch(hk, D), ldk_head, row_pitch(hv, D), ldv_head, (int)Tq, (int)Tk, (int)Hq,
                        (int)(Hq / Hkv), (int)D, (int)B, cu_q, cu_k, (int)(Tq / B), (int)(Tk / B), causal != 0, scale, out,
                        ldo_token, ldo_head, lse, attention_splits(Tq, Tk, Hq, B), static_cast<float *>(workspace)};
  return hip_status(launch_attention(a, static_cast<hipStream_t>(stream)));
}

size_t nvfp4_attention_backward_workspace_bytes(int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D, int64_t B) {
  if (check_attention_shape(Tq, Tk, Hq, Hkv, D, kAnyOffsets, kAnyOffsets, B, 1.0f) != NVFP4_OK || Hq == 0 || B == 0) return 0;
  const int dq = attention_splits(Tq, Tk, Hq, B), dkv = attention_backward_splits(Tq, Tk, Hq, Hkv, B);
  const size_t q = dq > 1 ? sizeof(float) * (size_t)dq * (size_t)Tq * (size_t)Hq * (size_t)D : 0;
  const size_t k = dkv > 1 ? 2 * sizeof(float) * (size_t)dkv * (size_t)Tk * (size_t)Hkv * (size_t)D : 0;
  return backward_rows_bytes(Tq, Hq) + (q > k ? q : k);  // one after the other
}

nvfp4_status_t nvfp4_attention_backward(const void *dout, int64_t lddo_token, int64_t lddo_head, const void *q,
                                        int64_t ldq_token, int64_t ldq_head, const void *k, int64_t ldk_token,
                                        int64_t ldk_head, const void *v, int64_t ldv_token, int64_t ldv_head,
                                        const void *out, int64_t ldo_token, int64_t ldo_head, const float *lse,
                                        int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D,
                                        const int32_t *cu_q, const int32_t *cu_k, int64_t B, int causal, float scale,
                                        void *dq, int64_t lddq_token, int64_t lddq_head, void *dk, int64_t lddk_token,
                                        int64_t lddk_head, void *dv, int64_t lddv_token, int64_t lddv_head,
                                        void *workspace, size_t workspace_bytes, void *stream) {
  nvfp4_status_t st = check_attention_shape(Tq, Tk, Hq, Hkv, D, cu_q, cu_k, B, scale);
  if (st != NVFP4_OK) return st;
  if ((Tq == 0 && Tk == 0) || Hq == 0 || B == 0) return NVFP4_OK;
  const Heads in[] = {{dout, Tq, Hq, lddo_token, lddo_head}, {q, Tq, Hq, ldq_token, ldq_head}, {k, Tk, Hkv, ldk_token, ldk_head},
                      {v, Tk, Hkv, ldv_token, ldv_head}, {out, Tq, Hq, ldo_token, ldo_head}};
  const Heads grads[] = {{dq, Tq, Hq, lddq_token, lddq_head}, {dk, Tk, Hkv, lddk_token, lddk_head},
                         {dv, Tk, Hkv, lddv_token, lddv_head}};
  for (const Heads &x : in)
    if ((st = check_heads(x, D, false)) != NVFP4_OK) return st;
  for (const Heads &x : grads)
    if ((st = check_heads(x, D, true)) != NVFP4_OK) return st;
  if (Tq > 0 && !lse) return NVFP4_ERR_NULL;
  for (const Heads &y : grads) {
    for (const Heads &x : in)
      if (y.p && y.T > 0 && y.p == x.p) return NVFP4_ERR_STRIDE;
    for (const Heads &x : grads)
      if (&x != &y && same_place(x, y)) return NVFP4_ERR_STRIDE;
  }
  const size_t need = nvfp4_attention_backward_workspace_bytes(Tq, Tk, Hq, Hkv, D, B);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return NVFP4_ERR_WORKSPACE;
  if (!aligned(lse, 4) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  if ((st = check_device()) != NVFP4_OK) return st;
  const AttentionGradArgs g{{q, k, v, row_pitch(in[1], D), ldq_head, row_pitch(in[2], D), ldk_head, row_pitch(in[3], D), ldv_head, (int)Tq, (int)Tk, (int)Hq,
                             (int)(Hq / Hkv), (int)D, (int)B, cu_q, cu_k, (int)(Tq / B), (int)(Tk / B), causal != 0, scale,
                             const_cast<void *>(out), ldo_token, ldo_head, const_cast<float *>(lse), attention_splits(Tq, Tk, Hq, B),
                             reinterpret_cast<float *>(static_cast<char *>(workspace) + backward_rows_bytes(Tq, Hq))},
                            dout, row_pitch(in[0], D), lddo_head, dq, dk, dv, lddq_token, lddq_head, lddk_token, lddk_head,
                            lddv_token, lddv_head, static_cast<float *>(workspace), attention_backward_splits(Tq, Tk, Hq, Hkv, B)};
  return hip_status(launch_attention_backward(g, static_cast<hipStream_t>(stream)));
}

nvfp4_status_t nvfp4_cache_append(const void *k, int64_t ldk_token, int64_t ldk_head, const void *v, int64_t ldv_token,
                                  int64_t ldv_head, int64_t T, int64_t Hkv, int64_t D, const int32_t *cu,
                                  const int32_t *lengths, int64_t B, void *k_cache, uint8_t *k_scales, void *v_cache,
                                  uint8_t *v_scales, int64_t pages, int64_t page_size, const int32_t *page_table,
                                  int64_t ld_table, int64_t max_pages, void *stream) {
  constexpr int64_t kThreads = (int64_t)1 << 31;
  nvfp4_status_t st = check_cache(k_cache, k_scales, v_cache, v_scales, pages, page_size, page_table, ld_table, max_pages,
                                  lengths, B, Hkv, D);
  if (st != NVFP4_OK) return st;
  if (T < 0 || (Hkv > 0 && T >= kThreads / (Hkv * ((D + 31) / 8)) - 15) || (!cu && T != B)) return NVFP4_ERR_SHAPE;
  if (T == 0 || Hkv == 0 || B == 0) return NVFP4_OK;
  if ((st = check_heads({k, T, Hkv, ldk_token, ldk_head}, D, false)) != NVFP4_OK ||
      (st = check_heads({v, T, Hkv, ldv_token, ldv_head}, D, false)) != NVFP4_OK)
    return st;
  if (!aligned(cu, 4)) return NVFP4_ERR_ALIGN;
  if ((st = check_device()) != NVFP4_OK) return st;
  if (pages == 0 || max_pages == 0) return NVFP4_OK;
  CacheAppendArgs a{};
  a.c = cache_args(k_cache, k_scales, v_cache, v_scales, pages, page_size, page_table, ld_table, max_pages, lengths, B, Hkv, D);
  a.k = k;
  a.v = v;
  a.ldk_t = ldk_token;
  a.ldk_h = ldk_head;
  a.ldv_t = ldv_token;
  a.ldv_h = ldv_head;
  a.T = (int)T;
  a.cu = cu;
  return hip_status(launch_cache_append(a, static_cast<hipStream_t>(stream)));
}

size_t nvfp4_paged_attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity) {
  if (B <= 0 || B >= (1 << 16) || Hq <= 0 || Hq > (1 << 16) || Hkv <= 0 || Hq % Hkv != 0 || D < 8 || D > kAttentionMaxD ||
      D % 8 != 0 || capacity < 0 || capacity >= kMaxCapacity)
    return 0;
  const int splits = paged_attention_splits(B, Hq, Hkv, capacity);
  return splits > 1 ? sizeof(float) * (size_t)B * (size_t)Hq * (size_t)splits * (size_t)(D + 2) : 0;
}

nvfp4_status_t nvfp4_paged_attention(const void *q, int64_t ldq_token, int64_t ldq_head, int64_t B, int64_t Hq,
                                     int64_t Hkv, int64_t D, const void *k_cache, const uint8_t *k_scales,
                                     const void *v_cache, const uint8_t *v_scales, int64_t pages, int64_t page_size,
                                     const int32_t *page_table, int64_t ld_table, int64_t max_pages,
                                     const int32_t *lengths, float scale, void *out, int64_t ldo_token,
                                     int64_t ldo_head, void *workspace, size_t workspace_bytes, void *stream) {
  nvfp4_status_t st = check_cache(k_cache, k_scales, v_cache, v_scales, pages, page_size, page_table, ld_table, max_pages,
                                  lengths, B, Hkv, D);
  if (st != NVFP4_OK) return st;
  if (Hq < 0 || Hq > (1 << 16) || (Hq > 0 && (Hkv == 0 || Hq % Hkv != 0))) return NVFP4_ERR_SHAPE;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return NVFP4_ERR_MODE;
  if (B == 0 || Hq == 0) return NVFP4_OK;
  const int64_t blocks = Hkv * ((Hq / Hkv + 31) / 32);
  if (blocks >= (1 << 16)) return NVFP4_ERR_SHAPE;
  const Heads hq{q, B, Hq, ldq_token, ldq_head}, ho{out, B, Hq, ldo_token, ldo_head};
  if ((st = check_heads(hq, D, false)) != NVFP4_OK || (st = check_heads(ho, D, true)) != NVFP4_OK) return st;
  if (!same_place_fits(ho, hq) || (pages > 0 && (out == k_cache || out == v_cache))) return NVFP4_ERR_STRIDE;
  const size_t need = nvfp4_paged_attention_workspace_bytes(B, Hq, Hkv, D, max_pages * page_size);
  if (need > 0 && (!workspace || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  if ((st = check_device()) != NVFP4_OK) return st;
  const PagedAttentionArgs a{
      cache_args(k_cache, k_scales, v_cache, v_scales, pages, page_size, page_table, ld_table, max_pages, lengths, B, Hkv, D),
      q, ldq_token, ldq_head, (int)Hq, (int)(Hq / Hkv), scale, out, ldo_token, ldo_head, static_cast<float *>(workspace),
      paged_attention_splits(B, Hq, Hkv, max_pages * page_size)};
  return hip_status(launch_paged_attention(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
