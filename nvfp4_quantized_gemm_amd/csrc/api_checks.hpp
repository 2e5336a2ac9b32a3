// Host-side validation shared by the C ABI's files (before any HIP call), the device check and the
// debug scans.
#pragma once
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include "../../include/nvfp4.h"
#include "debug_check.hpp"
#include "launch.hpp"

namespace nvfp4 {

constexpr int64_t kMaxElems = (int64_t)1 << 40;  // guards 64-bit size arithmetic

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// M == 0 (an empty tensor) is valid; K must name whole 16-value blocks.
inline nvfp4_status_t check_mk(int64_t M, int64_t K) {
  if (M < 0 || K < 16 || (K % 16) != 0) return NVFP4_ERR_SHAPE;
  if (M > kMaxElems / K) return NVFP4_ERR_SHAPE;
  if (M * (K / 16) >= ((int64_t)1 << 32)) return NVFP4_ERR_SHAPE;  // 32-bit block index
  return NVFP4_OK;
}

// Block size: values per E4M3 scale byte along K (16, 32 or 64), K a multiple of it.
inline nvfp4_status_t check_bs(int64_t K, int bs) {
  if (bs != 16 && bs != 32 && bs != 64) return NVFP4_ERR_SHAPE;
  if (K % bs != 0) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

inline int elem_size(nvfp4_dtype_t t) { return t == NVFP4_F32 ? 4 : 2; }
inline bool valid_dtype(int t) { return t == NVFP4_F32 || t == NVFP4_BF16; }

// The current device must be gfx950.  Queried once per device index and cached in atomics
// (0 unknown, 1 gfx950, 2 another device), so concurrent callers on any devices are race-free;
// device indices >= kMaxDevices are queried on every call.
inline nvfp4_status_t check_device() {
  static std::atomic<int8_t> state[kMaxDevices];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return NVFP4_ERR_HIP;
  const bool slot = dev >= 0 && dev < kMaxDevices;
  if (slot) {
    const int8_t s = state[dev].load(std::memory_order_acquire);
    if (s != 0) return s == 1 ? NVFP4_OK : NVFP4_ERR_DEVICE;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return NVFP4_ERR_HIP;
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (slot) state[dev].store(ok ? 1 : 2, std::memory_order_release);
  return ok ? NVFP4_OK : NVFP4_ERR_DEVICE;
}

// GEMM sizes beyond the 32-bit row / column / depth indices of the kernels.  K and the activation
// pitch are bounded too: the launchers pass K as a 32-bit value and A offsets are formed from lda.
inline nvfp4_status_t check_gemm_extent(int64_t M, int64_t N, int64_t K, int64_t lda) {
  if (N > kMaxElems / K || M > kMaxElems / N || M >= (1 << 30) || N >= (1 << 30) || K >= (1 << 30))
    return NVFP4_ERR_SHAPE;
  if (lda > kMaxElems / M) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

inline nvfp4_status_t hip_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

// Debug checks: -1 not yet read from NVFP4_DEBUG, 0 off, 1 on.
inline std::atomic<int> debug_state{-1};

inline bool debug_on() {
  int d = debug_state.load(std::memory_order_acquire);
  if (d < 0) {
    const char *v = std::getenv("NVFP4_DEBUG");
    int expected = -1;
    debug_state.compare_exchange_strong(expected, (v && v[0] && std::strcmp(v, "0") != 0) ? 1 : 0,
                                        std::memory_order_acq_rel);
    d = debug_state.load(std::memory_order_acquire);
  }
  return d == 1;
}

// With debug checks on, scan the device data a call is about to read (the header lists the rules).
inline nvfp4_status_t debug_scan(void *stream, std::initializer_list<DebugRegion> regions) {
  if (!debug_on()) return NVFP4_OK;
  bool violated = false, skipped = false;
  if (debug_scan_regions(regions.begin(), (int)regions.size(), static_cast<hipStream_t>(stream), &violated,
                         &skipped) != hipSuccess)
    return NVFP4_ERR_HIP;
  return violated ? NVFP4_ERR_PRECONDITION : NVFP4_OK;
}

// [rows][cols] fp32 or bf16 values at a pitch of ld elements
inline DebugRegion finite_values(const void *p, nvfp4_dtype_t t, int64_t rows, int64_t cols, int64_t ld) {
  return {p, t == NVFP4_F32 ? kCheckF32 : kCheckBF16, rows, cols, ld * elem_size(t)};
}
// [rows][cols] scale bytes at a pitch of ld bytes
inline DebugRegion scale_bytes(const void *p, int kind, int64_t rows, int64_t cols, int64_t ld) {
  return {p, kind, rows, cols, ld};
}
inline DebugRegion tensor_scale_of(const float *s, bool positive) {
  return {s, positive ? kCheckScalePos : kCheckScale, 1, 1, 0};
}
// the scale-byte region of a prepacked [N][K] weight (it follows the code region)
inline DebugRegion prepacked_scales(const void *b, int64_t N, int64_t K) {
  const int64_t units = ((N + 31) / 32) * ((K + 127) / 128);
  return {static_cast<const uint8_t *>(b) + units * 2048, kCheckE4M3, 1, units * 256, 0};
}


// MX formats: whole 32-value blocks.
inline nvfp4_status_t check_mx_mk(int64_t M, int64_t K) {
  if (M < 0 || K < 32 || (K % 32) != 0) return NVFP4_ERR_SHAPE;
  if (M > kMaxElems / K) return NVFP4_ERR_SHAPE;
  if (M * (K / 16) >= ((int64_t)1 << 32)) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

// A pitch of M rows of K elements: wide enough, and small enough for 64-bit offsets.
inline nvfp4_status_t check_pitch(int64_t ld, int64_t M, int64_t K) {
  if (ld < K) return NVFP4_ERR_STRIDE;
  return ld > kMaxElems / M ? NVFP4_ERR_SHAPE : NVFP4_OK;
}
// base and pitch of an optional [rows][ld] array on 16 bytes
inline bool rows_aligned(const void *p, int64_t ld, nvfp4_dtype_t t) {
  return !p || (aligned(p, 16) && (ld * elem_size(t)) % 16 == 0);
}
// A written [M][ld] array at an input's own address must have its rows (or be one row of the same elements): rows
// are read while others are written.
inline bool in_place_fits(const void *out, int64_t ld_out, nvfp4_dtype_t t_out, const void *in, int64_t ld_in,
                          nvfp4_dtype_t t_in, int64_t M) {
  return !out || out != in || (t_out == t_in && (M <= 1 || ld_out == ld_in));
}
// [T][H][D] rows at a token and a head pitch: offsets of 64 bits, and, where they are written, rows
// that do not overlap (tokens outermost or heads outermost)
inline bool head_rows_fit(int64_t T, int64_t H, int64_t D, int64_t ld_t, int64_t ld_h, bool written) {
  if (ld_t < 0 || ld_h < 0 || ld_t > kMaxElems / T || ld_h > kMaxElems / H) return false;
  if (!written) return true;
  if (T == 1) return H == 1 || ld_h >= D;
  if (H == 1) return ld_t >= D;
  return (ld_h >= D && ld_t >= (H - 1) * ld_h + D) || (ld_t >= D && ld_h >= (T - 1) * ld_t + D);
}

}  // namespace nvfp4
