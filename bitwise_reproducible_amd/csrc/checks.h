// Argument checks shared by the front ends of the layer operators (host code).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "repro.h"

namespace repro {

inline int status_of(hipError_t e) { return e == hipSuccess ? REPRO_OK : REPRO_EDEVICE; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline uintptr_t size_of(int32_t dtype) { return dtype == REPRO_BF16 ? 2 : 4; }

inline bool is_dtype(int32_t dtype) { return dtype == REPRO_F32 || dtype == REPRO_BF16; }

// Elements from the first to one past the last of a strided view; -1 when it
// leaves 2^60 (so that no address computed from it wraps).
inline int64_t extent(const int64_t* sizes, const int64_t* strides, int dims, int64_t inner) {
  constexpr int64_t kMost = int64_t(1) << 60;
  int64_t reach = inner;
  for (int d = 0; d < dims; ++d) {
    if (sizes[d] <= 1) continue;
    int64_t part;
    if (__builtin_mul_overflow(sizes[d] - 1, strides[d], &part) || part > kMost - reach) return -1;
    reach += part;
  }
  return reach;
}

// Whether no two elements of the view of up to three dimensions share an
// address: its dimensions, from the smallest stride up, each step over all of
// the ones before.
inline bool distinct(const int64_t* sizes, const int64_t* strides, int64_t inner, int dims = 3) {
  int order[3] = {0, 1, 2};
  for (int i = 0; i < dims; ++i)
    for (int j = i + 1; j < dims; ++j)
      if (strides[order[j]] < strides[order[i]]) {
        const int t = order[i];
        order[i] = order[j];
        order[j] = t;
      }
  int64_t reach = inner;
  for (int i = 0; i < dims; ++i) {
    const int d = order[i];
    if (sizes[d] <= 1) continue;
    if (strides[d] < reach) return false;
    reach += (sizes[d] - 1) * strides[d];
  }
  return true;
}

}  // namespace repro
