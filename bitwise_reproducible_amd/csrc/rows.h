// Loads and stores of a row's elements, eight at a time, whatever the row's
// alignment and length.
#pragma once

#include "heads.h"

namespace repro {
namespace {

// r's elements `by` (0..7) places down, zeros behind them.
template <int BF16>
__device__ __forceinline__ Raw<BF16, 8> moved_down(Raw<BF16, 8> r, int by) {
  uint32_t w[9] = {};
  constexpr int kWords = BF16 ? 4 : 8;
  __builtin_memcpy(w, &r, sizeof(r));
  if constexpr (BF16) {
    if (by & 1)
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[k] = __builtin_amdgcn_alignbit(w[k + 1], w[k], 16);
    by >>= 1;
  }
#pragma unroll
  for (int step = 1; step < kWords; step *= 2)
    if (by & step)
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[k] = k + step < kWords ? w[k + step] : 0;
  __builtin_memcpy(&r, w, sizeof(r));
  return r;
}

// Eight elements at element `o` of a row of `dim`; zeros past its end.  The
// last ones of a row are its last eight, moved: element by element they took
// longer than the rest of a row that was short.
template <int BF16, bool STREAM>
__device__ __forceinline__ Raw<BF16, 8> load8(const char* row, int o, int dim) {
  constexpr int kSize = BF16 ? 2 : 4;
  Raw<BF16, 8> r = {};
  if (o + 8 <= dim) {
    r.template load<STREAM>(row + (int64_t)o * kSize);
  } else if (o < dim && dim >= 8) {
    // The address is the same in every lane; a scalar load, which the compiler
    // would make of it, drops the lowest two bits of one off a word's border.
    int by = o + 8 - dim;
    asm volatile("" : "+v"(by));
    r.template load<STREAM>(row + (int64_t)(o - by) * kSize);
    r = moved_down<BF16>(r, by);
  } else if (o < dim) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (o + k >= dim) continue;
      if constexpr (BF16)
        r.w[k >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(row)[o + k] << (16 * (k & 1));
      else
        r.w[k >> 2][k & 3] = reinterpret_cast<const uint32_t*>(row)[o + k];
    }
  }
  return r;
}

template <int BF16, bool STREAM>
__device__ __forceinline__ void store8(char* row, int o, int dim, const Raw<BF16, 8>& r) {
  constexpr int kSize = BF16 ? 2 : 4;
  if (o + 8 <= dim) {
    r.template store<STREAM>(row + (int64_t)o * kSize);
  } else if (o < dim) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (o + k >= dim) continue;
      if constexpr (BF16)
        reinterpret_cast<uint16_t*>(row)[o + k] = (uint16_t)r.bits(k);
      else
        reinterpret_cast<uint32_t*>(row)[o + k] = r.bits(k);
    }
  }
}

}  // namespace
}  // namespace repro
