// Loads and stores of a row's elements, eight at a time, whatever the row's
// alignment and length.
#pragma once

#include "heads.h"

namespace repro {
namespace {

// Eight elements at element `o` of a row of `dim`; zeros past its end.
template <int BF16, bool STREAM>
__device__ __forceinline__ Raw<BF16, 8> load8(const char* row, int o, int dim) {
  constexpr int kSize = BF16 ? 2 : 4;
  Raw<BF16, 8> r = {};
  if (o + 8 <= dim) {
    r.template load<STREAM>(row + (int64_t)o * kSize);
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
