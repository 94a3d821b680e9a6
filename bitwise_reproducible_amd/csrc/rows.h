// Loads and stores of a row's elements, eight at a time, whatever the row's
// alignment and length.
#pragma once

#include "heads.h"

namespace repro {
namespace {

// r's elements `by` (0..7) places down, zeros behind them.
__device__ __forceinline__ Raw<1, 8> moved_down(Raw<1, 8> r, int by) {
  uint32_t w[5] = {r.w[0], r.w[1], r.w[2], r.w[3], 0};
  if (by & 1)
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __builtin_amdgcn_alignbit(w[k + 1], w[k], 16);
#pragma unroll
  for (int step = 1; step < 4; step *= 2)
    if (by & 2 * step)
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = k + step < 4 ? w[k + step] : 0;
  r.w = u4{w[0], w[1], w[2], w[3]};
  return r;
}

// Eight elements at element `o` of a row of `dim`; zeros past its end.  The
// last ones of a bfloat16 row are its last eight, moved: the gradients of 1665
// gated rows of 1111 take 34 us with that, and 50 us element by element.  For
// binary32, which has no words to put together, it is the other way round: 3111
// rows of 1001 with both gates take 13.6 us, and 12.5 us element by element.
template <int BF16, bool STREAM>
__device__ __forceinline__ Raw<BF16, 8> load8(const char* row, int o, int dim) {
  constexpr int kSize = BF16 ? 2 : 4;
  Raw<BF16, 8> r = {};
  if (o + 8 <= dim) {
    r.template load<STREAM>(row + (int64_t)o * kSize);
  } else if (BF16 != 0 && o < dim && dim >= 8) {
    // The address is the same in every lane; a scalar load, which the compiler
    // would make of it, drops the lowest two bits of one off a word's border.
    int by = o + 8 - dim;
    asm volatile("" : "+v"(by));
    r.template load<STREAM>(row + (int64_t)(o - by) * kSize);
    if constexpr (BF16) r = moved_down(r, by);
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
    // The last ones as four, two and one.
    const int left = dim - o;
    char* p = row + (int64_t)o * kSize;
    if constexpr (BF16) {
      typedef uint32_t u1_2 __attribute__((aligned(2)));
      u4 w = r.w;
      if (left & 4) {
        *reinterpret_cast<u2_2*>(p) = u2{w[0], w[1]};
        p += 8;
        w = u4{w[2], w[3], 0, 0};
      }
      if (left & 2) {
        *reinterpret_cast<u1_2*>(p) = w[0];
        p += 4;
        w[0] = w[1];
      }
      if (left & 1) *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    } else {
      typedef uint32_t u2_4 __attribute__((ext_vector_type(2), aligned(4)));
      u4 w = r.w[0];
      if (left & 4) {
        *reinterpret_cast<u4_4*>(p) = w;
        p += 16;
        w = r.w[1];
      }
      if (left & 2) {
        *reinterpret_cast<u2_4*>(p) = u2{w[0], w[1]};
        p += 8;
        w[0] = w[2];
      }
      if (left & 1) *reinterpret_cast<uint32_t*>(p) = w[0];
    }
  }
}

}  // namespace
}  // namespace repro
