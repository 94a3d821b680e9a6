// Cosines and sines of the position rotation.
//
// "OPEN-1B: A Fully Auditable Training Run", Table 2: rotary positions of
// base 5e5.  The frequencies are the caller's, in binary64.
//
// Mathematics.  The angle is x = p * f with the position p < 2^31 an integer:
// hi = fl64(p * f) and lo = fma(p, f, -hi) hold it exactly.  With
// k = round(hi * 2/pi), |k| <= 2^30, and pi/2 = P1 + P2 (two binary64 parts,
// the rest below 2^-108), the remainder is ((hi - k P1) - k P2) + lo: the
// first step is exact (its result is a multiple of 2^-53 below 1 in size, or
// k is 0), the second rounds once, so the remainder r, |r| <= pi/4, is off
// by about 2^-53.  sin r and cos r are their Taylor sums, to r^13 and r^14:
// the first terms left out are below 2.1e-14 and 1.0e-15 at pi/4, far below
// half a step of binary32 (3e-8); the quadrant k mod 4 selects and signs.
// Each entry is a function of p and f alone.
//
// Design for gfx950: a thread makes four neighbouring entries of the flat
// (position, frequency) order, so each wave stores two runs of 1 KB.
#include <hip/hip_runtime.h>

#include "internal.h"

namespace repro {
namespace {

constexpr int kPer = 4;  // entries of one thread: a 16-byte store of each table

// cos and sin of p * f, rounded to binary32.
__device__ __forceinline__ void cos_sin(double p, double f, float* c, float* s) {
  const double hi = p * f;
  const double lo = __builtin_fma(p, f, -hi);
  const double k = __builtin_rint(hi * 0x1.45f306dc9c883p-1);  // 2/pi
  double r = __builtin_fma(-k, 0x1.921fb54442d18p+0, hi);      // pi/2, upper part
  r = __builtin_fma(-k, 0x1.1a62633145c07p-54, r);             // pi/2, lower part
  r += lo;
  const double q = r * r;
  double a = 1.0 / 6227020800.0;  // 1/13!
  a = __builtin_fma(a, q, -1.0 / 39916800.0);
  a = __builtin_fma(a, q, 1.0 / 362880.0);
  a = __builtin_fma(a, q, -1.0 / 5040.0);
  a = __builtin_fma(a, q, 1.0 / 120.0);
  a = __builtin_fma(a, q, -1.0 / 6.0);
  const double sr = __builtin_fma(a * q, r, r);
  double b = -1.0 / 87178291200.0;  // -1/14!
  b = __builtin_fma(b, q, 1.0 / 479001600.0);
  b = __builtin_fma(b, q, -1.0 / 3628800.0);
  b = __builtin_fma(b, q, 1.0 / 40320.0);
  b = __builtin_fma(b, q, -1.0 / 720.0);
  b = __builtin_fma(b, q, 1.0 / 24.0);
  b = __builtin_fma(b, q, -0.5);
  const double cr = __builtin_fma(b, q, 1.0);
  // Past 2^30 (and for NaN) the quadrant no longer fits: NaN.
  const bool fits = __builtin_fabs(hi) <= 1073741824.0;
  const int quad = fits ? (int)k : 0;
  float cv = (float)((quad & 1) ? sr : cr);
  float sv = (float)((quad & 1) ? cr : sr);
  cv = ((quad + 1) & 2) ? -cv : cv;
  sv = (quad & 2) ? -sv : sv;
  *c = fits ? cv : __builtin_nanf("");
  *s = fits ? sv : __builtin_nanf("");
}

typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));

__global__ __launch_bounds__(256) void k_rope_table(const double* __restrict__ inv_freq, uint32_t half, int64_t start,
                                                    int64_t total, float* __restrict__ cos,
                                                    float* __restrict__ sin) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * kPer;
  if (e >= total) return;
  // total < 2^34; a 32-bit division where the index fits it.
  int64_t row;
  uint32_t col;
  if (total <= 0xffffffffLL) {
    row = (uint32_t)e / half;
    col = (uint32_t)e - (uint32_t)row * half;
  } else {
    row = e / half;
    col = (uint32_t)(e - row * half);
  }
  float c[kPer], s[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    cos_sin((double)(start + row), inv_freq[col], &c[i], &s[i]);
    if (++col == half) {
      col = 0;
      ++row;
    }
  }
  if (e + kPer <= total) {
    *reinterpret_cast<f4u*>(cos + e) = f4u{c[0], c[1], c[2], c[3]};
    *reinterpret_cast<f4u*>(sin + e) = f4u{s[0], s[1], s[2], s[3]};
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (e + i < total) {
        cos[e + i] = c[i];
        sin[e + i] = s[i];
      }
    }
  }
}

}  // namespace

hipError_t launch_rope_table(const double* inv_freq, int half, int64_t start, int64_t length, float* cos, float* sin,
                             hipStream_t stream) {
  const int64_t total = length * half;
  const int64_t grid = (total + 256 * kPer - 1) / (256 * kPer);
  hipLaunchKernelGGL(k_rope_table, dim3((unsigned)grid), dim3(256), 0, stream, inv_freq, (uint32_t)half, start, total,
                     cos, sin);
  return hipGetLastError();
}

}  // namespace repro
