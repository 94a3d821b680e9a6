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
// by about 2^-53.  sin r and cos r are their Taylor sums, to r^15 and r^16:
// the first terms left out are below 4.6e-17 and 2.1e-18 at pi/4; the quadrant
// k mod 4 selects and signs.  This is done for the positions that kRows
// divides, and for position 1; the rows between follow by turning the last
// row by f, c' = c cf - s sf and s' = s cf + c sf, in binary64, each turn off
// by less than 4 * 2^-53, so every value is within 7e-15 of its own and is
// then rounded once to binary32 (steps of 6e-8).  Each entry is a function of
// p and f alone.
//
// Design for gfx950.  Evaluated one by one the entries need some 70 binary64
// instructions each, more than the stores take; with kRows = 16 rows from one
// evaluation it is 15.  A thread makes two neighbouring columns of a block of
// rows, so a wave stores runs of 512 bytes.  Measured on MI355X, 131072 x 64
// (67 MB, 10 us at a plain copy's rate): 11.6-12.1 us a call, box to box; side
// by side 12.5, 12.7 with 8 rows, 14.5 with 32 (too few waves), 19.2 with
// every entry evaluated.
#include <hip/hip_runtime.h>

#include "internal.h"

namespace repro {
namespace {

constexpr int kRows = 16;
constexpr int kColumns = 2;

struct CosSin {
  double c, s;
  bool fits;
};

// cos and sin of p * f; past 2^30 (and for NaN) the quadrant does not fit.
__device__ __forceinline__ CosSin cos_sin(double p, double f) {
  const double hi = p * f;
  const double lo = __builtin_fma(p, f, -hi);
  const double k = __builtin_rint(hi * 0x1.45f306dc9c883p-1);  // 2/pi
  double r = __builtin_fma(-k, 0x1.921fb54442d18p+0, hi);      // pi/2, upper part
  r = __builtin_fma(-k, 0x1.1a62633145c07p-54, r);             // pi/2, lower part
  r += lo;
  const double q = r * r;
  double a = -1.0 / 1307674368000.0;  // -1/15!
  a = __builtin_fma(a, q, 1.0 / 6227020800.0);
  a = __builtin_fma(a, q, -1.0 / 39916800.0);
  a = __builtin_fma(a, q, 1.0 / 362880.0);
  a = __builtin_fma(a, q, -1.0 / 5040.0);
  a = __builtin_fma(a, q, 1.0 / 120.0);
  a = __builtin_fma(a, q, -1.0 / 6.0);
  const double sr = __builtin_fma(a * q, r, r);
  double b = 1.0 / 20922789888000.0;  // 1/16!
  b = __builtin_fma(b, q, -1.0 / 87178291200.0);
  b = __builtin_fma(b, q, 1.0 / 479001600.0);
  b = __builtin_fma(b, q, -1.0 / 3628800.0);
  b = __builtin_fma(b, q, 1.0 / 40320.0);
  b = __builtin_fma(b, q, -1.0 / 720.0);
  b = __builtin_fma(b, q, 1.0 / 24.0);
  b = __builtin_fma(b, q, -0.5);
  const double cr = __builtin_fma(b, q, 1.0);
  CosSin out;
  out.fits = __builtin_fabs(hi) <= 1073741824.0;
  const int quad = out.fits ? (int)k : 0;
  out.c = quad & 1 ? sr : cr;
  out.s = quad & 1 ? cr : sr;
  out.c = (quad + 1) & 2 ? -out.c : out.c;
  out.s = quad & 2 ? -out.s : out.s;
  return out;
}

typedef float f2u __attribute__((ext_vector_type(2), aligned(4)));

__global__ __launch_bounds__(256) void k_rope_table(const double* __restrict__ inv_freq, uint32_t half, int64_t start,
                                                    int64_t end, uint32_t threads, float* __restrict__ cos,
                                                    float* __restrict__ sin) {
  const uint32_t t = blockIdx.x * 256u + threadIdx.x;
  if (t >= threads) return;
  const uint32_t across = (half + kColumns - 1) / kColumns;
  const uint32_t block = t / across;
  const uint32_t col = (t - block * across) * kColumns;
  const int64_t first = (start / kRows + block) * kRows;  // may begin before start
  CosSin at[kColumns], turn[kColumns];
  double f[kColumns];
#pragma unroll
  for (int i = 0; i < kColumns; ++i) {
    f[i] = inv_freq[col + i < half ? col + i : col];
    at[i] = cos_sin((double)first, f[i]);
    turn[i] = cos_sin(1.0, f[i]);
  }
  const int64_t out = (first - start) * half + col;
#pragma unroll
  for (int row = 0; row < kRows; ++row) {
    const int64_t p = first + row;
    float c[kColumns], s[kColumns];
#pragma unroll
    for (int i = 0; i < kColumns; ++i) {
      const bool fits = __builtin_fabs((double)p * f[i]) <= 1073741824.0;
      c[i] = fits ? (float)at[i].c : __builtin_nanf("");
      s[i] = fits ? (float)at[i].s : __builtin_nanf("");
      const double next = __builtin_fma(at[i].c, turn[i].c, -(at[i].s * turn[i].s));
      at[i].s = __builtin_fma(at[i].s, turn[i].c, at[i].c * turn[i].s);
      at[i].c = next;
    }
    if (p < start || p >= end) continue;
    float* cp = cos + out + (int64_t)row * half;
    float* sp = sin + out + (int64_t)row * half;
    if (col + 1 < half) {
      *reinterpret_cast<f2u*>(cp) = f2u{c[0], c[1]};
      *reinterpret_cast<f2u*>(sp) = f2u{s[0], s[1]};
    } else {
      *cp = c[0];
      *sp = s[0];
    }
  }
}

}  // namespace

hipError_t launch_rope_table(const double* inv_freq, int half, int64_t start, int64_t length, float* cos, float* sin,
                             hipStream_t stream) {
  const int64_t end = start + length;
  const int64_t blocks = (end - 1) / kRows - start / kRows + 1;
  const int64_t threads = blocks * ((half + kColumns - 1) / kColumns);  // below 2^31: two entries or more each
  hipLaunchKernelGGL(k_rope_table, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream, inv_freq,
                     (uint32_t)half, start, end, (uint32_t)threads, cos, sin);
  return hipGetLastError();
}

}  // namespace repro
