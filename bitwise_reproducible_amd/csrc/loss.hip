// Softmax cross entropy with z-loss over a large vocabulary, from the hidden
// states and the output embedding, and its gradients, without the logits.
//
// "OPEN-1B: A Fully Auditable Training Run", section 3.2 (cross entropy and
// z-loss, fused and in pieces), under its Appendix A's fixed orders.
//
// Mathematics.  l = x w^T by block products (product.h).  The softmax is kept
// in powers of two: over a block of 128 entries n = rint(max l log2 e) and
// s = sum 2^(l log2 e - n), so blocks meet by exact powers of two, and the sum
// over them and its logarithm are binary64.  The gradient needs the logits
// once more: dl = e a - [v = label] g with e = 2^(l log2 e - lse log2 e),
// a = g (1 + 2 z lse) and g the loss's gradient; then dx = dl w, dw = dl^T x.
//
// Design for gfx950.  Products bound it: 2 N D V operations forward, 6 N D V
// backward.
//  - Each product's tile meets its epilogue in the accumulators.  A lane of a
//    tile holds one token's column, so a block's statistics are in-lane sums
//    and one exchange between the wave's halves.
//  - Backward, pieces of the vocabulary as wide as keeps dl within a bound.  dl
//    is stored once, by token, and the products that sum along a matrix's
//    columns turn it in the LDS (5% of their rate, against a second copy of dl
//    and transposed ones of x and w).
//  - dx sums over the vocabulary: in spans, whose number fills the chip where
//    tokens are few, each a chain of its own, folded in ascending order.
//  - Few tokens: kernels of their own (loss_few.h), for which the embedding
//    streams.
// Measured, 16384 tokens of width 2048, 128256 entries, bfloat16, on several
// cards: 7.2 to 8.1 ms forward (1060 to 1190 TFLOP/s) and 21.6 to 23.2 ms backward
// (1110 to 1190): for each piece of 8192 entries dl 491 us, dx 425, dw 395, and
// 132 for every fourth piece's fold.
#include <hip/hip_runtime.h>

#include "device_ops.h"
#include "product.h"
#include "rows.h"

namespace repro {
namespace {

constexpr float kLog2e = 0x1.715476p+0f;

// 2^t for t that is a rounding above 1/2 at most: t <= -200 gives 0, and where
// |n| is so large (from 2^23 on) that this rounding passes 1/2, the lowering to
// 1 keeps the sums finite.  The polynomial is the minimax one of degree 6 for
// the relative error on [-1/2, 1/2] (1.9e-9).
__device__ __forceinline__ float power_of_two(float t) {
  t = __builtin_amdgcn_fmed3f(t, -200.0f, 1.0f);  // NaN: -200
  const float u = __builtin_rintf(t), f = sub_c(t, u);
  float p = __builtin_fmaf(0x1.41d334p-13f, f, 0x1.5f456ap-10f);
  p = __builtin_fmaf(p, f, 0x1.3b2dbcp-7f);
  p = __builtin_fmaf(p, f, 0x1.c6aed4p-5f);
  p = __builtin_fmaf(p, f, 0x1.ebfbdap-3f);
  p = __builtin_fmaf(p, f, 0x1.62e430p-1f);
  p = __builtin_fmaf(p, f, 1.0f);
  return __builtin_ldexpf(p, (int)u);
}

// A label: its entry, or one of these.
enum { kIgnored = -1, kOutside = -2 };
__device__ __forceinline__ int label_of(const LossArgs& a, uint32_t token) {
  const int64_t at = (int64_t)token * a.label_stride;
  const int64_t y = a.label64 ? static_cast<const int64_t*>(a.labels)[at] : static_cast<const int32_t*>(a.labels)[at];
  if (y == a.ignore_index) return kIgnored;
  return y >= 0 && y < a.vocab ? (int)y : kOutside;
}

// ------------------------------------------------------------ laying out

// Eight elements' planes, four words of two each.  Binary32: the three bf16
// numbers whose sum an element is (high, middle, low); itself where it is not
// finite as a bf16 number.
template <int BF16>
__device__ __forceinline__ void planes_of(const Raw<BF16, 8>& r, uint32_t (*w)[4]) {
  if constexpr (BF16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[0][k] = r.w[k];
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = __uint_as_float(r.bits(2 * k)), y = __uint_as_float(r.bits(2 * k + 1));
      w[0][k] = round2(x, y);
      const float hx = __uint_as_float(w[0][k] << 16), hy = __uint_as_float(w[0][k] & 0xffff0000u);
      float restx = sub_c(x, hx), resty = sub_c(y, hy);
      restx = __builtin_fabsf(hx) < __builtin_inff() ? restx : 0.0f;
      resty = __builtin_fabsf(hy) < __builtin_inff() ? resty : 0.0f;
      w[1][k] = round2(restx, resty);
      w[2][k] = round2(sub_c(restx, __uint_as_float(w[1][k] << 16)),
                       sub_c(resty, __uint_as_float(w[1][k] & 0xffff0000u)));
    }
  }
}

// rows x cols of a strided matrix as planes of `pitch` elements a row, zeros in
// the columns from cols to `width`, in the rows up to `height`, and, where
// masked, in those whose label is ignored.  A wave a row.
template <int BF16>
__global__ __launch_bounds__(kThreads) void k_pack(LossArgs a, bool masked, const void* src, int64_t stride,
                                                   int64_t rows, int64_t height, int cols, int width, uint16_t* dst,
                                                   int64_t pitch, int64_t plane) {
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= height) return;
  const char* from = static_cast<const char*>(src) + row * stride * (BF16 ? 2 : 4);
  const bool there = row < rows && !(masked && label_of(a, (uint32_t)row) == kIgnored);
  for (int o = (threadIdx.x & 63) * 8; o < width; o += 512) {
    uint32_t w[BF16 ? 1 : 3][4] = {};
    if (there) planes_of<BF16>(load8<BF16, false>(from, o, cols), w);
#pragma unroll
    for (int p = 0; p < (BF16 ? 1 : 3); ++p)
      *reinterpret_cast<u4*>(dst + p * plane + row * pitch + o) = u4{w[p][0], w[p][1], w[p][2], w[p][3]};
  }
}

}  // namespace
}  // namespace repro

#include "loss_few.h"

namespace repro {
namespace {

// ------------------------------------------------------------------- tiles

// Workgroup -> tile (m, n) of tm x tn: each of the eight dies takes a run of
// neighbours, eight tiles of m for each n, whose rows its cache then shares.
struct TileAt {
  uint32_t m, n;
};
__device__ __forceinline__ TileAt tile_at(uint32_t id, uint32_t tm, uint32_t tn) {
  const uint32_t total = tm * tn, each = total / 8, more = total % 8, die = id % 8;
  id = die * each + (die < more ? die : more) + id / 8;
  const uint32_t group = id / (8 * tn), first = group * 8, high = tm - first < 8 ? tm - first : 8;
  const uint32_t rest = id - group * 8 * tn;
  return {first + rest % high, rest / high};
}

// A side whose rows `row` .. are along k, from `k` on over k_count.
__device__ __forceinline__ Side16 along_k(const Operand& o, int64_t row, int64_t k, int most, int64_t k_count) {
  const int64_t left = o.rows - row;
  const int rows = left < most ? (int)left : most;
  return {o.at + row * o.pitch + k, o.plane, (uint32_t)(o.pitch * 2),
          (uint32_t)((rows - 1) * o.pitch * 2 + k_count * 2), 0};
}

// A side whose rows are the k, from `k` on, columns `column` ...
__device__ __forceinline__ Side16 across_k(const Operand& o, int64_t k, int64_t column) {
  return {o.at + k * o.pitch + column, o.plane, (uint32_t)(o.pitch * 2), (uint32_t)((o.columns - column) * 2),
          o.rows - k};
}

__device__ __forceinline__ float other_half(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(threadIdx.x & 32 ? s[0] : s[1]);
}

// Statistics of every block of 128 entries of a piece, and the labels' logits.
template <int WM, int WN, int TN, int PARTS>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_logits(LossArgs a, Operand w, Operand x, int64_t first) {
  typedef Product<WM, WN, 4, TN, PARTS> P;
  __shared__ __attribute__((aligned(1024))) char ring[P::kLdsBytes];
  const uint32_t tm = (uint32_t)((w.rows + P::kBlockM - 1) / P::kBlockM);
  const uint32_t tn = (uint32_t)((x.rows + P::kBlockN - 1) / P::kBlockN);
  const TileAt t = tile_at(blockIdx.x, tm, tn);
  f32x16 acc[4][TN];
  P::run(along_k(w, (int64_t)t.m * P::kBlockM, 0, P::kBlockM, a.k),
         along_k(x, (int64_t)t.n * P::kBlockN, 0, P::kBlockN, a.k),
         (int)(a.k / kStageK), ring, acc);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, h = lane >> 5;
  const int64_t entry = first + (int64_t)t.m * P::kBlockM + (wave % WM) * 128;  // of this wave's block
  if (entry >= a.vocab) return;
  const int left = (int)(a.vocab - entry < 128 ? a.vocab - entry : 128);
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const uint32_t token = t.n * P::kBlockN + (wave / WM) * (TN * 32) + j * 32 + (lane & 31);
    float l[4][16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 16; ++k) l[i][k] = acc[i][j][k];
    if (left < 128) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (32 * i + 8 * (k >> 2) + 4 * h + (k & 3) >= left) l[i][k] = -__builtin_inff();
    }
    float most = l[0][0];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        most = fmaxf(most, fmaxf(l[i][k], l[i][k + 1]));
        odd |= __builtin_isunordered(l[i][k], l[i][k + 1]);
      }
    most = fmaxf(most, other_half(most));
    const float n = __builtin_rintf(mul_c(most, kLog2e));
    const float shift = n == -__builtin_inff() ? 0.0f : n;
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float e = power_of_two(__builtin_fmaf(l[i][k], kLog2e, -shift));
        c[k & 3] = i == 0 && k < 4 ? e : add_c(c[k & 3], e);
      }
    float s = add_c(add_c(c[0], c[1]), add_c(c[2], c[3]));
    if (odd || n == __builtin_inff()) s = __builtin_nanf("");
    s = add_c(s, other_half(s));
    if (token < a.tokens) {
      if (h == 0) a.stats[entry / 128 * a.padded_tokens + token] = make_float2(n, s);
      const int y = label_of(a, token) - (int)entry;
      const bool mine = y >= 0 && y < 128 && ((y >> 2) & 1) == h;
      if (__builtin_amdgcn_ballot_w64(mine) != 0) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (y == 32 * i + 8 * (k >> 2) + 4 * h + (k & 3)) v = l[i][k];
        if (mine) a.picked[token] = v;
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // one column's elements at a time in registers
  }
}

// ln v for v > 0 in binary64: v = 2^e f with f in [sqrt(1/2), sqrt(2)), and
// ln f = 2 artanh((f - 1) / (f + 1)) by its series.  Within 4e-16 of the exact
// one, relative to max(1, its size).
__device__ __forceinline__ double natural_log(double v) {
  int e;
  double f = frexp(v, &e);
  if (f < 0x1.6a09e667f3bcdp-1) {
    f = f * 2.0;
    e -= 1;
  }
  const double s = (f - 1.0) / (f + 1.0), q = s * s;
  double p = 1.0 / 23.0;
#pragma unroll
  for (int k = 21; k >= 1; k -= 2) p = p * q + 1.0 / k;
  return (double)e * 0x1.62e42fefa39efp-1 + 2.0 * s * p;
}

// lse and loss of each token from its blocks' statistics: 64 parts of a token,
// part p taking blocks p, p + 64, ..; 16 tokens of a workgroup.
constexpr int kCombineTokens = 16, kCombineParts = 64;
__global__ __launch_bounds__(kCombineTokens* kCombineParts) void k_combine(LossArgs a) {
  __shared__ double sums[kCombineParts][kCombineTokens];
  __shared__ float most[kCombineParts][kCombineTokens];
  const int at = threadIdx.x % kCombineTokens, part = threadIdx.x / kCombineTokens;
  const uint32_t token = blockIdx.x * kCombineTokens + at;
  const int64_t blocks = (a.vocab + 127) / 128;
  const bool on = token < a.tokens;
  const float2* stats = a.stats + token;
  // A part's first blocks are kept for the second pass: all of them up to
  // 131072 entries.
  constexpr int kKept = 16;
  float2 kept[kKept];
  float n = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int64_t b = part + (int64_t)i * kCombineParts;
    kept[i] = on && b < blocks ? stats[b * a.padded_tokens] : make_float2(-__builtin_inff(), 0.0f);
  }
#pragma unroll
  for (int i = 0; i < kKept; ++i) n = fmaxf(n, kept[i].x);
  if (on)
#pragma unroll 4
    for (int64_t b = part + kKept * kCombineParts; b < blocks; b += kCombineParts)
      n = fmaxf(n, stats[b * a.padded_tokens].x);
  most[part][at] = n;
  for (int m = kCombineParts / 2; m > 0; m >>= 1) {
    __syncthreads();
    if (part < m) most[part][at] = fmaxf(most[part][at], most[part + m][at]);
  }
  __syncthreads();
  n = most[0][at];
  double s = 0.0;
  const auto add = [&](const float2& v) {
    // A block below all others by 2^2000 adds nothing.
    s += ldexp((double)v.y, (int)fmaxf(v.x - n, -2000.0f));
  };
#pragma unroll
  for (int i = 0; i < kKept; ++i) add(kept[i]);  // +0 behind the last block
  if (on)
#pragma unroll 4
    for (int64_t b = part + kKept * kCombineParts; b < blocks; b += kCombineParts) add(stats[b * a.padded_tokens]);
  sums[part][at] = s;
  for (int m = 1; m < kCombineParts; m *= 2) {
    __syncthreads();
    if (part % (2 * m) == 0) sums[part][at] += sums[part + m][at];
  }
  if (part != 0 || !on) return;
  const double total = sums[0][at];
  // No entry above -inf: the logarithm of nothing.
  double lse = n == -__builtin_inff() ? (double)n : (double)n * 0x1.62e42fefa39efp-1 + natural_log(total);
  if (!(total == total)) lse = total;
  a.lse_out[token] = (float)lse;
  const int y = label_of(a, token);
  float loss = 0.0f;
  if (y == kOutside) loss = __builtin_nanf("");
  if (y >= 0) loss = (float)((lse - (double)a.picked[token]) + (double)a.z_weight * (lse * lse));
  a.loss[token] = loss;
}

// ---------------------------------------------------------------- gradients

// What the gradient's epilogue needs of each token: lse log2 e, a, g and the
// label.  Nothing reaches the gradient of an ignored token (or of padding):
// its e is 2^-inf.
// lse log2 e is rounded to binary32, so that the exponent takes one fused step.
// That moves e by up to 7e-7 where lse log2 e is 16 to 32; the step's own rounding
// moves a rare entry's (2^-16 to 2^-32) as much, and that of lse, as it is stored,
// 5e-7.  l - lse first and the factor behind it is no nearer: for 64 tokens and
// 128256 entries, with the oracle's operations, e is 4.3e-7 from 64 bits so and
// 4.0e-7 so, its sums over the tokens 0.9e-7 and 1.7e-7.
__global__ __launch_bounds__(kThreads) void k_tokens(LossArgs a) {
  const uint32_t token = blockIdx.x * kThreads + threadIdx.x;
  if (token >= a.padded_tokens) return;
  float4 t = make_float4(__builtin_inff(), 0.0f, 0.0f, __int_as_float(kIgnored));
  if (token < a.tokens) {
    const int y = label_of(a, token);
    if (y != kIgnored) {
      const float lse = a.lse_in[token], g = a.dloss[(int64_t)token * a.dloss_stride];
      t.x = (float)((double)lse * 0x1.71547652b82fep+0);
      t.y = (float)((double)g * (1.0 + 2.0 * (double)a.z_weight * (double)lse));
      t.z = g;
      t.w = __int_as_float(y);
      if (y == kOutside) t.y = __builtin_nanf("");
    }
  }
  a.per_token[token] = t;
}

// dl of a piece, as bf16 (or its three parts): a row for each token.
template <int WM, int WN, int TN, int PARTS>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_dlogits(LossArgs a, Operand w, Operand x, int64_t first,
                                                             uint16_t* dl, int64_t plane, int64_t pitch) {
  typedef Product<WM, WN, 4, TN, PARTS> P;
  __shared__ __attribute__((aligned(1024))) char ring[P::kLdsBytes];
  const uint32_t tm = (uint32_t)((w.rows + P::kBlockM - 1) / P::kBlockM);
  const uint32_t tn = a.padded_tokens / P::kBlockN;
  const TileAt t = tile_at(blockIdx.x, tm, tn);
  f32x16 acc[4][TN];
  P::run(along_k(w, (int64_t)t.m * P::kBlockM, 0, P::kBlockM, a.k),
         along_k(x, (int64_t)t.n * P::kBlockN, 0, P::kBlockN, a.k),
         (int)(a.k / kStageK), ring, acc);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, h = lane >> 5;
  const int at = (int)t.m * P::kBlockM + (wave % WM) * 128;  // this wave's first entry of the piece
  const int64_t left = a.vocab - first - at;
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const uint32_t token = t.n * P::kBlockN + (wave / WM) * (TN * 32) + j * 32 + (lane & 31);
    const float4 mine = a.per_token[token];
    float d[4][16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 16; ++k)
        d[i][k] = mul_c(power_of_two(__builtin_fmaf(acc[i][j][k], kLog2e, -mine.x)), mine.y);
    const int y = __float_as_int(mine.w) - (int)(first + at);
    if (__builtin_amdgcn_ballot_w64(y >= 0 && y < 128) != 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (y == 32 * i + 8 * (k >> 2) + 4 * h + (k & 3)) d[i][k] = sub_c(d[i][k], mine.z);
    }
    if (left < 128) {
      // Entries past the vocabulary: nothing, whatever their products held.
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (32 * i + 8 * (k >> 2) + 4 * h + (k & 3) >= left) d[i][k] = 0.0f;
    }
    // In bfloat16 dl is rounded to what the matrix cores take, before the products
    // that are rounded themselves: gradients lie 1.9e-3 to 2.6e-3 of their length
    // from 64 bits (2^-8 where one entry alone makes a token's), and 1.7e-3 is the
    // rounding of the result.  A second plane, of what this one leaves, would take
    // dx's and dw's products twice, 820 of the 1311 us of a piece: 22 ms to 36 for
    // the microbatch.  A model of this type that keeps its logits rounds their
    // gradient as well.
    constexpr int kPlanes = PARTS == 1 ? 1 : 3;
#pragma unroll
    for (int p = 0; p < kPlanes; ++p) {
      uint16_t* row = dl + p * plane + (int64_t)token * pitch + at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t lo[4], hi[4];  // entries 0, 1 and 2, 3 of each four
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float* v = d[i] + 4 * q;
          lo[q] = round2(v[0], v[1]);
          hi[q] = round2(v[2], v[3]);
          if constexpr (kPlanes > 1) {
            // What this part leaves for the next ones.
            if (p < kPlanes - 1) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t bits = (k < 2 ? lo[q] : hi[q]) >> (16 * (k & 1)) & 0xffff;
                const bool fine = (bits & 0x7f80) != 0x7f80;
                v[k] = fine ? sub_c(v[k], __uint_as_float(bits << 16)) : 0.0f;
              }
            }
          }
        }
        // The halves of the wave trade fours, so that each lane has eight
        // neighbours.
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const auto u = __builtin_amdgcn_permlane32_swap(lo[q], lo[q + 1], false, false);
          const auto v = __builtin_amdgcn_permlane32_swap(hi[q], hi[q + 1], false, false);
          *reinterpret_cast<uint4*>(row + 32 * i + 8 * (q + h)) = make_uint4(u[0], v[0], u[1], v[1]);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // one column's elements at a time in registers
  }
}

// Sums over the spans of a piece, binary32: partial[span][token][width].
template <int WM, int WN, int TN, int PARTS>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_dx(LossArgs a, Operand w, Operand dl, int64_t span, int64_t entries,
                                                        float* partial, int64_t width) {
  typedef Product<WM, WN, 4, TN, PARTS, true, false> T;
  __shared__ __attribute__((aligned(1024))) char ring[T::kLdsBytes];
  const uint32_t tm = (uint32_t)((a.dim + T::kBlockM - 1) / T::kBlockM), tn = a.padded_tokens / T::kBlockN;
  const uint32_t z = blockIdx.x / (tm * tn);
  const TileAt t = tile_at(blockIdx.x - z * tm * tn, tm, tn);
  const int64_t k0 = z * span, k = entries - k0 < span ? entries - k0 : span;
  f32x16 acc[4][TN];
  T::run(across_k(w, k0, (int64_t)t.m * T::kBlockM), along_k(dl, (int64_t)t.n * T::kBlockN, k0, T::kBlockN, k),
         (int)(k / kStageK), ring, acc);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, h = lane >> 5;
  const uint32_t token = t.n * T::kBlockN + (wave / WM) * (TN * 32) + (lane & 31);
  float* row = partial + ((int64_t)z * a.padded_tokens + token) * width + t.m * T::kBlockM + (wave % WM) * 128 + 4 * h;
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4*>(row + j * 32 * width + 32 * i + 8 * q) = make_float4(
            acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
}

// The spans' sums in ascending order, after those of earlier ones (before); the
// last ones' go to dx, rounded once.  Adding in the product's own epilogue cost
// more than the trip to memory: 539 us for 16384 x 2048 sums of 8192 entries,
// and 448 without.
template <int BF16>
__global__ __launch_bounds__(kThreads) void k_dx_fold(LossArgs a, const float* partial, int spans, int64_t width,
                                                      float* sums, bool before, bool last) {
  const uint32_t token = blockIdx.y + blockIdx.z * 32768;
  const int d = (blockIdx.x * kThreads + threadIdx.x) * 4;
  if (token >= a.tokens || d >= a.dim) return;
  const float* p = partial + (int64_t)token * width + d;
  float4* at = reinterpret_cast<float4*>(sums + (int64_t)token * width + d);
  float4 v = before ? *at : *reinterpret_cast<const float4*>(p);
#pragma unroll 8
  for (int s = before ? 0 : 1; s < spans; ++s)
    v = add4(v, *reinterpret_cast<const float4*>(p + (int64_t)s * a.padded_tokens * width));
  if (!last) {
    *at = v;
    return;
  }
  if (label_of(a, token) == kIgnored) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (d + k >= a.dim) continue;
    const int64_t to = (int64_t)token * a.dx_stride + d + k;
    if constexpr (BF16)
      static_cast<uint16_t*>(a.dx)[to] = (uint16_t)round2(e[k], 0.0f);
    else
      static_cast<float*>(a.dx)[to] = e[k];
  }
}

// Rows of dw, rounded once.  TN: 4, or 2 and two workgroups on a compute unit
// for few tokens, where the stores of one run beside the products of the other.
template <int BF16, int PARTS, int TN>
__global__ __launch_bounds__(256, TN == 4 ? 1 : 2) void k_dw(LossArgs a, Operand x, Operand dl, int64_t first,
                                                             int64_t rows) {
  typedef Product<2, 2, 4, TN, PARTS, true, true, TN == 4 ? 4 : 3> T;
  __shared__ __attribute__((aligned(1024))) char ring[T::kLdsBytes];
  const uint32_t tm = (uint32_t)((a.dim + T::kBlockM - 1) / T::kBlockM);
  const uint32_t tn = (uint32_t)((rows + T::kBlockN - 1) / T::kBlockN);
  const TileAt t = tile_at(blockIdx.x, tm, tn);
  f32x16 acc[4][TN];
  T::run(across_k(x, 0, (int64_t)t.m * T::kBlockM), across_k(dl, 0, (int64_t)t.n * T::kBlockN),
         (int)(a.padded_tokens / kStageK), ring, acc);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, h = lane >> 5;
  const int from = (int)t.m * T::kBlockM + (wave % 2) * 128;
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int64_t entry = (int64_t)t.n * T::kBlockN + (wave / 2) * (TN * 32) + j * 32 + (lane & 31);
    if (entry >= rows) continue;
    const int64_t row = (first + entry) * a.dw_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF16) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          lo[q] = round2(acc[i][j][4 * q], acc[i][j][4 * q + 1]);
          hi[q] = round2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        }
        uint16_t* out = static_cast<uint16_t*>(a.dw) + row;
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          // The other half holds the same entry's other fours.
          const auto u = __builtin_amdgcn_permlane32_swap(lo[q], lo[q + 1], false, false);
          const auto v = __builtin_amdgcn_permlane32_swap(hi[q], hi[q + 1], false, false);
          const int at = from + 32 * i + 8 * (q + h);
          const u4 word = {u[0], v[0], u[1], v[1]};
          if (at + 8 <= a.dim) {
            *reinterpret_cast<u4_2*>(out + at) = word;
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (at + k < a.dim) out[at + k] = (uint16_t)(word[k >> 1] >> (16 * (k & 1)));
          }
        }
      } else {
        float* out = static_cast<float*>(a.dw) + row;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int at = from + 32 * i + 8 * q + 4 * h;
          const u4 word = {__float_as_uint(acc[i][j][4 * q]), __float_as_uint(acc[i][j][4 * q + 1]),
                           __float_as_uint(acc[i][j][4 * q + 2]), __float_as_uint(acc[i][j][4 * q + 3])};
          if (at + 4 <= a.dim) {
            *reinterpret_cast<u4_4*>(out + at) = word;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (at + k < a.dim) out[at + k] = __uint_as_float(word[k]);
          }
        }
      }
    }
  }
}

// No tokens: dw is zero.
__global__ __launch_bounds__(kThreads) void k_no_dw(LossArgs a, int size) {
  const int64_t row = blockIdx.y + (int64_t)blockIdx.z * 32768;
  const int d = blockIdx.x * kThreads + threadIdx.x;
  if (row >= a.vocab || d >= a.dim) return;
  if (size == 2)
    static_cast<uint16_t*>(a.dw)[row * a.dw_stride + d] = 0;
  else
    static_cast<float*>(a.dw)[row * a.dw_stride + d] = 0.0f;
}

uint32_t tiles(int64_t n, int64_t of) { return (uint32_t)((n + of - 1) / of); }
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Elements from one row to the next.  Rows a multiple of 32 KB apart meet in the
// same channels: 1029 TFLOP/s at 32 KB for tiles of 8192 x 2048 over 16384 k,
// 1272 with 512 bytes more (1230 with 128).  Rows of 16 KB do not: 1283 as they
// are, 1256 and 1173 with as many more.
int64_t pitch_of(int64_t width) { return width % 16384 == 0 ? width + 256 : width; }

void pack(const LossArgs& a, bool bf16, bool masked, const void* src, int64_t stride, int64_t rows, int64_t height,
          int64_t width, uint16_t* dst, int64_t plane, hipStream_t stream) {
  const dim3 grid(tiles(height, kThreads / 64));
  if (bf16)
    hipLaunchKernelGGL(k_pack<1>, grid, dim3(kThreads), 0, stream, a, masked, src, stride, rows, height, a.dim,
                       (int)width, dst, pitch_of(width), plane);
  else
    hipLaunchKernelGGL(k_pack<0>, grid, dim3(kThreads), 0, stream, a, masked, src, stride, rows, height, a.dim,
                       (int)width, dst, pitch_of(width), plane);
}

// Tokens up to which the embedding goes to registers alone: binary32 rows, and
// bf16 rows that the tiles would need a copy of.  Width 2048, 128256 entries,
// us: binary32, so and through the LDS (kSplit): 8 tokens 246 and 258, 32 tokens
// 346 and 262, 64 tokens 538 and 262.
constexpr int64_t kFewest = 16, kFew = 64;
// The sums over tokens are padded to a multiple of this; tiles have as many
// (the kernels for few tokens fewer).
constexpr int tile_tokens(int64_t tokens) { return tokens <= 64 ? 64 : tokens <= 128 ? 128 : 256; }

// The kernels for a call's tiles: CALL(WM, WN, TN, PARTS).  WIDE: waves of 256
// tokens, and 32-token columns of each.
#define FOR_TILES(tile, bf16, WIDE, COLUMNS, CALL) \
  do {                                             \
    if (!(bf16)) {                                 \
      CALL(2, WIDE, COLUMNS, kParts);              \
    } else if ((tile) == 64) {                     \
      CALL(2, 1, 2, 1);                            \
    } else if ((tile) == 128) {                    \
      CALL(2, 2, 2, 1);                            \
    } else {                                       \
      CALL(2, WIDE, COLUMNS, 1);                   \
    }                                              \
  } while (0)

// Likewise of k_few_logits and k_few_dx: CALL(BF16, NT).
#define FOR_FEW(tokens, bf16, CALL)  \
  do {                               \
    if ((tokens) <= 16) {            \
      if (bf16) {                    \
        CALL(1, 1);                  \
      } else {                       \
        CALL(0, 1);                  \
      }                              \
    } else if ((tokens) <= 32) {     \
      if (bf16) {                    \
        CALL(1, 2);                  \
      } else {                       \
        CALL(0, 2);                  \
      }                              \
    } else {                         \
      if (bf16) {                    \
        CALL(1, 4);                  \
      } else {                       \
        CALL(0, 4);                  \
      }                              \
    }                                \
  } while (0)

const char* element(const void* base, int64_t at, bool bf16) {
  return static_cast<const char*>(base) + at * (bf16 ? 2 : 4);
}

struct Taker {  // parts of a workspace, 256-byte aligned
  uint8_t* base;
  int64_t used;
  template <typename T>
  T* take(int64_t count) {
    T* out = reinterpret_cast<T*>(base + used);
    used += up(count * (int64_t)sizeof(T), 256);
    return out;
  }
};

// Entries of a piece of the forward pass whose rows are packed: few enough to be
// read back from the caches.
constexpr int64_t kForwardPiece = 16384;
// Tiles of a launch: below 2^32 threads.
constexpr int64_t kMostTiles = int64_t(1) << 22;
// Elements of dl that a piece of the backward pass holds.
constexpr int64_t kPieceElements = int64_t(1) << 27;
// Tokens up to which dw's tiles are the smaller ones.  Gradients in bfloat16 at
// width 2048 and 128256 entries, us, so and with the large ones: 64 tokens 440 and
// 478, 256 tokens 631 and 645, 512 as fast, 1024 tokens 1667 and 1626.
constexpr int64_t kShortSum = 512;
// And where there are fewer large ones than compute units: binary32 gradients of
// 3068 tokens of width 448 over 883 entries (8 tiles) 414 us, 510 with large ones.
constexpr uint32_t kShortTiles = 256;
// Tokens up to which binary32 embeddings are split on their way: in all
// products with them, and in the forward pass.  Us of a call, width 2048, 128256
// entries, so and with a copy in parts, in turn on one card: forward 64 tokens
// 289 and 1074, 256 832 and 1151, 700 2049 and 2320, 1024 2754 and 2949 (more
// were not measured); backward, on another, 200 2683 and 3500.
constexpr int64_t kSplit = 256, kSplitForward = 1024;
// The tiles of binary32 are of 256 tokens alone: a call that pads to fewer would
// run them past its own.
static_assert(tile_tokens(kSplit + 1) == 256, "fewer tokens than a binary32 tile has take the other kernels");
// Pieces of one span whose sums wait to be folded together.
constexpr int64_t kWaiting = 4;

// Everything that the sizes alone decide.
struct Plan {
  bool bf16, few, split, packed;  // packed: the embedding's rows are
  int planes, tile;
  int64_t k, tokens, forward_piece, spans, span, piece;  // span, piece: entries
  int64_t waiting;                                       // spans whose sums are folded together
};

Plan plan_of(const LossArgs& a, const LossLayout& l) {
  Plan p;
  p.bf16 = l.bf16;
  p.few = a.tokens <= (!l.bf16 ? kSplit : l.direct_w ? 0 : kFew);
  p.split = !l.bf16 && a.tokens > kFewest && l.near_w;
  p.planes = l.bf16 ? 1 : 3;
  p.tile = tile_tokens(a.tokens);
  p.k = up(a.dim, 64);
  p.tokens = up(a.tokens, p.tile);
  // Packed rows: a piece of as many as fill the chip twice.
  p.forward_piece = 256 * (512 / (p.tokens > 0 ? p.tokens / p.tile : 1));
  if (p.forward_piece < kForwardPiece) p.forward_piece = kForwardPiece;
  p.packed = !l.direct_w && !p.few;
  if (!p.packed) p.forward_piece = 256 * (kMostTiles / (p.tokens > 0 ? p.tokens / p.tile : 1));
  if (p.forward_piece > a.vocab) p.forward_piece = a.vocab;
  // Spans: enough side by side to fill the chip (of shorter ones, and twice,
  // where a wave has so little to load), also in a piece.
  const int64_t out_tiles = (int64_t)tiles(a.tokens, p.tile) * tiles(a.dim, 256);
  const int64_t beside = out_tiles > 0 && out_tiles < 256 ? 256 / out_tiles : 1;
  int64_t spans = a.tokens <= 64 ? (out_tiles > 0 ? (512 + out_tiles - 1) / out_tiles : 1) : beside;
  const int64_t shortest = a.tokens <= 64 ? 512 : 1024;
  const int64_t most = (a.vocab + shortest - 1) / shortest;
  if (spans > most) spans = most;
  const int64_t least = (p.tokens * a.vocab * beside + kPieceElements - 1) / kPieceElements;
  if (spans < least) spans = least;
  if (spans < 1) spans = 1;
  p.span = up((a.vocab + spans - 1) / spans, 256);
  p.spans = (a.vocab + p.span - 1) / p.span;
  int64_t together = kPieceElements / (p.span * (p.tokens > 0 ? p.tokens : 1));
  if (together < 1) together = 1;
  if (together > p.spans) together = p.spans;
  p.piece = together * p.span;
  p.waiting = together > 1 ? together : p.spans < kWaiting ? p.spans : kWaiting;
  return p;
}

struct Parts {
  uint16_t *x, *w;  // packed rows, where they are not used as they are
  // forward
  float2* stats;
  float* picked;
  // backward
  float4* per_token;
  uint16_t* dl;
  float *partial, *sums;
  int64_t width;  // of partial and sums
  int64_t bytes;
};

Parts lay_out(const LossArgs& a, const LossLayout& l, const Plan& p, bool backward, void* workspace) {
  Taker t = {static_cast<uint8_t*>(workspace), 0};
  Parts s = {};
  // The backward pass sums over the tokens, so that those past the last and
  // the ignored ones have to be zeros: a copy.
  if (backward)
    s.x = t.take<uint16_t>(p.planes * p.tokens * pitch_of(p.k));
  else if (!l.direct_x)
    s.x = t.take<uint16_t>(p.planes * a.tokens * pitch_of(p.k));
  const int64_t piece = backward ? p.piece : p.forward_piece;
  if (p.packed && (backward || !p.split || a.tokens > kSplitForward)) s.w = t.take<uint16_t>(p.planes * piece * pitch_of(p.k));
  if (!backward) {
    s.stats = t.take<float2>((a.vocab + 127) / 128 * p.tokens);
    s.picked = t.take<float>(p.tokens);
  } else {
    s.width = up(a.dim, 256);
    s.per_token = t.take<float4>(p.tokens);
    s.dl = t.take<uint16_t>(p.planes * p.tokens * pitch_of(piece));
    s.partial = t.take<float>(p.waiting * p.tokens * s.width);
    if (p.waiting < p.spans) s.sums = t.take<float>(p.tokens * s.width);
  }
  s.bytes = t.used;
  return s;
}

// Rows first .. first + rows of the embedding, packed where they have to be;
// `room`: of a piece.
Operand embedding(const LossArgs& a, const LossLayout& l, const Plan& p, const Parts& s, int64_t first, int64_t rows,
                  int64_t room, hipStream_t stream) {
  const char* at = element(a.w, first * a.w_stride, p.bf16);
  if (l.direct_w) return {reinterpret_cast<const uint16_t*>(at), 0, a.w_stride, rows, a.dim};
  const int64_t pitch = pitch_of(p.k), plane = room * pitch;
  pack(a, p.bf16, false, at, a.w_stride, rows, rows, p.k, s.w, plane, stream);
  return {s.w, plane, pitch, rows, p.k};
}

}  // namespace

int64_t loss_workspace(const LossArgs& a, const LossLayout& l, bool backward) {
  if (a.tokens == 0) return 0;
  return lay_out(a, l, plan_of(a, l), backward, nullptr).bytes;
}

hipError_t launch_loss(LossArgs a, const LossLayout& l, void* workspace, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  const Plan p = plan_of(a, l);
  const Parts s = lay_out(a, l, p, false, workspace);
  a.k = p.k;
  a.padded_tokens = (uint32_t)p.tokens;
  a.stats = s.stats;
  a.picked = s.picked;
  const int64_t x_pitch = pitch_of(p.k), x_plane = a.tokens * x_pitch;
  if (!l.direct_x) pack(a, p.bf16, false, a.x, a.x_stride, a.tokens, a.tokens, p.k, s.x, x_plane, stream);
  const Operand x = l.direct_x ? Operand{static_cast<const uint16_t*>(a.x), 0, a.x_stride, a.tokens, a.dim}
                               : Operand{s.x, x_plane, x_pitch, a.tokens, p.k};
  const bool split = p.split && a.tokens <= kSplitForward;
  if (split) {
    if (a.tokens <= 64)
      hipLaunchKernelGGL((k_split_logits<2, false>), dim3(tiles(a.vocab, 128) * tiles(a.tokens, 64)), dim3(256), 0,
                         stream, a, x, 0, nullptr, 0, 0);
    else
      hipLaunchKernelGGL((k_split_logits<4, false>), dim3(tiles(a.vocab, 128) * tiles(a.tokens, 128)), dim3(256), 0,
                         stream, a, x, 0, nullptr, 0, 0);
  } else if (p.few) {
#define RUN(BF16, NT)                                                                                                  \
  hipLaunchKernelGGL((k_few_logits<BF16, NT, false>), dim3(tiles(a.vocab, 128) * tiles(a.tokens, 16 * NT)), dim3(256), \
                     0, stream, a, x, 0, nullptr, 0, 0)
    FOR_FEW(a.tokens, p.bf16, RUN);
#undef RUN
  }
  for (int64_t first = 0; !p.few && !split && first < a.vocab; first += p.forward_piece) {
    const int64_t rows = a.vocab - first < p.forward_piece ? a.vocab - first : p.forward_piece;
    const Operand w = embedding(a, l, p, s, first, rows, p.forward_piece, stream);
    const uint32_t grid = tiles(rows, 256) * tiles(a.tokens, p.tile);
#define RUN(WM, WN, TN, PARTS) \
  hipLaunchKernelGGL((k_logits<WM, WN, TN, PARTS>), dim3(grid), dim3(64 * WM * WN), 0, stream, a, w, x, first)
    FOR_TILES(p.tile, p.bf16, 4, 2, RUN);
#undef RUN
  }
  hipLaunchKernelGGL(k_combine, dim3(tiles(a.tokens, kCombineTokens)), dim3(kCombineTokens * kCombineParts), 0, stream,
                     a);
  return hipGetLastError();
}

hipError_t launch_loss_grad(LossArgs a, const LossLayout& l, void* workspace, hipStream_t stream) {
  if (a.tokens == 0) {
    hipLaunchKernelGGL(k_no_dw, dim3(tiles(a.dim, kThreads), a.vocab < 32768 ? (uint32_t)a.vocab : 32768, tiles(a.vocab, 32768)),
                       dim3(kThreads), 0, stream, a, l.bf16 ? 2 : 4);
    return hipGetLastError();
  }
  const Plan p = plan_of(a, l);
  const Parts s = lay_out(a, l, p, true, workspace);
  a.k = p.k;
  a.padded_tokens = (uint32_t)p.tokens;
  a.per_token = s.per_token;
  hipLaunchKernelGGL(k_tokens, dim3(tiles(p.tokens, kThreads)), dim3(kThreads), 0, stream, a);
  const int64_t x_pitch = pitch_of(p.k), x_plane = p.tokens * x_pitch;
  pack(a, p.bf16, true, a.x, a.x_stride, a.tokens, p.tokens, p.k, s.x, x_plane, stream);
  const Operand x = {s.x, x_plane, x_pitch, p.tokens, p.k};
  int64_t waiting = 0;
  bool before = false;
  for (int64_t first = 0; first < a.vocab; first += p.piece) {
    const int64_t rows = a.vocab - first < p.piece ? a.vocab - first : p.piece;
    const int64_t width = up(rows, 256), pitch = pitch_of(width);  // of dl's rows
    const int64_t plane = p.tokens * pitch;
    const Operand dl = {s.dl, plane, pitch, p.tokens, width};
    const uint32_t token_tiles = tiles(p.tokens, p.tile), spans = tiles(rows, p.span);
    const bool last = first + p.piece >= a.vocab;
    float* partial = s.partial + waiting * p.tokens * s.width;
    if (p.few) {
      if (p.split) {
        if (a.tokens <= 64)
          hipLaunchKernelGGL((k_split_logits<2, true>), dim3(tiles(width, 128) * tiles(a.tokens, 64)), dim3(256), 0,
                             stream, a, x, first, s.dl, plane, pitch);
        else
          hipLaunchKernelGGL((k_split_logits<4, true>), dim3(tiles(width, 128) * tiles(a.tokens, 128)), dim3(256), 0,
                             stream, a, x, first, s.dl, plane, pitch);
      } else {
#define RUN(BF16, NT)                                                                                               \
  hipLaunchKernelGGL((k_few_logits<BF16, NT, true>), dim3(tiles(width, 128) * tiles(a.tokens, 16 * NT)), dim3(256), \
                     0, stream, a, x, first, s.dl, plane, pitch)
        FOR_FEW(a.tokens, p.bf16, RUN);
#undef RUN
      }
#define RUN(BF16, NT)                                                                                                 \
  hipLaunchKernelGGL((k_few_dx<BF16, NT>),                                                                            \
                     dim3((uint32_t)(s.width / (BF16 ? 128 : 64)) * tiles(a.tokens, 16 * NT) * spans), dim3(64), 0,   \
                     stream, a, first, rows, dl, p.span, partial, s.width)
      FOR_FEW(a.tokens, p.bf16, RUN);
#undef RUN
    } else {
      const Operand w = embedding(a, l, p, s, first, rows, p.piece, stream);
#define RUN(WM, WN, TN, PARTS)                                                                                    \
  hipLaunchKernelGGL((k_dlogits<WM, WN, TN, PARTS>), dim3(tiles(rows, 256) * token_tiles), dim3(64 * WM * WN), 0, \
                     stream, a, w, x, first, s.dl, plane, pitch)
      FOR_TILES(p.tile, p.bf16, 4, 2, RUN);
#undef RUN
#define RUN(WM, WN, TN, PARTS)                                                                                      \
  hipLaunchKernelGGL((k_dx<WM, WN, TN, PARTS>), dim3(tiles(a.dim, 256) * token_tiles * spans), dim3(64 * WM * WN), \
                     0, stream, a, w, dl, p.span, width, partial, s.width)
      FOR_TILES(p.tile, p.bf16, 2, 4, RUN);
#undef RUN
    }
    const bool narrow = p.tokens <= kShortSum || tiles(a.dim, 256) * tiles(rows, 256) < kShortTiles;
#define RUN(BF16, PARTS, TN)                                                                                         \
  hipLaunchKernelGGL((k_dw<BF16, PARTS, TN>), dim3(tiles(a.dim, 256) * tiles(rows, 64 * TN)), dim3(256), 0, stream, \
                     a, x, dl, first, rows)
    if (p.bf16) {
      if (narrow)
        RUN(1, 1, 2);
      else
        RUN(1, 1, 4);
    } else {
      if (narrow)
        RUN(0, kParts, 2);
      else
        RUN(0, kParts, 4);
    }
#undef RUN
    waiting += spans;
    if (waiting < p.waiting && !last) continue;
    const dim3 fold(tiles(a.dim, 4 * kThreads), a.tokens < 32768 ? (uint32_t)a.tokens : 32768, tiles(a.tokens, 32768));
    if (p.bf16)
      hipLaunchKernelGGL(k_dx_fold<1>, fold, dim3(kThreads), 0, stream, a, s.partial, (int)waiting, s.width, s.sums,
                         before, last);
    else
      hipLaunchKernelGGL(k_dx_fold<0>, fold, dim3(kThreads), 0, stream, a, s.partial, (int)waiting, s.width, s.sums,
                         before, last);
    waiting = 0;
    before = true;
  }
  return hipGetLastError();
}

}  // namespace repro
