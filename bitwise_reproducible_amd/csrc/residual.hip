// The residual stream between two blocks: the norm, gate and scale after one,
// the sum, and the norm before the next, in one pass; and its gradients.
//
// "OPEN-1B: A Fully Auditable Training Run", section 3.1 (a pre-norm decoder
// block with RMS norms), under its Appendix A's fixed orders.
//
// Mathematics.  y = xs x + bs (gate p) with p the block's output u, or
// u r(u) gain_u, is rounded to the tensors' type once, as it is stored, and
// z = y r(y) gain is that of the rounded sum, so that the backward pass finds
// the same statistics in what the forward pass left.  The norm's gradient
// needs one sum besides S = sum y^2, T = sum dn y, over the same registers:
// dn's part of the gradient is (dn - y (T r / D) r) r.
//
// Design for gfx950.  Four to seven transfers of each element bound it:
//  - A row stays in the registers of one wave, or of 4, 8 or 16 where it is
//    wider, in chunks of eight elements: chunk c is lane c mod L's (of L).
//    So 16-byte loads cover 1 KB of neighbours, the sums need six lane
//    exchanges and (wide rows) one trip through LDS, and all tensors of the
//    row are under way at once.
//  - The channels' gradients gather in registers over a workgroup's rows, one
//    row of the workspace a workgroup, folded by a second kernel.  The number
//    of workgroups is a function of the sizes, and so is the order of every
//    sum: repro.h declares it with the numbers below.
// Measured, 16384 rows of 2048 in bfloat16: 39 us forward (268 MB, partly from
// the caches; 46 to 49 without them), 45 us and 5 for the fold backward.  8192
// rows in binary32 with norms, gate and gains: 78 us and 5 backward.
#include <hip/hip_runtime.h>

#include "rows.h"

namespace repro {
namespace {

// Waves of a row, by its width; a lane has one or two chunks.
constexpr int kOneWave = 1024, kFourWaves = 4096, kEightWaves = 8192;

constexpr int threads_of(int waves) { return waves == 1 ? kThreads : 64 * waves; }

template <int BF16>
__device__ __forceinline__ void put8(char* row, int o, int dim, const float* e, bool stream) {
  const Raw<BF16, 8> r = narrow<BF16, 8>(e);
  if (stream) {
    keep_apart();
    store8<BF16, true>(row, o, dim, r);
    keep_apart();
  } else {
    store8<BF16, false>(row, o, dim, r);
  }
}

// Eight elements of a gain, of its own type; zeros past its end.
__device__ __forceinline__ void gain8(const void* gain, int is_bf16, int o, int dim, float* g) {
  const char* p = static_cast<const char*>(gain);
  if (is_bf16)
    widen(load8<1, false>(p, o, dim), g);
  else
    widen(load8<0, false>(p, o, dim), g);
}

template <int BF16>
__device__ __forceinline__ char* row_at(const RowView& v, uint32_t b, uint32_t s) {
  return static_cast<char*>(const_cast<void*>(v.data)) + (BF16 ? 2 : 4) * (b * v.stride[0] + s * v.stride[1]);
}

// The sum over a row of each lane's value: lanes, then waves, perfect trees.
// `slot`: a part of `red` that no wave may still be reading.
template <int WAVES>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int slot) {
  v = group_sum(v, 6);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    v = tree<WAVES>(red[slot]);
  }
  return v;
}

__device__ __forceinline__ float root_of(float S, const ResidualArgs& a) {
  return div_c(1.0f, sqrt_c(add_c(mul_c(S, a.inv_dim), a.eps)));
}

// p = u (r gain) of eight elements.
__device__ __forceinline__ void after_block(const ResidualArgs& a, const float* u, float r, int o, float* p) {
#pragma unroll
  for (int k = 0; k < 8; ++k) p[k] = a.block_norm ? mul_c(u[k], r) : u[k];
  if (a.block_gain != nullptr) {
    float g[8];
    gain8(a.block_gain, a.gain_bf16, o, a.dim, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = mul_c(p[k], g[k]);
  }
}

// A row's gate: each element's own, or one for the channel.
template <int BF16>
__device__ __forceinline__ bool gate8(const ResidualArgs& a, const char* gate, int o, float* g) {
  if (gate != nullptr) {
    widen(load8<BF16, false>(gate, o, a.dim), g);
    return true;
  }
  if (a.channel_gate == nullptr) return false;
  gain8(a.channel_gate, a.gain_bf16, o, a.dim, g);
  return true;
}

template <int BF16, int WAVES, int C>
__global__ __launch_bounds__(threads_of(WAVES)) void k_residual(ResidualArgs a) {
  __shared__ float red[2][16];
  constexpr int kLanes = 64 * WAVES;
  const uint32_t t = WAVES == 1 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (WAVES == 1 && t >= a.rows) return;
  const int j = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const uint32_t b = quotient(t, a.by_seq), s = t - b * a.by_seq.divisor;
  const char* x = row_at<BF16>(a.x, b, s);
  Raw<BF16, 8> xr[C], ur[C];
#pragma unroll
  for (int i = 0; i < C; ++i) xr[i] = load8<BF16, false>(x, 8 * (j + i * kLanes), a.dim);
  float e[C][8];
  const bool sum = a.block.data != nullptr;
  if (sum) {
    const char* u = row_at<BF16>(a.block, b, s);
#pragma unroll
    for (int i = 0; i < C; ++i) ur[i] = load8<BF16, false>(u, 8 * (j + i * kLanes), a.dim);
    float r = 0.0f;
    if (a.block_norm) {
      float S = 0.0f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float q[8];
        widen(ur[i], q);
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = mul_c(q[k], q[k]);
        S = i == 0 ? tree<8>(q) : add_c(S, tree<8>(q));
      }
      r = root_of(row_sum<WAVES>(S, red, 0), a);
    }
    const char* gate = a.gate.data == nullptr ? nullptr : row_at<BF16>(a.gate, b, s);
    char* y = row_at<BF16>(a.out[0], b, s);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int o = 8 * (j + i * kLanes);
      float u8[8], p[8], g[8], x8[8];
      widen(ur[i], u8);
      widen(xr[i], x8);
      after_block(a, u8, r, o, p);
      if (gate8<BF16>(a, gate, o, g)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = mul_c(p[k], g[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) p[k] = add_c(mul_c(x8[k], a.x_scale), mul_c(p[k], a.block_scale));
      const Raw<BF16, 8> rounded = narrow<BF16, 8>(p);
      widen(rounded, e[i]);
      put8<BF16>(y, o, a.dim, p, a.stream);
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) widen(xr[i], e[i]);
  }
  float S = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k] = mul_c(e[i][k], e[i][k]);
    S = i == 0 ? tree<8>(q) : add_c(S, tree<8>(q));
  }
  const float r = root_of(row_sum<WAVES>(S, red, 1), a);
  char* z = row_at<BF16>(a.out[1], b, s);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int o = 8 * (j + i * kLanes);
#pragma unroll
    for (int k = 0; k < 8; ++k) e[i][k] = mul_c(e[i][k], r);
    if (a.gain != nullptr) {
      float g[8];
      gain8(a.gain, a.gain_bf16, o, a.dim, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) e[i][k] = mul_c(e[i][k], g[k]);
    }
    put8<BF16>(z, o, a.dim, e[i], a.stream);
  }
}

// What the backward pass gathers: nothing, the gain's gradient, or it with
// the block's gain's and the channel gate's (kBlock: also all that the block's
// norm and gate need).
enum Form { kNone, kGain, kBlock };

// What a row brings.
template <int BF16, int C, int FORM>
struct Row8 {
  Raw<BF16, 8> y[C], dz[C], dy[C];
  Raw<BF16, 8> u[FORM == kBlock ? C : 1], gate[FORM == kBlock ? C : 1];
};

template <int BF16, int WAVES, int C, int FORM>
__device__ __forceinline__ void fetch_row(const ResidualArgs& a, uint32_t t, int j, Row8<BF16, C, FORM>& f) {
  constexpr int kLanes = 64 * WAVES;
  const uint32_t b = quotient(t, a.by_seq), s = t - b * a.by_seq.divisor;
  const char* y = row_at<BF16>(a.x, b, s);
  const char* dz = row_at<BF16>(a.dz, b, s);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    f.y[i] = load8<BF16, false>(y, 8 * (j + i * kLanes), a.dim);
    f.dz[i] = load8<BF16, false>(dz, 8 * (j + i * kLanes), a.dim);
  }
  if (FORM == kBlock) {
    const char* u = row_at<BF16>(a.block, b, s);
#pragma unroll
    for (int i = 0; i < C; ++i) f.u[i] = load8<BF16, false>(u, 8 * (j + i * kLanes), a.dim);
    if (a.gate.data != nullptr) {
      const char* gate = row_at<BF16>(a.gate, b, s);
#pragma unroll
      for (int i = 0; i < C; ++i) f.gate[i] = load8<BF16, false>(gate, 8 * (j + i * kLanes), a.dim);
    }
  }
  if (a.dy.data != nullptr) {
    const char* dy = row_at<BF16>(a.dy, b, s);
#pragma unroll
    for (int i = 0; i < C; ++i) f.dy[i] = load8<BF16, false>(dy, 8 * (j + i * kLanes), a.dim);
  }
}

template <int BF16, int WAVES, int C, int FORM>
__global__ __launch_bounds__(threads_of(WAVES)) void k_residual_grad(ResidualArgs a) {
  __shared__ float red[2][4][16];
  constexpr int kLanes = 64 * WAVES, kRows = WAVES == 1 ? kThreads / 64 : 1;
  const int wave = threadIdx.x >> 6, j = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const uint32_t apart = a.blocks * kRows;
  uint64_t t = blockIdx.x * kRows + (WAVES == 1 ? wave : 0);
  float acc[FORM == kNone ? 1 : FORM == kGain ? 1 : 3][FORM == kNone ? 1 : C][8] = {};
  const bool has_dy = a.dy.data != nullptr;
  // With one chunk a lane, the channels' vectors stay in registers, and the
  // next row travels during this one's arithmetic.
  constexpr bool kHeld = C == 1;
  float held[3][8];
  const void* const vectors[3] = {a.gain, a.block_gain, a.channel_gate};
  if constexpr (kHeld) {
#pragma unroll
    for (int n = 0; n < (FORM == kBlock ? 3 : 1); ++n)
      if (vectors[n] != nullptr) gain8(vectors[n], a.gain_bf16, 8 * j, a.dim, held[n]);
  }
  const auto vector = [&](int n, int o, float* g) {
    if constexpr (kHeld) {
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = held[n][k];
    } else {
      gain8(vectors[n], a.gain_bf16, o, a.dim, g);
    }
  };
  int turn = 0;
  Row8<BF16, C, FORM> f, next;
  if (kHeld && t < a.rows) fetch_row<BF16, WAVES, C, FORM>(a, (uint32_t)t, j, f);
  for (; t < a.rows; t += apart, turn ^= 1) {
    if (!kHeld)
      fetch_row<BF16, WAVES, C, FORM>(a, (uint32_t)t, j, f);
    else if (t + apart < a.rows)
      fetch_row<BF16, WAVES, C, FORM>(a, (uint32_t)(t + apart), j, next);
    const uint32_t b = quotient((uint32_t)t, a.by_seq), s = (uint32_t)t - b * a.by_seq.divisor;
    float S = 0.0f, T = 0.0f, U = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int o = 8 * (j + i * kLanes);
      float y[8], d[8], q[8];
      widen(f.y[i], y);
      widen(f.dz[i], d);
      if (a.gain != nullptr) {
        float g[8];
        vector(0, o, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = mul_c(d[k], g[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        q[k] = mul_c(y[k], y[k]);
        d[k] = mul_c(d[k], y[k]);
      }
      S = i == 0 ? tree<8>(q) : add_c(S, tree<8>(q));
      T = i == 0 ? tree<8>(d) : add_c(T, tree<8>(d));
      if (FORM == kBlock && a.block_norm) {
        widen(f.u[i], q);
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = mul_c(q[k], q[k]);
        U = i == 0 ? tree<8>(q) : add_c(U, tree<8>(q));
      }
    }
    S = group_sum(S, 6);
    T = group_sum(T, 6);
    if (FORM == kBlock) U = group_sum(U, 6);
    if constexpr (WAVES > 1) {
      if ((threadIdx.x & 63) == 0) {
        red[turn][0][wave] = S;
        red[turn][1][wave] = T;
        red[turn][2][wave] = U;
      }
      __syncthreads();
      S = tree<WAVES>(red[turn][0]);
      T = tree<WAVES>(red[turn][1]);
      U = tree<WAVES>(red[turn][2]);
    }
    const float r = root_of(S, a);
    const float w = mul_c(mul_c(mul_c(T, r), a.inv_dim), r);
    const float ru = FORM == kBlock && a.block_norm ? root_of(U, a) : 0.0f;
    // Read or widened anew: both halves' elements at once take too many
    // registers.
    if constexpr (WAVES == 16 && C == 2) {
      asm volatile("" ::: "memory");
      fetch_row<BF16, WAVES, C, FORM>(a, (uint32_t)t, j, f);
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        forget(f.y[i]);
        forget(f.dz[i]);
        if (FORM == kBlock) forget(f.u[i]);
      }
    }
    float dp[FORM == kBlock ? C : 1][8];
    float B = 0.0f;
    const bool gated = FORM == kBlock && a.gate.data != nullptr;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int o = 8 * (j + i * kLanes);
      float y[8], d[8], h[8];
      widen(f.y[i], y);
      widen(f.dz[i], d);
      if (FORM != kNone && a.sums[0] != nullptr) {
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[0][i][k] = add_c(acc[0][i][k], mul_c(d[k], mul_c(y[k], r)));
      }
      if (a.gain != nullptr) {
        float g[8];
        vector(0, o, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = mul_c(d[k], g[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = mul_c(sub_c(d[k], mul_c(y[k], w)), r);
      if (has_dy) {
        widen(f.dy[i], h);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = add_c(h[k], d[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] = mul_c(d[k], a.x_scale);
      put8<BF16>(row_at<BF16>(a.out[0], b, s), o, a.dim, h, a.stream);
      if (a.out[1].data == nullptr) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = mul_c(d[k], a.block_scale);  // dt
      if constexpr (FORM == kBlock) {
        float u[8], p[8], g[8];
        widen(f.u[i], u);
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = a.block_norm ? mul_c(u[k], ru) : u[k];
        if (a.block_gain != nullptr) {
          vector(1, o, g);
#pragma unroll
          for (int k = 0; k < 8; ++k) p[k] = mul_c(p[k], g[k]);
        }
        if (gated)
          widen(f.gate[i], g);
        else if (a.channel_gate != nullptr)
          vector(2, o, g);
        if (gated || a.channel_gate != nullptr) {
#pragma unroll
          for (int k = 0; k < 8; ++k) p[k] = mul_c(d[k], p[k]);
          if (gated) {
            put8<BF16>(row_at<BF16>(a.out[2], b, s), o, a.dim, p, a.stream);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[2][i][k] = add_c(acc[2][i][k], p[k]);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) d[k] = mul_c(d[k], g[k]);  // dp
        }
        if (a.block_norm) {
          if (a.block_gain != nullptr) {
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[1][i][k] = add_c(acc[1][i][k], mul_c(d[k], mul_c(u[k], ru)));
            vector(1, o, g);
#pragma unroll
            for (int k = 0; k < 8; ++k) d[k] = mul_c(d[k], g[k]);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            dp[i][k] = d[k];
            p[k] = mul_c(d[k], u[k]);
          }
          B = i == 0 ? tree<8>(p) : add_c(B, tree<8>(p));
          continue;
        }
      }
      put8<BF16>(row_at<BF16>(a.out[1], b, s), o, a.dim, d, a.stream);
    }
    if (FORM == kBlock && a.block_norm) {
      B = row_sum<WAVES>(B, red[turn], 3);
      const float v = mul_c(mul_c(mul_c(B, ru), a.inv_dim), ru);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float u[8];
        widen(f.u[i], u);
#pragma unroll
        for (int k = 0; k < 8; ++k) dp[i][k] = mul_c(sub_c(dp[i][k], mul_c(u[k], v)), ru);
        put8<BF16>(row_at<BF16>(a.out[1], b, s), 8 * (j + i * kLanes), a.dim, dp[i], a.stream);
      }
    }
    if (kHeld) f = next;
  }
  if constexpr (FORM != kNone) {
    constexpr int kSums = FORM == kGain ? 1 : 3;
    __shared__ float part[kRows > 1 ? kRows : 1][kRows > 1 ? 64 * 8 : 1];
#pragma unroll
    for (int n = 0; n < kSums; ++n) {
      if (a.sums[n] == nullptr) continue;
      float* row = a.partial[n] + (int64_t)blockIdx.x * a.dim;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int o = 8 * (j + i * kLanes);
        if constexpr (kRows > 1) {
          __syncthreads();
#pragma unroll
          for (int k = 0; k < 8; ++k) part[wave][k * 64 + j] = acc[n][i][k];
          __syncthreads();
          if (wave == 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int at = k * 64 + j;
              const float v = add_c(add_c(part[0][at], part[1][at]), add_c(part[2][at], part[3][at]));
              if (o + k < a.dim) row[o + k] = v;
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (o + k < a.dim) row[o + k] = acc[n][i][k];
        }
      }
    }
  }
}

// sums[n][i] = the sum of the workgroups' rows.  Each column has 128 threads'
// parts, which take every 128th row in ascending order, then a tree.  A thread
// holds kFoldWide columns' parts.
constexpr int kFoldThreads = 1024, kFoldRows = 128, kFoldWide = 4;
constexpr int kFoldColumns = kFoldThreads / kFoldRows * kFoldWide;
__global__ __launch_bounds__(kFoldThreads) void k_channel_fold(ResidualArgs a) {
  const int n = blockIdx.y;
  if (a.sums[n] == nullptr) return;
  constexpr int kAcross = kFoldColumns / kFoldWide;
  const int column = threadIdx.x % kAcross * kFoldWide, part = threadIdx.x / kAcross;
  const int i = blockIdx.x * kFoldColumns + column;
  float v[kFoldWide] = {};
  const float* p = a.partial[n] + i;
  if (i + kFoldWide <= a.dim) {
    typedef float wide __attribute__((ext_vector_type(kFoldWide), aligned(4)));
#pragma unroll 8
    for (uint32_t row = part; row < a.blocks; row += kFoldRows) {
      const wide w = *reinterpret_cast<const wide*>(p + (int64_t)row * a.dim);
#pragma unroll
      for (int k = 0; k < kFoldWide; ++k) v[k] = add_c(v[k], w[k]);
    }
  } else if (i < a.dim) {
    for (uint32_t row = part; row < a.blocks; row += kFoldRows)
#pragma unroll
      for (int k = 0; k < kFoldWide; ++k)
        if (i + k < a.dim) v[k] = add_c(v[k], p[(int64_t)row * a.dim + k]);
  }
  __shared__ float sums[kFoldRows][kFoldColumns];
#pragma unroll
  for (int k = 0; k < kFoldWide; ++k) sums[part][column + k] = v[k];
  for (int m = kFoldRows / 2; m > 0; m >>= 1) {
    __syncthreads();
    if (part < m)
#pragma unroll
      for (int k = 0; k < kFoldWide; ++k)
        sums[part][column + k] = add_c(sums[part][column + k], sums[part + m][column + k]);
  }
  if (part == 0)
#pragma unroll
    for (int k = 0; k < kFoldWide; ++k)
      if (i + k < a.dim) a.sums[n][i + k] = sums[0][column + k];
}

template <int BF16, int WAVES, int C>
hipError_t run(const ResidualArgs& a, bool backward, hipStream_t stream) {
  const dim3 block(threads_of(WAVES));
  if (!backward) {
    const uint32_t grid = WAVES == 1 ? (a.rows + 3) / 4 : a.rows;
    hipLaunchKernelGGL((k_residual<BF16, WAVES, C>), dim3(grid), block, 0, stream, a);
  } else if (a.block.data != nullptr) {
    hipLaunchKernelGGL((k_residual_grad<BF16, WAVES, C, kBlock>), dim3(a.blocks), block, 0, stream, a);
  } else if (a.sums[0] != nullptr) {
    hipLaunchKernelGGL((k_residual_grad<BF16, WAVES, C, kGain>), dim3(a.blocks), block, 0, stream, a);
  } else {
    hipLaunchKernelGGL((k_residual_grad<BF16, WAVES, C, kNone>), dim3(a.blocks), block, 0, stream, a);
  }
  return hipGetLastError();
}

template <int BF16>
hipError_t select(const ResidualArgs& a, bool backward, hipStream_t stream) {
  const int chunks = (a.dim + 7) / 8;
  if (a.dim <= kOneWave)
    return chunks <= 64 ? run<BF16, 1, 1>(a, backward, stream) : run<BF16, 1, 2>(a, backward, stream);
  if (a.dim <= kFourWaves)
    return chunks <= 256 ? run<BF16, 4, 1>(a, backward, stream) : run<BF16, 4, 2>(a, backward, stream);
  return a.dim <= kEightWaves ? run<BF16, 8, 2>(a, backward, stream) : run<BF16, 16, 2>(a, backward, stream);
}

}  // namespace

// Rows of the channels' gradients, and workgroups of the backward pass.  With
// a norm or a gate after the block (`branch`), a lane's registers leave room for
// two or three workgroups on a CU; without, for six.  16384 rows of 2048 in bfloat16 without them take 54 us
// in 512 workgroups and 45 us in 1024; 8192 in binary32 with both, 78 and 85 us.
constexpr uint32_t kBlockGroups = 512, kGainGroups = 1024;

bool plan_residual(ResidualArgs* a, bool branch) {
  const uint32_t each = a->dim <= kOneWave ? kThreads / 64 : 1;
  const uint32_t groups = (a->rows + each - 1) / each;
  const uint32_t most = branch ? kBlockGroups : kGainGroups;
  a->blocks = groups < most ? groups : most;
  // A launch of the forward pass holds fewer than 2^32 threads.
  const int64_t threads = a->dim > kEightWaves ? 1024 : a->dim > kFourWaves ? 512 : 256;
  return (int64_t)groups * threads <= 0xffffffffLL;
}

hipError_t launch_residual(const ResidualArgs& a, int dtype, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  return dtype == REPRO_BF16 ? select<1>(a, false, stream) : select<0>(a, false, stream);
}

hipError_t launch_residual_grad(const ResidualArgs& a, int dtype, hipStream_t stream) {
  if (a.rows > 0) {
    const hipError_t e = dtype == REPRO_BF16 ? select<1>(a, true, stream) : select<0>(a, true, stream);
    if (e != hipSuccess) return e;
  }
  if (a.sums[0] == nullptr && a.sums[1] == nullptr && a.sums[2] == nullptr) return hipSuccess;
  hipLaunchKernelGGL(k_channel_fold, dim3((a.dim + kFoldColumns - 1) / kFoldColumns, 3),
                     dim3(kFoldThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace repro
