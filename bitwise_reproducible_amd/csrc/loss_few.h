// The vocabulary loss for few tokens: the same words as the tiles of loss.hip
// give, from kernels that the embedding streams through once for each product.
//
// Mathematics.  As loss.hip.  The 16 x 16 matrix instructions take 32 k at
// once, in the groups of eight that the 32 x 32 ones take.
//
// Design for gfx950.  With up to 64 tokens reading the embedding bounds both
// products of each pass, so it goes from memory to registers without a stop:
// binary32 rows are split there, where the tiles need a copy of three planes
// (2.5 times the embedding's bytes written and read), and rows of any
// alignment are read as they lie.  More binary32 tokens run in groups, of 128 for
// the logits (up to 1024 tokens forward, 256 backward) and of 64 for dx.  Width
// 2048, 128256 entries in binary32: 246 to 267 us forward for 8 tokens (4.1 TB/s),
// 262 to 289 for 64; backward 890 for 16.
#pragma once

#include <hip/hip_runtime.h>

#include "product.h"
#include "rows.h"

namespace repro {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Planes of eight elements, as fragments.
template <int BF16>
__device__ __forceinline__ void fragments(const Raw<BF16, 8>& r, bf8 (&f)[BF16 ? 1 : 3]) {
  uint32_t w[BF16 ? 1 : 3][4];
  planes_of<BF16>(r, w);
#pragma unroll
  for (int p = 0; p < (BF16 ? 1 : 3); ++p) f[p] = __builtin_bit_cast(bf8, (u4){w[p][0], w[p][1], w[p][2], w[p][3]});
}

// acc goes on over 32 k: one product, or the six parts of one.
template <int BF16>
__device__ __forceinline__ void chain(const bf8 (&a)[BF16 ? 1 : 3], const bf8 (&b)[BF16 ? 1 : 3], f32x4& acc) {
#pragma unroll
  for (int p = 0; p < (BF16 ? 1 : kParts); ++p)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[BF16 ? 0 : plane_a(p)], b[BF16 ? 0 : plane_b(p)], acc, 0, 0, 0);
}

constexpr int kLogitPitch = 132;  // floats from one token's logits in the LDS to the next's

// The statistics of a block's logits, l[token][entry], or their dl (GRAD).
// last: no tokens come behind these ones.
template <int BF16, int kTokens, bool GRAD>
__device__ __forceinline__ void finish(const LossArgs& a, const float* l, int64_t first, int64_t entry, uint32_t token0,
                                       bool last, uint16_t* dl, int64_t plane, int64_t pitch) {
  constexpr int kPlanes = BF16 ? 1 : 3;
  const int left = (int)(a.vocab - entry < 128 ? a.vocab - entry : 128);
  if constexpr (GRAD) {
    // Eight entries of a token for each thread.
    for (int at = threadIdx.x; at < kTokens * 16; at += 256) {
      const uint32_t token = token0 + at / 16;
      const int e0 = at % 16 * 8;
      if (token >= a.padded_tokens) continue;
      const float4 mine = a.per_token[token];
      const float* from = l + at / 16 * kLogitPitch + e0;
      const int y = __float_as_int(mine.w) - (int)entry - e0;
      float d[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        d[k] = mul_c(power_of_two(__builtin_fmaf(from[k], kLog2e, -mine.x)), mine.y);
        if (k == y) d[k] = sub_c(d[k], mine.z);
        if (e0 + k >= left) d[k] = 0.0f;
      }
      Raw<BF16, 8> v = narrow<BF16, 8>(d);
      uint32_t words[kPlanes][4];
      planes_of<BF16>(v, words);
#pragma unroll
      for (int p = 0; p < kPlanes; ++p)
        *reinterpret_cast<u4*>(dl + p * plane + token * pitch + (entry - first) + e0) =
            u4{words[p][0], words[p][1], words[p][2], words[p][3]};
    }
    // No token: zeros for the sums over them.
    if (last && token0 + kTokens < a.padded_tokens) {
      for (uint32_t at = threadIdx.x; at < (a.padded_tokens - (token0 + kTokens)) * 16; at += 256)
#pragma unroll
        for (int p = 0; p < kPlanes; ++p)
          *reinterpret_cast<u4*>(dl + p * plane + (token0 + kTokens + at / 16) * pitch + (entry - first) + at % 16 * 8) = u4{};
    }
  } else {
    // A chain of a token for each thread, eight neighbours a token.
    for (int at = threadIdx.x; at < kTokens * 8; at += 256) {
      const uint32_t token = token0 + at / 8;
      const int c = at % 8;
      const float* from = l + at / 8 * kLogitPitch + c;
      float most = -__builtin_inff();
      bool odd = false;
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const float v = c + 8 * u < left ? from[8 * u] : -__builtin_inff();
        most = fmaxf(most, v);
        odd |= !(v == v);
      }
#pragma unroll
      for (int m = 1; m < 8; m *= 2) most = fmaxf(most, __shfl_xor(most, m, 64));
      const float n = __builtin_rintf(mul_c(most, kLog2e));
      const float shift = n == -__builtin_inff() ? 0.0f : n;
      float s = 0.0f;
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const float v = c + 8 * u < left ? from[8 * u] : -__builtin_inff();
        const float e = power_of_two(__builtin_fmaf(v, kLog2e, -shift));
        s = u == 0 ? e : add_c(s, e);
      }
      if (odd || n == __builtin_inff()) s = __builtin_nanf("");
#pragma unroll
      for (int m = 1; m < 8; m *= 2) s = add_c(s, __shfl_xor(s, m, 64));
      if (token >= a.tokens) continue;
      if (c == 0) a.stats[entry / 128 * a.padded_tokens + token] = make_float2(n, s);
      const int64_t y = label_of(a, token) - entry;
      if (y >= 0 && y < left && (y & 7) == c) a.picked[token] = from[y - c];
    }
  }
}

// Logits of a block of 128 entries and NT * 16 tokens, four waves of 32 entries
// each, to l[token][entry]; then their statistics, or dl (GRAD).
template <int BF16, int NT, bool GRAD>
__global__ __launch_bounds__(256) void k_few_logits(LossArgs a, Operand x, int64_t first, uint16_t* dl, int64_t plane,
                                                    int64_t pitch) {
  constexpr int kPlanes = BF16 ? 1 : 3, kSize = BF16 ? 2 : 4, kTokens = NT * 16;
  constexpr int kAhead = BF16 ? 8 : 4;  // steps of 32 k whose entries are under way: 16 KB a wave
  __shared__ __attribute__((aligned(16))) float l[kTokens * kLogitPitch];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const uint32_t groups = (uint32_t)((a.tokens + kTokens - 1) / kTokens);
  const int64_t entry = first + (int64_t)(blockIdx.x / groups) * 128;
  const uint32_t token0 = blockIdx.x % groups * kTokens;
  const char* w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t row = entry + wave * 32 + i * 16 + r;
    w[i] = static_cast<const char*>(a.w) + (row < a.vocab ? row : a.vocab - 1) * a.w_stride * kSize;
  }
  const uint16_t* xr[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t row = token0 + t * 16 + r;
    xr[t] = x.at + (row < x.rows ? row : x.rows - 1) * x.pitch + 8 * q;
  }
  const int whole = a.dim / 32, steps = (a.dim + 31) / 32;
  const auto load = [&](int i, int step) {
    const int o = step * 32 + 8 * q;
    Raw<BF16, 8> v = {};
    if (step < whole)
      v.template load<false>(w[i] + (int64_t)o * kSize);
    else if (step < steps)
      v = load8<BF16, false>(w[i], o, a.dim);
    return v;
  };
  Raw<BF16, 8> ahead[kAhead][2];
#pragma unroll
  for (int s = 0; s < kAhead; s += 2)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ahead[s][i] = load(i, s);
      ahead[s + 1][i] = load(i, s + 1);
    }
  f32x4 acc[2][NT] = {};
  const auto load_x = [&](int step, bf8 (*b)[kPlanes]) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int p = 0; p < kPlanes; ++p)
        b[t][p] = *reinterpret_cast<const bf8*>(xr[t] + p * x.plane + (int64_t)step * 32);
  };
  bf8 b[2][NT][kPlanes];
  load_x(0, b[0]);
  for (int s0 = 0; s0 < steps; s0 += kAhead) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const int s = s0 + d;
      if (s >= steps) break;
      if (s + 1 < steps) load_x(s + 1, b[(d + 1) & 1]);
      bf8 f[2][kPlanes];
#pragma unroll
      for (int i = 0; i < 2; ++i) fragments<BF16>(ahead[d][i], f[i]);
      // Both halves of a cache line at once (64 k of bf16).
      if (d & 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ahead[d - 1][i] = load(i, s - 1 + kAhead);
          ahead[d][i] = load(i, s + kAhead);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) chain<BF16>(f[i], b[d & 1][t], acc[i][t]);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<f32x4*>(l + (t * 16 + r) * kLogitPitch + wave * 32 + i * 16 + 4 * q) = acc[i][t];
  __syncthreads();
  finish<BF16, kTokens, GRAD>(a, l, first, entry, token0, blockIdx.x % groups == groups - 1, dl, plane, pitch);
}

// The same for binary32 from rows of 4-byte alignment, TN * 32 tokens: the
// embedding goes to the LDS as it is, and each of the four waves splits the 32
// rows that it alone reads; the tokens' planes go there beside it.  A stage is
// 32 k of all, six products of three and three planes.  Two workgroups of a
// compute unit run beside each other: one splits while the other multiplies.
// 517 tokens of width 1001 over 32003 entries: 231 us, 236 to 258 a call.
template <int TN, bool GRAD>
__global__ __launch_bounds__(256, 2) void k_split_logits(LossArgs a, Operand x, int64_t first, uint16_t* dl,
                                                         int64_t plane, int64_t pitch) {
  constexpr int kTokens = TN * 32, kStages = 2;
  constexpr int kLoadsW = 4, kLoadsX = kTokens / 64;  // transfers of a wave: of the embedding, of a plane
  constexpr int kLoads = kLoadsW + 3 * kLoadsX;
  constexpr uint32_t kBytesW = 128 * 128, kBytesX = kTokens * 64, kStageBytes = kBytesW + 3 * kBytesX;
  static_assert(kTokens * kLogitPitch * 4 <= kStages * kStageBytes, "the logits take the ring's place");
  __shared__ __attribute__((aligned(1024))) char ring[kStages * kStageBytes];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t r = lane & 31, h = lane >> 5;
  const uint32_t groups = (uint32_t)((a.tokens + kTokens - 1) / kTokens);
  const int64_t entry = first + (int64_t)(blockIdx.x / groups) * 128;
  const uint32_t token0 = blockIdx.x % groups * kTokens;
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)ring;

  // The embedding's rows: eight pieces of 16 bytes, which turn with the row.
  const uint32_t w_pitch = (uint32_t)(a.w_stride * 4);
  // (dl's width goes on to a multiple of 256 entries: none may be left here.
  // Such a workgroup transfers nothing, and stores zeros.)
  const int rows = (int)(a.vocab - entry < 128 ? a.vocab - entry : 128);
  const i32x4 w_buffer = buffer_of(reinterpret_cast<const uint16_t*>(static_cast<const float*>(a.w) + entry * a.w_stride),
                                   rows > 0 ? (rows - 1) * w_pitch + (uint32_t)a.dim * 4 : 0);
  const auto turn = [](uint32_t row) { return (row & 7) ^ ((row >> 3) & 1); };
  uint32_t w_off[kLoadsW];
#pragma unroll
  for (int i = 0; i < kLoadsW; ++i) {
    const uint32_t row = (wave * kLoadsW + i) * 8 + (lane >> 3);
    w_off[i] = row * w_pitch + ((lane & 7) ^ turn(row)) * 16;
  }
  typedef Stages<false, kTokens, 4, TN> X;
  const int64_t x_left = x.rows - token0;
  const int x_rows = x_left < kTokens ? (int)x_left : kTokens;
  const Side16 side = {x.at + token0 * x.pitch, x.plane, (uint32_t)(x.pitch * 2),
                       (uint32_t)((x_rows - 1) * x.pitch * 2 + a.k * 2), 0};
  X xs(side, wave, lane, 0);
  i32x4 x_buffer[3];
#pragma unroll
  for (int p = 0; p < 3; ++p) x_buffer[p] = xs.buffer(p);
  uint32_t soffset = 0;
  const auto issue = [&](int slot) {
    const uint32_t at = base + slot * kStageBytes;
#pragma unroll
    for (int i = 0; i < kLoadsW; ++i) to_lds(at + (wave * kLoadsW + i) * 1024, w_off[i], w_buffer, soffset);
#pragma unroll
    for (int p = 0; p < 3; ++p) xs.issue(x_buffer[p], at + kBytesW + p * kBytesX, wave, 0, kLoadsX);
    soffset += 128;
    xs.advance();
  };

  const int steps = rows > 0 ? (a.dim + 31) / 32 : 0;
  f32x16 acc[TN] = {};
  const uint32_t own = (wave * 32 + r) * 128;
  if (steps > 0) issue(0);
  for (int s = 0; s < steps; ++s) {
    wait_stage<0>();
    if (s + 1 < steps) issue((s + 1) & 1);
    const char* at = ring + (s & 1) * kStageBytes;
    bf8 f[2][3];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      Raw<0, 8> v;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v.w[i] = *reinterpret_cast<const u4*>(at + own + ((half * 4 + h * 2 + i) ^ turn(r)) * 16);
      if (s == steps - 1) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (s * 32 + half * 16 + (int)h * 8 + k >= a.dim) v.w[k >> 2][k & 3] = 0;
      }
      fragments<0>(v, f[half]);
    }
    s16x4 b[TN][3][2][2];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int half = 0; half < 2; ++half) xs.read(at + kBytesW + p * kBytesX, half, j, 0, b[j][p][half]);
#pragma unroll
    for (int part = 0; part < kParts; ++part)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const s16x4(&v)[2] = b[j][plane_b(part)][half];
          acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              f[half][plane_a(part)],
              __builtin_bit_cast(bf8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7)), acc[j], 0, 0, 0);
        }
  }
  __syncthreads();
  float* l = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<f32x4*>(l + (j * 32 + r) * kLogitPitch + wave * 32 + 8 * q + 4 * h) =
          f32x4{acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
  __syncthreads();
  finish<0, kTokens, GRAD>(a, l, first, entry, token0, blockIdx.x % groups == groups - 1, dl, plane, pitch);
}

// dx's sums over the spans of a piece, as k_dx: a wave has 16 E columns (E: a
// 16-byte vector's elements) of NT * 16 tokens.  A lane loads E neighbouring
// columns of eight rows; matrix tile t takes the columns t of each lane, so the
// rows of a fragment are E apart and eight k meet in one lane.
template <int BF16, int NT>
__global__ __launch_bounds__(64) void k_few_dx(LossArgs a, int64_t first, int64_t entries, Operand dl, int64_t span,
                                               float* partial, int64_t width) {
  constexpr int kPlanes = BF16 ? 1 : 3, E = BF16 ? 8 : 4, kSize = BF16 ? 2 : 4, kTokens = NT * 16;
  const int lane = threadIdx.x, r = lane & 15, q = lane >> 4;
  const uint32_t columns = (uint32_t)(width / (16 * E)), groups = (uint32_t)((a.tokens + kTokens - 1) / kTokens);
  const uint32_t z = blockIdx.x / (columns * groups), rest = blockIdx.x % (columns * groups);
  const uint32_t token0 = rest % groups * kTokens;
  const int d0 = (int)(rest / groups) * 16 * E + E * r;
  const int64_t k0 = z * span, k1 = k0 + span < dl.columns ? k0 + span : dl.columns;
  const char* w = static_cast<const char*>(a.w) + first * a.w_stride * kSize;
  const bool full = d0 + E <= a.dim;
  const auto load = [&](int64_t k, u4 (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      int64_t row = k + 8 * q + j;
      if (row >= entries) row = entries - 1;  // dl is zero there
      const char* at = w + (row * a.w_stride + d0) * kSize;
      v[j] = u4{};
      if (full) {
        if constexpr (BF16)
          v[j] = *reinterpret_cast<const u4_2*>(at);
        else
          v[j] = *reinterpret_cast<const u4_4*>(at);
      } else if (d0 < a.dim) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (d0 + e >= a.dim) continue;
          if constexpr (BF16)
            v[j][e >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(at)[e] << (16 * (e & 1));
          else
            v[j][e] = reinterpret_cast<const uint32_t*>(at)[e];
        }
      }
    }
  };
  const uint16_t* dr[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint32_t row = token0 + t * 16 + r;
    dr[t] = dl.at + (int64_t)(row < a.padded_tokens ? row : a.padded_tokens - 1) * dl.pitch + 8 * q;
  }
  const auto load_dl = [&](int64_t k, bf8 (*b)[kPlanes]) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int p = 0; p < kPlanes; ++p) b[t][p] = *reinterpret_cast<const bf8*>(dr[t] + p * dl.plane + k);
  };
  f32x4 acc[E][NT] = {};
  u4 ahead[2][8];
  bf8 b[2][NT][kPlanes];
  load(k0, ahead[0]);
  load_dl(k0, b[0]);
  for (int64_t k = k0; k < k1; k += 64) {  // k1 - k0 is a multiple of 256
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const int64_t next = k + 32 * (d + 1);
      if (next < k1) {
        load(next, ahead[d ^ 1]);
        load_dl(next, b[d ^ 1]);
      }
#pragma unroll
      for (int t = 0; t < E; ++t) {
        bf8 f[kPlanes];
        if constexpr (BF16) {
          u4 word;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            word[j] = __builtin_amdgcn_perm(ahead[d][2 * j + 1][t >> 1], ahead[d][2 * j][t >> 1],
                                            t & 1 ? 0x07060302u : 0x05040100u);
          f[0] = __builtin_bit_cast(bf8, word);
        } else {
          Raw<0, 8> v;
#pragma unroll
          for (int j = 0; j < 8; ++j) v.w[j >> 2][j & 3] = ahead[d][j][t];
          fragments<0>(v, f);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) chain<BF16>(f, b[d][n], acc[t][n]);
      }
    }
  }
  // Lane (token r of 16, rows 4 q ..): tile t's row m is column E m + t.
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint32_t token = token0 + n * 16 + r;
    if (token >= a.padded_tokens) continue;
    float* to = partial + ((int64_t)z * a.padded_tokens + token) * width + (rest / groups) * 16 * E;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int t = 0; t < E; t += 4)
        *reinterpret_cast<f32x4*>(to + E * (4 * q + m) + t) =
            f32x4{acc[t][n][m], acc[t + 1][n][m], acc[t + 2][n][m], acc[t + 3][n][m]};
  }
}

}  // namespace
}  // namespace repro
