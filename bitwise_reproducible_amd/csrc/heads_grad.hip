// The backward pass of the head norm with the position rotation.
//
// "OPEN-1B: A Fully Auditable Training Run", section 3.1 (the operation that
// heads.hip describes), under its Appendix A's fixed orders.
//
// Mathematics.  With n = x r the norm's gradient needs one sum besides
// S = sum x^2, T = sum dn x, taken over the same registers at the same time:
// dx = (dn - x (T r / D) r) r.  dz is dy turned back by the same angle, and
// dn = dz gain, dgain = sum dz n.
//
// Design for gfx950 (heads.h has the lanes).  Three transfers of each element
// bound it, with some 300 vector instructions for every eight heads of 128:
//  - As the forward pass, with kHeads heads of a token in a group, x and dy
//    read once; from 32 MB on, stores go past the caches, and loads where
//    each vector is of whole cache lines (one of half a line would be fetched
//    twice: heads of 64 54 against 50 us).  The choice stands inside the loop
//    over a group's heads; as compiled, cached loads of the second head wait
//    for the first's, streamed ones do not.
//  - The gains' gradients gather in registers over a group's heads and
//    tokens, then over groups (exchanges, LDS), then one row per workgroup in
//    the workspace, folded by a second kernel.  The number of workgroups is a
//    function of the sizes, and so is the order of every sum: repro.h declares
//    it, with the numbers below, so none of them changes without the contract.
//  - With gains, the next item's loads go out before this one's arithmetic.
//    As compiled, the table's row at the top of each step waits for them and
//    for the last step's stores, and its own trip follows; and 15 to 100
//    scalars (both sides' strides and pointers) move through vector lanes.
//
// Measured on MI355X: 16384 tokens of 20 heads of 128 in bf16 (252 MB, 37 us
// at a plain copy's rate) 42.9-43.5 us a call; 50.4 with one kernel for all
// sizes, 48.4 with four heads a group, 44.1 with the table's row after the
// heads; 55.5 with gains.  8192 such tokens in binary32 with gains (252 MB)
// 49.4 us, 80.8 with eight pairs a lane; 43.2 without gains.
#include <hip/hip_runtime.h>

#include "heads.h"

namespace repro {
namespace {

// Heads of a token in a group: 2, or 1 with gains, whose gradients take the
// registers.
template <bool GAIN>
constexpr int kHeads = GAIN ? 1 : 2;

// What a group reads for one item.
template <int BF16, int V, int HEADS>
struct Fetched {
  Raw<BF16, V> xlo[HEADS], xhi[HEADS], ylo[HEADS], yhi[HEADS];
};

template <int BF16, int V, int HEADS, bool STREAM>
__device__ __forceinline__ void load_pairs(Fetched<BF16, V, HEADS>& f, int h, const char* x, const char* dy,
                                           const Lane& l) {
  constexpr int kSize = BF16 ? 2 : 4;
  f.xlo[h].template load<STREAM>(x + l.oa * kSize);
  f.xhi[h].template load<STREAM>(x + l.ob * kSize);
  f.ylo[h].template load<STREAM>(dy + l.oa * kSize);
  f.yhi[h].template load<STREAM>(dy + l.ob * kSize);
}

template <int BF16, int V, int HEADS>
__device__ __forceinline__ Fetched<BF16, V, HEADS> fetch(const HeadsArgs& a, const HeadSide& side, const Item& it,
                                                         bool on, int64_t apart, const Lane& l) {
  Fetched<BF16, V, HEADS> f = {};
  const char* x = static_cast<const char*>(side.x) + head_at<BF16>(side.x_stride, it);
  const char* dy = static_cast<const char*>(side.dy) + head_at<BF16>(side.dy_stride, it);
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    if (!on || h >= it.heads) continue;
    if (a.stream_loads) {
      keep_apart();
      load_pairs<BF16, V, HEADS, true>(f, h, x + h * apart * side.x_stride[2], dy + h * apart * side.dy_stride[2], l);
      keep_apart();
    } else {
      load_pairs<BF16, V, HEADS, false>(f, h, x + h * apart * side.x_stride[2], dy + h * apart * side.dy_stride[2], l);
    }
  }
  return f;
}

// GAIN: some side has a gain, whose gradient's row of this workgroup goes to
// side.partial[block]; workgroups then take several items in turn.
template <int BF16, int V, bool INTER, int MODE, bool GAIN>
__global__ __launch_bounds__(kThreads) void k_heads_grad(HeadsArgs a) {
  constexpr int kSize = BF16 ? 2 : 4;
  constexpr int HEADS = kHeads<GAIN>;
  const bool keys = blockIdx.x >= a.side[0].blocks;
  const HeadSide& side = a.side[keys];
  const uint32_t block = blockIdx.x - (keys ? a.side[0].blocks : 0);
  const int j = threadIdx.x & ((1 << a.log_group) - 1);
  const Lane l = lane_of<V, INTER, MODE>(a, j);
  const bool has_gain = GAIN && side.gain != nullptr;
  float g[GAIN ? 2 * V : 1], acc[GAIN ? 2 * V : 1];
  if constexpr (GAIN) {
#pragma unroll
    for (int k = 0; k < 2 * V; ++k) acc[k] = g[k] = 0.0f;  // lanes past the head must add zeros
    if (l.active && has_gain) load_gain<V>(side.gain, a.gain_bf16, l, g);
  }
  const uint32_t groups = side.blocks * (uint32_t)(kThreads >> a.log_group);
  const uint32_t mine = (block * (uint32_t)kThreads + threadIdx.x) >> a.log_group;
  const int64_t apart = (int64_t)side.by_chunks.divisor * kSize;  // between a group's heads, in head strides
  // The trip count is that of the workgroup's first group, so that whole
  // waves stay together in the exchanges; it is one without a gain.
  const uint32_t lead = block * (uint32_t)(kThreads >> a.log_group);
  const uint32_t steps = GAIN ? (side.items - lead + groups - 1) / groups : 1;
  bool live = mine < side.items;
  Item it = item_of<HEADS>(a, side, live ? mine : 0);
  Row<V> row;
  if constexpr (!GAIN) row = row_of<V>(a, live && l.rotated, it.b, it.s, l);  // before the heads, as in heads.hip
  Fetched<BF16, V, HEADS> f = fetch<BF16, V, HEADS>(a, side, it, live && l.active, apart, l);
  for (uint32_t step = 0; step < steps; ++step) {
    const bool on = live && l.active;
    if constexpr (GAIN) row = row_of<V>(a, on && l.rotated, it.b, it.s, l);
    char* out = static_cast<char*>(side.out) + head_at<BF16>(side.out_stride, it);
    const int heads = it.heads;
    float e[HEADS][2 * V], d[HEADS][2 * V], S[HEADS], r[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      widen(f.xlo[h], e[h]);
      widen(f.xhi[h], e[h] + V);
      widen(f.ylo[h], d[h]);
      widen(f.yhi[h], d[h] + V);
    }
    if constexpr (GAIN) {
      // The next item's data travels during this one's arithmetic.
      const uint64_t i = mine + (uint64_t)(step + 1) * groups;
      live = i < side.items;
      it = item_of<HEADS>(a, side, live ? (uint32_t)i : 0);
      f = fetch<BF16, V, HEADS>(a, side, it, live && l.active, apart, l);
    }
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      float t[2 * V];
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) t[k] = mul_c(e[h][k], e[h][k]);
      S[h] = head_sum<V, INTER, MODE>(t, l, a.log_group);
    }
    roots<HEADS>(a, S, r);
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      const bool counts = on && h < heads;
      if (MODE == kWhole || l.rotated) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          float& da = d[h][first_of<V, INTER>(k)];
          float& db = d[h][second_of<V, INTER>(k)];
          const float za = add_c(mul_c(da, row.c[k]), mul_c(db, row.s[k]));
          const float zb = sub_c(mul_c(db, row.c[k]), mul_c(da, row.s[k]));
          da = za;
          db = zb;
        }
      }
      // d is dz, then dn.
      float t[2 * V];
      if constexpr (GAIN) {
        if (has_gain) {
          if (counts) {
#pragma unroll
            for (int k = 0; k < 2 * V; ++k) acc[k] = add_c(acc[k], mul_c(d[h][k], mul_c(e[h][k], r[h])));
          }
#pragma unroll
          for (int k = 0; k < 2 * V; ++k) d[h][k] = mul_c(d[h][k], g[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) t[k] = mul_c(d[h][k], e[h][k]);
      const float T = head_sum<V, INTER, MODE>(t, l, a.log_group);
      const float w = mul_c(mul_c(mul_c(T, r[h]), a.inv_dim), r[h]);
      if (counts) {
#pragma unroll
        for (int k = 0; k < 2 * V; ++k) d[h][k] = mul_c(sub_c(d[h][k], mul_c(e[h][k], w)), r[h]);
        store_lane<BF16, V, INTER, MODE>(out + h * apart * side.out_stride[2], l, d[h], a.stream);
      }
    }
  }
  if constexpr (GAIN) {
    if (!has_gain) return;  // a whole workgroup is of one side
    __shared__ float part[kThreads / 64][64 * 2 * V];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    // Groups of a wave, neighbours first.
#pragma unroll
    for (int k = 0; k < 2 * V; ++k) {
      float v = acc[k];
      if (a.log_group < 3) v = add_c(v, __shfl_xor(v, 4, 64));
      if (a.log_group < 4) v = add_c(v, __shfl_xor(v, 8, 64));
      if (a.log_group < 5) v = level16(v);
      if (a.log_group < 6) v = level32(v);
      if (lane == j) part[wave][j * 2 * V + k] = v;
    }
    __syncthreads();
    if (wave == 0 && lane == j && l.active) {
      float* row = side.partial + (int64_t)block * a.dim;
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) {
        const int at = j * 2 * V + k;
        const float v = add_c(add_c(part[0][at], part[1][at]), add_c(part[2][at], part[3][at]));
        if ((l.counted >> pair_of<V, INTER>(k)) & 1u) row[k < V ? l.oa + k : l.ob + k - V] = v;
      }
    }
  }
}

// dgain[i] = the sum of a side's rows: 8 columns of a workgroup, each with
// 128 threads that take every 128th row in ascending order, then a tree.
constexpr int kFoldColumns = 8, kFoldRows = 128;
__global__ __launch_bounds__(kFoldColumns* kFoldRows) void k_gain_fold(HeadsArgs a) {
  const HeadSide& side = a.side[blockIdx.y];
  if (side.gain == nullptr) return;
  const int column = threadIdx.x % kFoldColumns, part = threadIdx.x / kFoldColumns;
  const int i = blockIdx.x * kFoldColumns + column;
  float v = 0.0f;
  if (i < a.dim) {
    const float* p = side.partial + i;
#pragma unroll 8
    for (uint32_t row = part; row < side.blocks; row += kFoldRows) v = add_c(v, p[(int64_t)row * a.dim]);
  }
  __shared__ float sums[kFoldRows][kFoldColumns];
  sums[part][column] = v;
  for (int n = kFoldRows / 2; n > 0; n >>= 1) {
    __syncthreads();
    if (part < n) sums[part][column] = add_c(sums[part][column], sums[part + n][column]);
  }
  if (part == 0 && i < a.dim) side.dgain[i] = sums[0][column];
}

// Rows of the gains' gradients in all, for the 256 compute units: 3 a unit
// with 8 pairs a lane and 5 with fewer.  All are resident at once: registers
// leave room for 4 with 8 pairs (3 for ragged halves and for binary32), for 5
// and more with fewer.  Each side's rows are rounded up for themselves, so a
// call may take one more than the number here, whose workgroup then runs
// after the others where the units are full.  Measured (us a call): 16384
// tokens in bf16 55.0 with 768, 57.2 with 640, 66.3 with 1024 (which came to
// 1025, one more than are resident), 60.6 with 2048; 8192 in binary32 49.4
// with 1280, 53.6 with 1024, 53.9 with 2048.
uint32_t gain_blocks(int vector) { return vector == 8 ? 768 : 1280; }

template <int BF16, int V, int MODE>
hipError_t run(const HeadsArgs& a, bool inter, bool gain, hipStream_t stream) {
  const dim3 grid(a.side[0].blocks + a.side[1].blocks), block(kThreads);
  if (gain) {
    if (inter)
      hipLaunchKernelGGL((k_heads_grad<BF16, V, true, MODE, true>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((k_heads_grad<BF16, V, false, MODE, true>), grid, block, 0, stream, a);
  } else {
    if (inter)
      hipLaunchKernelGGL((k_heads_grad<BF16, V, true, MODE, false>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((k_heads_grad<BF16, V, false, MODE, false>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t select(const HeadsArgs& a, int dtype, bool inter, bool gain, hipStream_t stream) {
  if (a.vector == 1)
    return dtype == REPRO_BF16 ? run<1, 1, kMixed>(a, inter, gain, stream) : run<0, 1, kMixed>(a, inter, gain, stream);
  if (dtype == REPRO_BF16) {
    if (a.vector == 4) return run<1, 4, kRagged>(a, inter, gain, stream);
    if (a.mode == kWhole) return run<1, 8, kWhole>(a, inter, gain, stream);
    return a.mode == kMixed ? run<1, 8, kMixed>(a, inter, gain, stream) : run<1, 8, kRagged>(a, inter, gain, stream);
  }
  if (a.vector == 8) return run<0, 8, kRagged>(a, inter, gain, stream);
  if (a.mode == kWhole) return run<0, 4, kWhole>(a, inter, gain, stream);
  return a.mode == kMixed ? run<0, 4, kMixed>(a, inter, gain, stream) : run<0, 4, kRagged>(a, inter, gain, stream);
}

}  // namespace

bool plan_heads_backward(HeadsArgs* a, int dtype) {
  const bool gain = a->side[0].gain != nullptr || a->side[1].gain != nullptr;
  if (!plan_heads(a, dtype, gain ? kHeads<true> : kHeads<false>)) return false;
  if (!gain) return true;
  // Items that a group takes in turn, the same on both sides.
  const uint32_t most = gain_blocks(a->vector);
  const uint32_t steps = (a->side[0].blocks + a->side[1].blocks + most - 1) / most;
  for (HeadSide& side : a->side)
    if (steps > 1) side.blocks = (side.blocks + steps - 1) / steps;
  return true;
}

hipError_t launch_heads_grad(const HeadsArgs& a, int dtype, bool inter, hipStream_t stream) {
  const bool gain = a.side[0].gain != nullptr || a.side[1].gain != nullptr;
  if (a.side[0].blocks + a.side[1].blocks > 0) {
    const hipError_t e = select(a, dtype, inter, gain, stream);
    if (e != hipSuccess) return e;
  }
  if (!gain) return hipSuccess;
  hipLaunchKernelGGL(k_gain_fold, dim3((a.dim + kFoldColumns - 1) / kFoldColumns, 2),
                     dim3(kFoldColumns * kFoldRows), 0, stream, a);
  return hipGetLastError();
}

}  // namespace repro
