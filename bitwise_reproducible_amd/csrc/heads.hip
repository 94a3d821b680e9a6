// The norm of every query and key head with the position rotation, in one
// pass.
//
// "OPEN-1B: A Fully Auditable Training Run", section 3.1: the pages' model
// normalises query and key heads and rotates them by position.
//
// Mathematics (repro.h has it element by element).  S = sum x^2 of a head of
// D elements gives r = 1/sqrt(S/D + eps); x r (times a gain) is rotated in
// pairs.  The head is read once and stays in registers: the sum is a tree
// inside a few lanes, and the result leaves from the registers it came into.
//
// Design for gfx950 (heads.h has the lanes).  Two transfers of each element
// bound it, and some 200 vector instructions for every eight heads of 128 come
// close behind, so both are kept down:
//  - A lane holds V = 8 pairs of bf16 or 4 of binary32: 16-byte loads.
//  - A group takes the same token of up to kHeads heads and keeps the table's
//    row in registers between them; the roots of its heads are taken by
//    different lanes.  The loads of all its heads travel together, but as
//    compiled they go out only once most of the row is there: two trips to
//    memory in turn, three with positions, which covers itself where many
//    waves are resident and not in short calls.
//  - The sums' exchanges stay inside the vector unit: no LDS traffic.
//  - The raw vectors are widened twice rather than held wide.
//  - Sizes that leave no ragged lanes or no passing part run kernels without
//    the code for them.
//  - From 32 MB on, results are stored past the caches.
//
// Measured on MI355X, 16384 tokens of 20 heads of 128 in bf16 (168 MB in all,
// 25 us at a plain copy's rate): 26.5-26.9 us a call, 27.6 with gains; 8192
// such tokens in binary32 26.4.  Before: 38.8 with one kernel for all sizes
// and every root in every lane, 36.5 without nontemporal stores, 28.0 with
// four heads a group, 32.0 at six waves a SIMD with spills.
#include <hip/hip_runtime.h>

#include "heads.h"

namespace repro {
namespace {

constexpr int kHeads = 2;

template <int BF16, int V, bool INTER, int MODE>
__global__ __launch_bounds__(kThreads, 5) void k_heads(HeadsArgs a) {
  constexpr int kSize = BF16 ? 2 : 4;
  const bool keys = blockIdx.x >= a.side[0].blocks;
  const HeadSide& side = a.side[keys];
  const uint32_t block = blockIdx.x - (keys ? a.side[0].blocks : 0);
  const uint32_t group = (block * (uint32_t)kThreads + threadIdx.x) >> a.log_group;
  const Lane l = lane_of<V, INTER, MODE>(a, threadIdx.x & ((1 << a.log_group) - 1));
  const bool live = group < side.items;
  const Item it = item_of<kHeads>(a, side, live ? group : 0);
  const char* x = static_cast<const char*>(side.x) + head_at<BF16>(side.x_stride, it);
  const int64_t step = (int64_t)side.by_chunks.divisor * kSize;  // between a group's heads, in head strides
  const bool on = live && l.active;
  // The row before the heads: its branch is left with a part of it in
  // registers, so the compiler waits for it there, and the other way round
  // that wait would be for the heads as well.
  const Row<V> row = row_of<V>(a, on && l.rotated, it.b, it.s, l);

  Raw<BF16, V> lo[kHeads], hi[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    lo[h] = {};
    hi[h] = {};
    if (on && h < it.heads) {
      const char* p = x + h * step * side.x_stride[2];
      lo[h].template load<false>(p + l.oa * kSize);
      hi[h].template load<false>(p + l.ob * kSize);
    }
  }

  float S[kHeads], r[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    float t[2 * V];
    widen(lo[h], t);
    widen(hi[h], t + V);
#pragma unroll
    for (int k = 0; k < 2 * V; ++k) t[k] = mul_c(t[k], t[k]);
    S[h] = head_sum<V, INTER, MODE>(t, l, a.log_group);
  }
  roots<kHeads>(a, S, r);
  if (!on) return;
  char* out = static_cast<char*>(side.out) + head_at<BF16>(side.out_stride, it);
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (h >= it.heads) return;
    float e[2 * V];
    forget(lo[h]);
    forget(hi[h]);
    widen(lo[h], e);
    widen(hi[h], e + V);
#pragma unroll
    for (int k = 0; k < 2 * V; ++k) e[k] = mul_c(e[k], r[h]);
    if (side.gain != nullptr) {
      float g[2 * V];  // from the cache for each head: held, they would cost an eighth of the waves
      load_gain<V>(side.gain, a.gain_bf16, l, g);
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) e[k] = mul_c(e[k], g[k]);
    }
    if (MODE == kWhole || l.rotated) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float& ea = e[first_of<V, INTER>(k)];
        float& eb = e[second_of<V, INTER>(k)];
        const float ya = sub_c(mul_c(ea, row.c[k]), mul_c(eb, row.s[k]));
        const float yb = add_c(mul_c(eb, row.c[k]), mul_c(ea, row.s[k]));
        ea = ya;
        eb = yb;
      }
    }
    store_lane<BF16, V, INTER, MODE>(out + h * step * side.out_stride[2], l, e, a.stream);
  }
}

template <int BF16, int V, int MODE>
hipError_t run(const HeadsArgs& a, bool inter, hipStream_t stream) {
  const dim3 grid(a.side[0].blocks + a.side[1].blocks), block(kThreads);
  if (inter)
    hipLaunchKernelGGL((k_heads<BF16, V, true, MODE>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((k_heads<BF16, V, false, MODE>), grid, block, 0, stream, a);
  return hipGetLastError();
}

// Pairs of a lane.  16-byte vectors (8 pairs of bf16, 4 of binary32) wherever
// a head then fills most of four lanes, which a group has at least; a binary32
// head beyond 256 takes 8 to fit the wave.
int vector_of(int dtype, int dim) {
  if (dim < 16) return 1;
  if (dtype == REPRO_BF16) return dim <= 32 ? 4 : 8;
  return dim <= 256 ? 4 : 8;
}

FastDiv divide_by(uint32_t d) {
  FastDiv f = {d, 0, 0};
  int s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  if (s > 0) {
    // ceil(2^(31+s) / d), below 2^32; exact for numerators below 2^31.
    f.factor = (uint32_t)(((uint64_t(1) << (31 + s)) + d - 1) / d);
    f.shift = s - 1;
  }
  return f;
}

}  // namespace

bool plan_heads(HeadsArgs* a, int dtype, int per) {
  const int V = vector_of(dtype, a->dim);
  const int passing = a->dim / 2 - a->half;
  a->rot_lanes = (a->half + V - 1) / V;
  a->lanes = a->rot_lanes + (passing + V - 1) / V;
  const bool ragged = a->half % V != 0 || passing % V != 0;
  a->vector = V;
  a->mode = ragged ? kRagged : (passing > 0 ? kMixed : kWhole);
  a->log_group = 2;
  while ((1 << a->log_group) < a->lanes) ++a->log_group;
  a->by_seq = divide_by(a->seq > 0 ? a->seq : 1);
  const uint32_t groups = kThreads >> a->log_group;
  for (HeadSide& side : a->side) {
    const int64_t chunks = ((int64_t)side.heads + per - 1) / per;
    const int64_t items = chunks * a->tokens;
    if (items > 0x7fffffff) return false;
    side.items = (uint32_t)items;
    side.by_chunks = divide_by(chunks > 0 ? (uint32_t)chunks : 1);
    side.blocks = (uint32_t)((items + groups - 1) / groups);
  }
  // A launch holds fewer than 2^32 threads.
  return ((int64_t)a->side[0].blocks + a->side[1].blocks) * kThreads <= 0xffffffffLL;
}

bool plan_heads_forward(HeadsArgs* a, int dtype) { return plan_heads(a, dtype, kHeads); }

hipError_t launch_heads(const HeadsArgs& a, int dtype, bool inter, hipStream_t stream) {
  if (a.side[0].blocks + a.side[1].blocks == 0) return hipSuccess;
  if (a.vector == 1) return dtype == REPRO_BF16 ? run<1, 1, kMixed>(a, inter, stream) : run<0, 1, kMixed>(a, inter, stream);
  if (dtype == REPRO_BF16) {
    if (a.vector == 4) return run<1, 4, kRagged>(a, inter, stream);
    if (a.mode == kWhole) return run<1, 8, kWhole>(a, inter, stream);
    return a.mode == kMixed ? run<1, 8, kMixed>(a, inter, stream) : run<1, 8, kRagged>(a, inter, stream);
  }
  if (a.vector == 8) return run<0, 8, kRagged>(a, inter, stream);
  if (a.mode == kWhole) return run<0, 4, kWhole>(a, inter, stream);
  return a.mode == kMixed ? run<0, 4, kMixed>(a, inter, stream) : run<0, 4, kRagged>(a, inter, stream);
}

}  // namespace repro
