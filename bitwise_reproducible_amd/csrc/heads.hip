// The norm of every query and key head with the position rotation in the
// same pass, and its backward pass.
//
// "OPEN-1B: A Fully Auditable Training Run", section 3.1: the pages' model
// normalises query and key heads and rotates them by position.
//
// Mathematics (repro.h has it element by element).  A head is D elements in
// pairs; S = sum x^2 gives r = 1/sqrt(S/D + eps), and since n = x r the
// backward pass needs one more sum only, T = sum dn x, which is taken over
// the same registers at the same time as S: dx = (dn - n (T r / D)) r.  So
// each head is read once, both sums are trees inside a few lanes, and the
// result leaves from the registers it came into.
//
// Design for gfx950 (memory bound: two transfers of each element forward,
// three backward):
//  - A group of lanes, a power of two, holds one head: a lane has V pairs in
//    two vectors of V elements, lo and hi.  Without interleaving lo and hi
//    are the halves' vectors at i and i + h, so that a rotated pair meets in
//    one lane and no element crosses lanes; interleaved (and in the part
//    that passes) they are 2V neighbours.  V = 8: 16-byte loads of bf16, and
//    a head of 128 is eight lanes.
//  - Sections (rotated, passing) whose pair count V does not divide end in a
//    lane whose vectors are moved back to the section's end.  The elements
//    it shares with its neighbour are left out of its sums; both lanes store
//    the same bits to them.  A section of fewer than V pairs is one lane that
//    stores element by element.
//  - A group takes the same token of up to kHeads heads and keeps the table's
//    row and the gains in registers between them.
//  - The tree of S and T: pair sums within the lane, then lanes by exchanges
//    inside the vector unit (lane rows and half-rows mirrored, the two last
//    levels by row swaps): no LDS traffic.
//  - The gains' gradients gather in registers over a group's heads and
//    tokens, then over groups (exchanges, LDS), then one row per workgroup
//    in the workspace, folded by a second kernel.  The number of workgroups
//    is a function of the sizes, so is the order of every sum.
#include <hip/hip_runtime.h>

#include "device_ops.h"
#include "internal.h"

namespace repro {
namespace {

constexpr int kThreads = 256;

// Vectors of V elements at any element's alignment (gfx950 loads and stores
// 4, 8 and 16 bytes at any address).
template <int BF16, int V>
struct Raw;
typedef uint32_t u4_2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u4_4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

template <>
struct Raw<1, 8> {
  u4 w;
  __device__ void load(const void* p) { w = *static_cast<const u4_2*>(p); }
  __device__ void store(void* p) const { *static_cast<u4_2*>(p) = w; }
  __device__ uint32_t bits(int i) const { return w[i >> 1] >> (16 * (i & 1)); }
};
template <>
struct Raw<1, 1> {
  uint16_t w;
  __device__ void load(const void* p) { w = *static_cast<const uint16_t*>(p); }
  __device__ void store(void* p) const { *static_cast<uint16_t*>(p) = w; }
  __device__ uint32_t bits(int) const { return w; }
};
template <>
struct Raw<0, 8> {
  u4 w[2];
  __device__ void load(const void* p) {
    w[0] = static_cast<const u4_4*>(p)[0];
    w[1] = static_cast<const u4_4*>(p)[1];
  }
  __device__ void store(void* p) const {
    static_cast<u4_4*>(p)[0] = w[0];
    static_cast<u4_4*>(p)[1] = w[1];
  }
  __device__ uint32_t bits(int i) const { return w[i >> 2][i & 3]; }
};
template <>
struct Raw<0, 4> {
  u4 w;
  __device__ void load(const void* p) { w = *static_cast<const u4_4*>(p); }
  __device__ void store(void* p) const { *static_cast<u4_4*>(p) = w; }
  __device__ uint32_t bits(int i) const { return w[i]; }
};
template <>
struct Raw<0, 1> {
  uint32_t w;
  __device__ void load(const void* p) { w = *static_cast<const uint32_t*>(p); }
  __device__ void store(void* p) const { *static_cast<uint32_t*>(p) = w; }
  __device__ uint32_t bits(int) const { return w; }
};

template <int BF16, int V>
__device__ __forceinline__ void widen(const Raw<BF16, V>& r, float* x) {
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = __uint_as_float(BF16 ? r.bits(i) << 16 : r.bits(i));
}

// Rounding to bf16 is to nearest, ties to even, once per element.
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef float fl2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t round2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((fl2{a, b}), bf2));
}

template <int BF16, int V>
__device__ __forceinline__ Raw<BF16, V> narrow(const float* x) {
  Raw<BF16, V> r;
  if constexpr (BF16 && V == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = round2(x[2 * i], x[2 * i + 1]);
  } else if constexpr (BF16) {
    r.w = (uint16_t)round2(x[0], 0.0f);
  } else if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i >> 2][i & 3] = __float_as_uint(x[i]);
  } else if constexpr (V == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = __float_as_uint(x[i]);
  } else {
    r.w = __float_as_uint(x[0]);
  }
  return r;
}

// v + the value of the lane whose index differs in bit K, or any lane that
// holds the same value there: after the levels below K all lanes of a 2^K
// block are equal.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float level16(float v) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return add_c(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float level32(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return add_c(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
// Perfect tree over the 2^log_group lanes of a group (uniform branches).
__device__ __forceinline__ float group_sum(float v, int log_group) {
  if (log_group > 0) v = add_c(v, dpp<0xB1>(v));   // lanes 1,0,3,2 of each four
  if (log_group > 1) v = add_c(v, dpp<0x4E>(v));   // lanes 2,3,0,1 of each four
  if (log_group > 2) v = add_c(v, dpp<0x141>(v));  // mirrored in each eight
  if (log_group > 3) v = add_c(v, dpp<0x140>(v));  // mirrored in each sixteen
  if (log_group > 4) v = level16(v);
  if (log_group > 5) v = level32(v);
  return v;
}

template <int V>
__device__ __forceinline__ float tree(const float* t) {
  float u[V];
#pragma unroll
  for (int i = 0; i < V; ++i) u[i] = t[i];
#pragma unroll
  for (int n = V; n > 1; n >>= 1)
#pragma unroll
    for (int i = 0; i < n / 2; ++i) u[i] = add_c(u[2 * i], u[2 * i + 1]);
  return u[0];
}

// What one lane of a group holds.  Element k < V of a lane is lo[k], at
// oa + k; element V + k is hi[k], at ob + k.
struct Lane {
  int oa, ob;
  uint32_t counted;  // bit k: element k is this lane's in the sums
  int slot;          // first rotated pair (rotated lanes)
  bool active, rotated, part;  // part: only the counted elements are stored
};

// Bit k of m becomes bits 2k and 2k + 1 (m < 2^8).
__device__ __forceinline__ uint32_t doubled(uint32_t m) {
  m = (m | (m << 4)) & 0x0F0Fu;
  m = (m | (m << 2)) & 0x3333u;
  m = (m | (m << 1)) & 0x5555u;
  return m | (m << 1);
}

template <int V, bool INTER>
__device__ __forceinline__ Lane lane_of(const HeadsArgs& a, int j) {
  constexpr uint32_t kSlots = (1u << V) - 1u, kAll = (1u << (2 * V)) - 1u;
  const int half = a.half, pairs = a.dim / 2 - half;  // rotated and passing pairs
  Lane l;
  l.active = j < a.lanes;
  l.rotated = j < a.rot_lanes;
  // Pairs of the section before this lane's vectors, had they not been moved
  // back, and where they begin; negative: before the section.
  const int want = (l.rotated ? j : j - a.rot_lanes) * V;
  const int count = l.rotated ? half : pairs;
  const int moved = min(want, count - V);
  l.part = count < V;
  l.slot = l.rotated ? max(moved, 0) : 0;
  if (l.rotated) {
    const uint32_t slots = (half < V ? (1u << half) - 1u : kSlots) & ~((1u << (want - l.slot)) - 1u);
    l.oa = INTER ? 2 * l.slot : l.slot;
    l.ob = INTER ? l.oa + V : l.slot + half;
    l.counted = INTER ? doubled(slots) : slots | (slots << V);
  } else {
    l.oa = 2 * (half + moved);
    l.ob = l.oa + V;
    l.counted = l.active ? kAll & ~((1u << (2 * (want - moved))) - 1u) : 0u;
  }
  return l;
}

template <int V>
__device__ __forceinline__ void load_gain(const void* gain, int is_bf16, const Lane& l, float* lo, float* hi) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (is_bf16) {
      const uint16_t* g = static_cast<const uint16_t*>(gain);
      lo[k] = __uint_as_float((uint32_t)g[l.oa + k] << 16);
      hi[k] = __uint_as_float((uint32_t)g[l.ob + k] << 16);
    } else {
      lo[k] = static_cast<const float*>(gain)[l.oa + k];
      hi[k] = static_cast<const float*>(gain)[l.ob + k];
    }
  }
}

// The row of (batch b, token s) in the table; -1 outside it.
__device__ __forceinline__ int64_t table_row(const HeadsArgs& a, uint32_t b, uint32_t s) {
  int64_t p = s;
  if (a.positions != nullptr) {
    const int64_t at = b * a.pos_stride[0] + s * a.pos_stride[1];
    p = a.pos64 ? static_cast<const int64_t*>(a.positions)[at] : static_cast<const int32_t*>(a.positions)[at];
  }
  return p >= 0 && p < a.table_rows ? p : -1;
}

// V cosines and sines of a row (row >= 0), from this lane's first pair on.
template <int V>
struct Row {
  typedef float vec __attribute__((ext_vector_type(V), aligned(4)));
  vec c, s;
};
template <int V>
__device__ __forceinline__ Row<V> load_table(const HeadsArgs& a, int64_t row, const Lane& l) {
  typedef typename Row<V>::vec vec;
  Row<V> t;
  const float* cp = a.cos + row * a.table_stride + l.slot;
  const float* sp = a.sin + row * a.table_stride + l.slot;
  if (l.part) {  // fewer than V pairs: the row may end before the vector
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = min(k, a.half - 1);
      t.c[k] = cp[i];
      t.s[k] = sp[i];
    }
  } else {
    t.c = *reinterpret_cast<const vec*>(cp);
    t.s = *reinterpret_cast<const vec*>(sp);
  }
  return t;
}
// The row of this lane's token: NaN outside the table, zeros for lanes that
// rotate nothing.
template <int V>
__device__ __forceinline__ Row<V> row_of(const HeadsArgs& a, bool wanted, uint32_t b, uint32_t s, const Lane& l) {
  Row<V> t;
  t.c = t.s = 0.0f;
  if (wanted) {
    const int64_t row = table_row(a, b, s);
    t.c = t.s = __builtin_nanf("");
    if (row >= 0) t = load_table<V>(a, row, l);
  }
  return t;
}

// Pair k of a lane's 2V elements: e[first(k)], e[second(k)].
template <int V, bool INTER>
__device__ __forceinline__ constexpr int first_of(int k) {
  return INTER ? 2 * k : k;
}
template <int V, bool INTER>
__device__ __forceinline__ constexpr int second_of(int k) {
  return INTER ? 2 * k + 1 : V + k;
}

// Stores a lane's 2V elements at the head's first element.
template <int BF16, int V>
__device__ __forceinline__ void store_lane(void* head, const Lane& l, const float* e) {
  constexpr int kSize = BF16 ? 2 : 4;
  char* p = static_cast<char*>(head);
  const Raw<BF16, V> lo = narrow<BF16, V>(e), hi = narrow<BF16, V>(e + V);
  if (!l.part) {
    lo.store(p + l.oa * kSize);
    hi.store(p + l.ob * kSize);
    return;
  }
#pragma unroll
  for (int k = 0; k < 2 * V; ++k) {
    if (!((l.counted >> k) & 1u)) continue;
    const uint32_t w = k < V ? lo.bits(k) : hi.bits(k - V);
    char* q = p + (k < V ? l.oa + k : l.ob + k - V) * kSize;
    if constexpr (BF16)
      *reinterpret_cast<uint16_t*>(q) = (uint16_t)w;
    else
      *reinterpret_cast<uint32_t*>(q) = w;
  }
}

// The sum over a head of terms t[0..2V) of each lane: pairs, the lane's
// pairs, lanes.  Uncounted terms are +0.
template <int V, bool INTER>
__device__ __forceinline__ float head_sum(float* t, const Lane& l, bool ragged, int log_group) {
  if (ragged) {
#pragma unroll
    for (int k = 0; k < 2 * V; ++k) t[k] = (l.counted >> k) & 1u ? t[k] : 0.0f;
  }
  float p[V];
#pragma unroll
  for (int k = 0; k < V; ++k) p[k] = add_c(t[first_of<V, INTER>(k)], t[second_of<V, INTER>(k)]);
  return group_sum(tree<V>(p), log_group);
}

struct Item {
  uint32_t b, s, first_head;
  int heads;
};

__device__ __forceinline__ Item item_of(const HeadsArgs& a, const HeadSide& side, uint32_t i, int per) {
  Item it;
  const uint32_t chunk = i / a.tokens;
  const uint32_t t = i - chunk * a.tokens;
  it.b = t / a.seq;
  it.s = t - it.b * a.seq;
  it.first_head = chunk * per;
  it.heads = min(per, side.heads - (int)it.first_head);
  return it;
}

template <int BF16>
__device__ __forceinline__ int64_t head_at(const int64_t* stride, const Item& it) {
  return (BF16 ? 2 : 4) *
         (it.b * stride[0] + it.s * stride[1] + (int64_t)it.first_head * stride[2]);
}

template <int BF16, int V, bool INTER, int HEADS>
__global__ __launch_bounds__(kThreads) void k_heads(HeadsArgs a) {
  constexpr int kSize = BF16 ? 2 : 4;
  const bool keys = blockIdx.x >= a.side[0].blocks;
  const HeadSide& side = a.side[keys];
  const uint32_t block = blockIdx.x - (keys ? a.side[0].blocks : 0);
  const uint32_t group = (block * (uint32_t)kThreads + threadIdx.x) >> a.log_group;
  const Lane l = lane_of<V, INTER>(a, threadIdx.x & ((1 << a.log_group) - 1));
  const bool live = group < side.items;
  const Item it = item_of(a, side, live ? group : 0, HEADS);
  const char* x = static_cast<const char*>(side.x) + head_at<BF16>(side.x_stride, it);
  char* out = static_cast<char*>(side.out) + head_at<BF16>(side.out_stride, it);
  const bool on = live && l.active;

  Raw<BF16, V> lo[HEADS], hi[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    lo[h] = {};
    hi[h] = {};
    if (on && h < it.heads) {
      const char* p = x + h * side.x_stride[2] * kSize;
      lo[h].load(p + l.oa * kSize);
      hi[h].load(p + l.ob * kSize);
    }
  }
  const Row<V> row = row_of<V>(a, on && l.rotated, it.b, it.s, l);
  float g[2 * V];
  const bool has_gain = side.gain != nullptr;
  if (on && has_gain) load_gain<V>(side.gain, a.gain_bf16, l, g, g + V);

#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    float e[2 * V], t[2 * V];
    widen(lo[h], e);
    widen(hi[h], e + V);
#pragma unroll
    for (int k = 0; k < 2 * V; ++k) t[k] = mul_c(e[k], e[k]);
    const float S = head_sum<V, INTER>(t, l, a.ragged, a.log_group);
    const float r = div_c(1.0f, sqrt_c(add_c(mul_c(S, a.inv_dim), a.eps)));
    if (!on || h >= it.heads) continue;
#pragma unroll
    for (int k = 0; k < 2 * V; ++k) e[k] = mul_c(e[k], r);
    if (has_gain) {
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) e[k] = mul_c(e[k], g[k]);
    }
    if (l.rotated) {
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
    store_lane<BF16, V>(out + h * side.out_stride[2] * kSize, l, e);
  }
}

// The backward pass.  GAIN: some side has a gain, whose gradient's row of
// this workgroup goes to side.partial[block].
template <int BF16, int V, bool INTER, int HEADS, bool GAIN>
__global__ __launch_bounds__(kThreads) void k_heads_grad(HeadsArgs a) {
  constexpr int kSize = BF16 ? 2 : 4;
  const bool keys = blockIdx.x >= a.side[0].blocks;
  const HeadSide& side = a.side[keys];
  const uint32_t block = blockIdx.x - (keys ? a.side[0].blocks : 0);
  const int j = threadIdx.x & ((1 << a.log_group) - 1);
  const Lane l = lane_of<V, INTER>(a, j);
  const bool has_gain = GAIN && side.gain != nullptr;
  float g[GAIN ? 2 * V : 1], acc[GAIN ? 2 * V : 1];
  if constexpr (GAIN) {
#pragma unroll
    for (int k = 0; k < 2 * V; ++k) acc[k] = 0.0f;
    if (l.active && has_gain) load_gain<V>(side.gain, a.gain_bf16, l, g, g + V);
  }
  const uint32_t groups = side.blocks * (uint32_t)(kThreads >> a.log_group);
  const uint32_t mine = (block * (uint32_t)kThreads + threadIdx.x) >> a.log_group;
  // The trip count is the workgroup's first group's, so whole waves stay
  // together in the exchanges.
  const uint32_t lead = block * (uint32_t)(kThreads >> a.log_group);
  for (uint32_t step = 0; lead + (uint64_t)step * groups < side.items; ++step) {
    const uint64_t i = mine + (uint64_t)step * groups;
    const bool live = i < side.items;
    const bool on = live && l.active;
    const Item it = item_of(a, side, live ? (uint32_t)i : 0, HEADS);
    const char* x = static_cast<const char*>(side.x) + head_at<BF16>(side.x_stride, it);
    const char* dy = static_cast<const char*>(side.dy) + head_at<BF16>(side.dy_stride, it);
    char* out = static_cast<char*>(side.out) + head_at<BF16>(side.out_stride, it);
    Raw<BF16, V> xlo[HEADS], xhi[HEADS], ylo[HEADS], yhi[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      xlo[h] = {};
      xhi[h] = {};
      ylo[h] = {};
      yhi[h] = {};
      if (on && h < it.heads) {
        const char* p = x + h * side.x_stride[2] * kSize;
        const char* q = dy + h * side.dy_stride[2] * kSize;
        xlo[h].load(p + l.oa * kSize);
        xhi[h].load(p + l.ob * kSize);
        ylo[h].load(q + l.oa * kSize);
        yhi[h].load(q + l.ob * kSize);
      }
    }
    const Row<V> row = row_of<V>(a, on && l.rotated, it.b, it.s, l);
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      float e[2 * V], d[2 * V], t[2 * V];
      widen(xlo[h], e);
      widen(xhi[h], e + V);
      widen(ylo[h], d);
      widen(yhi[h], d + V);
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) t[k] = mul_c(e[k], e[k]);
      const float S = head_sum<V, INTER>(t, l, a.ragged, a.log_group);
      const float r = div_c(1.0f, sqrt_c(add_c(mul_c(S, a.inv_dim), a.eps)));
      if (on && l.rotated) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          float& da = d[first_of<V, INTER>(k)];
          float& db = d[second_of<V, INTER>(k)];
          const float za = add_c(mul_c(da, row.c[k]), mul_c(db, row.s[k]));
          const float zb = sub_c(mul_c(db, row.c[k]), mul_c(da, row.s[k]));
          da = za;
          db = zb;
        }
      }
      // d is dz, then dn; t = dn * x.
      float n[2 * V];
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) n[k] = mul_c(e[k], r);
      if constexpr (GAIN) {
        if (has_gain) {
          const bool counts = on && h < it.heads;
#pragma unroll
          for (int k = 0; k < 2 * V; ++k) {
            const float term = mul_c(d[k], n[k]);
            acc[k] = add_c(acc[k], counts ? term : 0.0f);
            d[k] = mul_c(d[k], g[k]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) t[k] = mul_c(d[k], e[k]);
      const float T = head_sum<V, INTER>(t, l, a.ragged, a.log_group);
      const float w = mul_c(mul_c(T, r), a.inv_dim);
      if (!on || h >= it.heads) continue;
#pragma unroll
      for (int k = 0; k < 2 * V; ++k) d[k] = mul_c(sub_c(d[k], mul_c(n[k], w)), r);
      store_lane<BF16, V>(out + h * side.out_stride[2] * kSize, l, d);
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
      if (a.log_group < 1) v = add_c(v, __shfl_xor(v, 1, 64));
      if (a.log_group < 2) v = add_c(v, __shfl_xor(v, 2, 64));
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
        if ((l.counted >> k) & 1u) row[k < V ? l.oa + k : l.ob + k - V] = v;
      }
    }
  }
}

// dgain[i] = the sum of a side's rows: 16 columns of a workgroup, each with
// 16 threads that take every sixteenth row in ascending order, then a tree.
constexpr int kFoldColumns = 16;
__global__ __launch_bounds__(256) void k_gain_fold(HeadsArgs a) {
  const HeadSide& side = a.side[blockIdx.y];
  if (side.gain == nullptr) return;
  const int column = threadIdx.x % kFoldColumns, part = threadIdx.x / kFoldColumns;
  const int i = blockIdx.x * kFoldColumns + column;
  float v = 0.0f;
  if (i < a.dim) {
    const float* p = side.partial + i;
#pragma unroll 8
    for (uint32_t row = part; row < side.blocks; row += 16) v = add_c(v, p[(int64_t)row * a.dim]);
  }
  __shared__ float sums[16][kFoldColumns];
  sums[part][column] = v;
  __syncthreads();
  if (part == 0 && i < a.dim) {
    float t[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) t[k] = sums[k][column];
    side.dgain[i] = tree<16>(t);
  }
}

constexpr int kForwardHeads = 4;
constexpr int kBackwardHeads = 2;
// Rows of a gain's gradient: enough workgroups to fill the chip several
// times, few enough that the second kernel is short.
constexpr uint32_t kMaxGainBlocks = 2048;

int vector_of(int dtype, int dim) { return dim < 16 ? 1 : 8; }

template <int BF16, int V>
hipError_t run(const HeadsArgs& a, bool inter, bool backward, bool gain, hipStream_t stream) {
  const dim3 grid(a.side[0].blocks + a.side[1].blocks), block(kThreads);
  if (grid.x == 0) return hipSuccess;
  if (!backward) {
    if (inter)
      hipLaunchKernelGGL((k_heads<BF16, V, true, kForwardHeads>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((k_heads<BF16, V, false, kForwardHeads>), grid, block, 0, stream, a);
  } else if (gain) {
    if (inter)
      hipLaunchKernelGGL((k_heads_grad<BF16, V, true, kBackwardHeads, true>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((k_heads_grad<BF16, V, false, kBackwardHeads, true>), grid, block, 0, stream, a);
  } else {
    if (inter)
      hipLaunchKernelGGL((k_heads_grad<BF16, V, true, kBackwardHeads, false>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((k_heads_grad<BF16, V, false, kBackwardHeads, false>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace

bool plan_heads(HeadsArgs* a, int dtype, bool backward) {
  const int V = vector_of(dtype, a->dim);
  const int passing = a->dim / 2 - a->half;
  a->rot_lanes = (a->half + V - 1) / V;
  a->lanes = a->rot_lanes + (passing + V - 1) / V;
  a->ragged = a->half % V != 0 || passing % V != 0;
  a->log_group = 0;
  while ((1 << a->log_group) < a->lanes) ++a->log_group;
  const int per = backward ? kBackwardHeads : kForwardHeads;
  const uint32_t groups = kThreads >> a->log_group;
  for (HeadSide& side : a->side) {
    const int64_t chunks = (side.heads + per - 1) / per;
    const int64_t items = chunks * a->tokens;
    if (items > 0x7fffffff) return false;
    side.items = (uint32_t)items;
    int64_t blocks = (items + groups - 1) / groups;
    if (backward && side.gain != nullptr && blocks > kMaxGainBlocks) blocks = kMaxGainBlocks;
    side.blocks = (uint32_t)blocks;
  }
  // A launch holds fewer than 2^32 threads.
  return ((int64_t)a->side[0].blocks + a->side[1].blocks) * kThreads <= 0xffffffffLL;
}

hipError_t launch_heads(const HeadsArgs& a, int dtype, bool inter, bool backward, hipStream_t stream) {
  const bool gain = a.side[0].gain != nullptr || a.side[1].gain != nullptr;
  const bool small = vector_of(dtype, a.dim) == 1;
  hipError_t e;
  if (dtype == REPRO_BF16)
    e = small ? run<1, 1>(a, inter, backward, gain, stream) : run<1, 8>(a, inter, backward, gain, stream);
  else
    e = small ? run<0, 1>(a, inter, backward, gain, stream) : run<0, 8>(a, inter, backward, gain, stream);
  if (e != hipSuccess || !backward || !gain) return e;
  hipLaunchKernelGGL(k_gain_fold, dim3((a.dim + kFoldColumns - 1) / kFoldColumns, 2), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace repro
