// Device helpers shared by the head kernels (heads.hip, heads_grad.hip): the
// lanes of a head, its loads and stores, and the sums over it.
//
// A group of lanes, a power of two from four up, holds one head: a lane has V
// pairs in two vectors of V elements, lo and hi, of one section of the head,
// the rotated one (h pairs) or the one that passes (D/2 - h).  Without
// interleaving pair i of a section is its elements i and i + its pairs, lo and
// hi are vectors of its halves, so that a rotated pair meets in one lane and
// no element crosses lanes; interleaved they are 2V neighbours.  A section
// whose pair count V does not divide ends in a lane whose vectors are moved
// back to the section's end: the pairs it shares with its neighbour are left
// out of its sums, and both lanes store the same bits to them.  A section of
// fewer than V pairs is one lane that stores element by element.
#pragma once

#include <hip/hip_runtime.h>

#include "device_ops.h"
#include "internal.h"

namespace repro {
namespace {

constexpr int kThreads = 256;

// What the sizes leave for a kernel to handle: kWhole, every lane rotates
// whole vectors; kMixed, some lanes pass theirs; kRagged, V does not divide
// every section.
enum Mode { kWhole, kMixed, kRagged };

// Vectors of V elements at any element's alignment (gfx950 loads and stores
// 4, 8 and 16 bytes at any address).
template <int BF16, int V>
struct Raw;
typedef uint32_t u4_2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u4_4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2_2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

// STREAM: the access bypasses cache retention.
template <bool STREAM, typename R, typename A>
__device__ __forceinline__ R load_as(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const A*>(p));
  return *static_cast<const A*>(p);
}
template <bool STREAM, typename R, typename A>
__device__ __forceinline__ void store_as(R w, void* p) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(w, static_cast<A*>(p));
  else
    *static_cast<A*>(p) = w;
}

template <>
struct Raw<1, 8> {
  u4 w;
  template <bool STREAM>
  __device__ void load(const void* p) { w = load_as<STREAM, u4, u4_2>(p); }
  template <bool STREAM>
  __device__ void store(void* p) const { store_as<STREAM, u4, u4_2>(w, p); }
  __device__ uint32_t bits(int i) const { return w[i >> 1] >> (16 * (i & 1)); }
};
template <>
struct Raw<1, 4> {
  u2 w;
  template <bool STREAM>
  __device__ void load(const void* p) { w = load_as<STREAM, u2, u2_2>(p); }
  template <bool STREAM>
  __device__ void store(void* p) const { store_as<STREAM, u2, u2_2>(w, p); }
  __device__ uint32_t bits(int i) const { return w[i >> 1] >> (16 * (i & 1)); }
};
template <>
struct Raw<1, 1> {
  uint16_t w;
  template <bool STREAM>
  __device__ void load(const void* p) { w = *static_cast<const uint16_t*>(p); }
  template <bool STREAM>
  __device__ void store(void* p) const { *static_cast<uint16_t*>(p) = w; }
  __device__ uint32_t bits(int) const { return w; }
};
template <>
struct Raw<0, 8> {
  u4 w[2];
  template <bool STREAM>
  __device__ void load(const void* p) {
    w[0] = load_as<STREAM, u4, u4_4>(p);
    w[1] = load_as<STREAM, u4, u4_4>(static_cast<const u4_4*>(p) + 1);
  }
  template <bool STREAM>
  __device__ void store(void* p) const {
    store_as<STREAM, u4, u4_4>(w[0], p);
    store_as<STREAM, u4, u4_4>(w[1], static_cast<u4_4*>(p) + 1);
  }
  __device__ uint32_t bits(int i) const { return w[i >> 2][i & 3]; }
};
template <>
struct Raw<0, 4> {
  u4 w;
  template <bool STREAM>
  __device__ void load(const void* p) { w = load_as<STREAM, u4, u4_4>(p); }
  template <bool STREAM>
  __device__ void store(void* p) const { store_as<STREAM, u4, u4_4>(w, p); }
  __device__ uint32_t bits(int i) const { return w[i]; }
};
template <>
struct Raw<0, 1> {
  uint32_t w;
  template <bool STREAM>
  __device__ void load(const void* p) { w = *static_cast<const uint32_t*>(p); }
  template <bool STREAM>
  __device__ void store(void* p) const { *static_cast<uint32_t*>(p) = w; }
  __device__ uint32_t bits(int) const { return w; }
};

// Makes the compiler widen the vector anew where it is used next, instead of
// holding the wide elements (twice its registers) until then.
template <int BF16, int V>
__device__ __forceinline__ void forget(Raw<BF16, V>& r) {
  constexpr int kWords = sizeof(r) / 4;
  if constexpr (kWords > 0) {
    uint32_t w[kWords];
    __builtin_memcpy(w, &r, sizeof(r));
#pragma unroll
    for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
    __builtin_memcpy(&r, w, sizeof(r));
  }
}

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
  if constexpr (BF16 && V > 1) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.w[i] = round2(x[2 * i], x[2 * i + 1]);
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


// The two sides of a branch on whether to stream differ in nothing else: this
// keeps the compiler from making one access of both, without the hint.
__device__ __forceinline__ void keep_apart() { asm volatile(""); }

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
// Perfect tree over the 2^log_group >= 4 lanes of a group (uniform branches).
__device__ __forceinline__ float group_sum(float v, int log_group) {
  v = add_c(v, dpp<0xB1>(v));                      // lanes 1,0,3,2 of each four
  v = add_c(v, dpp<0x4E>(v));                      // lanes 2,3,0,1 of each four
  if (log_group > 2) v = add_c(v, dpp<0x141>(v));  // mirrored in each eight
  if (log_group > 3) v = add_c(v, dpp<0x140>(v));  // mirrored in each sixteen
  if (log_group > 4) v = level16(v);
  if (log_group > 5) v = level32(v);
  return v;
}

template <int N>
__device__ __forceinline__ float tree(const float* t) {
  float u[N];
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = t[i];
#pragma unroll
  for (int n = N; n > 1; n >>= 1)
#pragma unroll
    for (int i = 0; i < n / 2; ++i) u[i] = add_c(u[2 * i], u[2 * i + 1]);
  return u[0];
}

// What one lane of a group holds.  Element k < V of a lane is lo[k], at
// oa + k; element V + k is hi[k], at ob + k.
struct Lane {
  int oa, ob;
  uint32_t counted;  // bit k: pair k is this lane's in the sums
  int slot;          // first rotated pair (rotated lanes)
  bool active, rotated, part;  // part: only the counted pairs are stored
};

template <int V, bool INTER, int MODE>
__device__ __forceinline__ Lane lane_of(const HeadsArgs& a, int j) {
  constexpr uint32_t kAll = (1u << V) - 1u;
  const int half = a.half, pairs = a.dim / 2 - half;  // rotated and passing pairs
  Lane l;
  l.active = j < a.lanes;
  l.rotated = MODE == kWhole ? l.active : j < a.rot_lanes;
  const bool turned = MODE == kWhole || l.rotated;
  const int begin = turned ? 0 : 2 * half;                 // of the section, in elements
  const int count = turned ? half : pairs;                 // its pairs
  const int want = (turned ? j : j - a.rot_lanes) * V;     // its pairs before this lane's
  int first = want;
  l.counted = kAll;
  l.part = false;
  if constexpr (MODE == kRagged) {
    first = min(want, count - V);  // moved back
    l.part = count < V;
    if (l.rotated) {
      // Too few pairs: the vectors reach past the section, not before it.
      first = max(first, 0);
      if (l.part) l.counted = (1u << count) - 1u;
    }
    l.counted = l.active ? l.counted & ~((1u << (want - first)) - 1u) : 0u;
  }
  l.slot = first;
  l.oa = begin + (INTER ? 2 * first : first);
  l.ob = l.oa + (INTER ? V : count);
  return l;
}

// A lane's elements of a gain (the same places as the head's).
template <int V>
__device__ __forceinline__ void load_gain(const void* gain, int is_bf16, const Lane& l, float* g) {
  if (is_bf16) {
    Raw<1, V> lo, hi;
    lo.template load<false>(static_cast<const uint16_t*>(gain) + l.oa);
    hi.template load<false>(static_cast<const uint16_t*>(gain) + l.ob);
    widen(lo, g);
    widen(hi, g + V);
  } else {
    Raw<0, V> lo, hi;
    lo.template load<false>(static_cast<const float*>(gain) + l.oa);
    hi.template load<false>(static_cast<const float*>(gain) + l.ob);
    widen(lo, g);
    widen(hi, g + V);
  }
}

// V cosines and sines of a row of the table, from a lane's first pair on.
template <int V>
struct Row {
  typedef float vec __attribute__((ext_vector_type(V), aligned(4)));
  vec c, s;
};

// The row of (batch b, token s) in the table: NaN outside it, zeros for lanes
// that rotate nothing.
template <int V>
__device__ __forceinline__ Row<V> row_of(const HeadsArgs& a, bool wanted, uint32_t b, uint32_t s, const Lane& l) {
  typedef typename Row<V>::vec vec;
  Row<V> t;
  t.c = t.s = 0.0f;
  if (!wanted) return t;
  int64_t p = s;
  if (a.positions != nullptr) {
    const int64_t at = b * a.pos_stride[0] + s * a.pos_stride[1];
    p = a.pos64 ? static_cast<const int64_t*>(a.positions)[at] : static_cast<const int32_t*>(a.positions)[at];
  }
  if (p < 0 || p >= a.table_rows) {
    t.c = t.s = __builtin_nanf("");
    return t;
  }
  const float* cp = a.cos + p * a.table_stride + l.slot;
  const float* sp = a.sin + p * a.table_stride + l.slot;
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

// Pair k of a lane's 2V elements: e[first_of(k)], e[second_of(k)].
template <int V, bool INTER>
__device__ __forceinline__ constexpr int first_of(int k) {
  return INTER ? 2 * k : k;
}
template <int V, bool INTER>
__device__ __forceinline__ constexpr int second_of(int k) {
  return INTER ? 2 * k + 1 : V + k;
}

template <int V, bool INTER>
__device__ __forceinline__ constexpr int pair_of(int element) {
  return INTER ? element / 2 : element % V;
}

// Stores a lane's 2V elements at the head's first element.
template <int BF16, int V, bool INTER, int MODE>
__device__ __forceinline__ void store_lane(void* head, const Lane& l, const float* e, bool stream) {
  constexpr int kSize = BF16 ? 2 : 4;
  char* p = static_cast<char*>(head);
  const Raw<BF16, V> lo = narrow<BF16, V>(e), hi = narrow<BF16, V>(e + V);
  if (MODE == kRagged && l.part) {
#pragma unroll
    for (int k = 0; k < 2 * V; ++k) {
      if (!((l.counted >> pair_of<V, INTER>(k)) & 1u)) continue;
      const uint32_t w = k < V ? lo.bits(k) : hi.bits(k - V);
      char* q = p + (k < V ? l.oa + k : l.ob + k - V) * kSize;
      if constexpr (BF16)
        *reinterpret_cast<uint16_t*>(q) = (uint16_t)w;
      else
        *reinterpret_cast<uint32_t*>(q) = w;
    }
  } else if (stream) {
    keep_apart();
    lo.template store<true>(p + l.oa * kSize);
    hi.template store<true>(p + l.ob * kSize);
    keep_apart();
  } else {
    lo.template store<false>(p + l.oa * kSize);
    hi.template store<false>(p + l.ob * kSize);
  }
}

// The sum over a head of the terms t[0..2V) of each lane: pairs, the lane's
// pairs, lanes.  Uncounted pairs are +0, and lanes past the head hold zeros.
template <int V, bool INTER, int MODE>
__device__ __forceinline__ float head_sum(const float* t, const Lane& l, int log_group) {
  float p[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    p[k] = add_c(t[first_of<V, INTER>(k)], t[second_of<V, INTER>(k)]);
    if (MODE == kRagged) p[k] = (l.counted >> k) & 1u ? p[k] : 0.0f;
  }
  return group_sum(tree<V>(p), log_group);
}

// r[h] = 1 / sqrt(S[h] / D + eps) of HEADS (a power of two up to 4) heads.
// The correctly rounded root and quotient are some 40 instructions, and all
// lanes of a group hold the same sums: lane h of each four takes head h's,
// and the four read each other's result.
template <int HEADS>
__device__ __forceinline__ void roots(const HeadsArgs& a, const float* S, float* r) {
  float d[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h) d[h] = add_c(mul_c(S[h], a.inv_dim), a.eps);
  float mine = d[0];
  if constexpr (HEADS == 4) {
    const float low = threadIdx.x & 1 ? d[1] : d[0], high = threadIdx.x & 1 ? d[3] : d[2];
    mine = threadIdx.x & 2 ? high : low;
  } else if constexpr (HEADS == 2) {
    mine = threadIdx.x & 1 ? d[1] : d[0];
  }
  const float root = div_c(1.0f, sqrt_c(mine));
  if constexpr (HEADS == 4) {
    r[0] = dpp<0x00>(root);
    r[1] = dpp<0x55>(root);
    r[2] = dpp<0xAA>(root);
    r[3] = dpp<0xFF>(root);
  } else if constexpr (HEADS == 2) {
    r[0] = dpp<0xA0>(root);  // lanes 0,0,2,2
    r[1] = dpp<0xF5>(root);  // lanes 1,1,3,3
  } else {
    r[0] = root;
  }
}

// A group's work: heads first_head, first_head + chunks, ... of one token,
// `heads` of them.  So the groups beside each other in a wave have neighbouring
// heads at every step, and their stores fill whole cache lines also where a
// head does not: with neighbouring heads in one group, nontemporal stores of
// 80-byte heads ran at half the rate.
struct Item {
  uint32_t b, s, first_head;
  int heads;
};

// i / d for i < 2^31 by a product (FastDiv, filled on the host).
__device__ __forceinline__ uint32_t quotient(uint32_t i, const FastDiv& d) {
  return d.divisor == 1 ? i : __umulhi(i, d.factor) >> d.shift;
}

// Item i: chunks of one token side by side, so that a wave's groups share the
// table's rows.
template <int HEADS>
__device__ __forceinline__ Item item_of(const HeadsArgs& a, const HeadSide& side, uint32_t i) {
  const uint32_t t = quotient(i, side.by_chunks);
  Item it;
  it.b = quotient(t, a.by_seq);
  it.s = t - it.b * a.by_seq.divisor;
  it.first_head = i - t * side.by_chunks.divisor;
  it.heads = 0;
#pragma unroll
  for (int h = 0; h < HEADS; ++h) it.heads += it.first_head + h * side.by_chunks.divisor < (uint32_t)side.heads;
  return it;
}

// The byte offset of an item's first head.
template <int BF16>
__device__ __forceinline__ int64_t head_at(const int64_t* stride, const Item& it) {
  return (BF16 ? 2 : 4) * (it.b * stride[0] + it.s * stride[1] + (int64_t)it.first_head * stride[2]);
}

}  // namespace
}  // namespace repro
