// The global l2 norm of a list of gradient tensors, and their clipping.
//
// "OPEN-1B: A Fully Auditable Training Run", section 3.2 "Optimizer"
// (gradients clipped to a global l2 norm) and Appendix A.1 (TreeFold, the
// order of every sum here).
//
// Mathematics.  S_t = TreeFold(g_0^2, g_1^2, ...) of each tensor in index
// order; S = TreeFold(S_0, S_1, ...); norm = sqrt(S); every element is then
// multiplied by coef = min(1, max_norm / (norm + 1e-6)).  For terms >= +0 a
// TreeFold equals one perfect pairwise tree over the terms padded with +0 to
// a power of two, so any aligned power-of-two tile of it can be summed alone.
//
// Design for gfx950 (memory bound; the norm has to be whole before the first
// output leaves, so the gradients are read twice and written once):
//  - The list is laid out once: a table of tiles, each 64 KB (or 16 KB in a
//    small list) of one tensor with its addresses, so that one launch covers
//    every tensor and a workgroup finds its work with one scalar load.
//  - A wave takes a quarter of a tile in 1 KB loads, all in flight at once,
//    16 bytes a lane at whatever alignment the tensor starts.  A lane's terms
//    fold in the lane; the chunks' lane sums then fold together: at each of
//    the first levels two chunks share one exchange (a lane keeps one chunk's
//    sum and hands over the other's), so 16 chunks need 21 exchanges in place
//    of 96, and the order of the additions is still the tree's.
//  - Tensors' sums: one workgroup for each tensor; not launched when every
//    tensor is one tile, nor for small lists of up to 512 tiles, whose last
//    kernel folds the tiles in LDS.
//  - Large lists (64 MB and more, past the caches) move with nontemporal
//    accesses, and are scaled by one wave for each 1 KB with the coefficient
//    in memory, the shape in which a plain copy runs fastest here.  Small
//    lists stay in the caches between the passes; there each workgroup of the
//    scaling kernel issues its loads and folds the sums itself while they
//    travel, which saves a launch.
//
// Measured on MI355X (whole calls, us).  1.61e9 parameters in BF16 (219
// tensors): 1430, of which squares 475 (6.8 TB/s) and scaling 950 (6.8 TB/s,
// a plain copy's rate); with the small lists' kernels 1735, with all 16
// chunks in flight and nontemporal accesses 1600, scaling 4 KB a wave 1529.
// Walking back from the last tile or keeping the last 128 MB cached gained
// nothing.  The two forms at 52 MB: 31.5 small, 35.9 large; at 105 MB: 67.2
// small, 62.4 large.  49 tensors of 2048: 9.1, the two launches alone 8.5.
#include <hip/hip_runtime.h>

#include "device_ops.h"
#include "internal.h"

namespace repro {
namespace {

constexpr int64_t kMagic = 0x7265706c69737431;
constexpr int64_t kMaxTiles = (int64_t(1) << 24) - 1;  // 256 threads each, below 2^32 in all
constexpr int64_t kLargeList = int64_t(64) << 20;  // bytes from which tiles are 64 KB; both sides measured above
constexpr int kWaveFold = 1024;                    // most sums that a wave folds by itself
constexpr int kNested = 512;                       // most tiles that the last kernel folds (nested() below)

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4_2 __attribute__((ext_vector_type(4), aligned(2)));  // any element's alignment

// A tile's addresses come from memory, so the compiler cannot see that they
// are global; said here, or every access would also wait on LDS.
template <typename T>
using Global = __attribute__((address_space(1))) T;
template <typename T>
__device__ __forceinline__ Global<T>* global(const void* p) {
  return (Global<T>*)(uintptr_t)p;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}

// The value of lane ^ (1 << LEVEL), inside a row of sixteen lanes.
template <int LEVEL>
__device__ __forceinline__ float across(float v) {
  static_assert(LEVEL >= 0 && LEVEL < 4, "levels between rows: add_level4, add_level5");
  if constexpr (LEVEL == 0) return dpp<0xB1>(v);
  if constexpr (LEVEL == 1) return dpp<0x4E>(v);
  if constexpr (LEVEL == 2) {
    // Fours 0 and 2 of a row take the lane four above, fours 1 and 3 below.
    const int x = __float_as_int(v);
    const int up = __builtin_amdgcn_update_dpp(0, x, 0x104, 0xf, 0x5, false);
    return __int_as_float(__builtin_amdgcn_update_dpp(up, x, 0x114, 0xf, 0xA, false));
  }
  if constexpr (LEVEL == 3) return dpp<0x128>(v);
}
// v plus the value across, for the two levels between rows.
__device__ __forceinline__ float add_level4(float v) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return add_c(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float add_level5(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return add_c(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// One level at which two chunks share an exchange: a lane with bit LEVEL
// clear keeps the even chunk, one with it set the odd chunk.
template <int LEVEL, int N>
__device__ __forceinline__ void pair_level(float* v, int lane) {
  const bool odd = (lane >> LEVEL) & 1;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float keep = odd ? v[2 * i + 1] : v[2 * i];
    const float give = odd ? v[2 * i] : v[2 * i + 1];
    v[i] = add_c(keep, across<LEVEL>(give));
  }
}

// The perfect tree over C chunks of 64 lane sums each, lanes first; every
// lane returns it.
template <int C>
__device__ __forceinline__ float fold_chunks(float* v, int lane) {
  static_assert(C == 16 || C == 4 || C == 1, "chunks of a wave");
  float s;
  if constexpr (C == 16) {
    pair_level<0, 16>(v, lane);
    pair_level<1, 8>(v, lane);
    pair_level<2, 4>(v, lane);
    pair_level<3, 2>(v, lane);
    s = v[0];
  } else if constexpr (C == 4) {
    pair_level<0, 4>(v, lane);
    pair_level<1, 2>(v, lane);
    s = v[0];
    s = add_c(s, across<2>(s));
    s = add_c(s, across<3>(s));
  } else {
    s = v[0];
    s = add_c(s, across<0>(s));
    s = add_c(s, across<1>(s));
    s = add_c(s, across<2>(s));
    s = add_c(s, across<3>(s));
  }
  s = add_level4(s);
  s = add_level5(s);
  // Now lane & (C - 1) is the chunk.
  if constexpr (C >= 4) {
    s = add_c(s, across<0>(s));
    s = add_c(s, across<1>(s));
  }
  if constexpr (C >= 16) {
    s = add_c(s, across<2>(s));
    s = add_c(s, across<3>(s));
  }
  return s;
}

__device__ __forceinline__ float square(float x) { return mul_c(x, x); }
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The fold of the squares in one 16-byte load.
template <int BF16>
__device__ __forceinline__ float fold_load(u4 w) {
  if constexpr (BF16) {
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = add_c(square(low(w[i])), square(high(w[i])));
    return add_c(add_c(p[0], p[1]), add_c(p[2], p[3]));
  } else {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = square(__uint_as_float(w[i]));
    return add_c(add_c(q[0], q[1]), add_c(q[2], q[3]));
  }
}

// STREAM: the access bypasses cache retention.
template <bool STREAM>
__device__ __forceinline__ u4 load16(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(global<const u4_2>(p));
  return *global<const u4_2>(p);
}
template <bool STREAM>
__device__ __forceinline__ void store16(u4 w, void* p) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(w, global<u4_2>(p));
  else
    *global<u4_2>(p) = w;
}

// A tile's loads of one lane: chunk c of the wave, at element
// first + c * 64 * kPer of the tile.
template <int BF16>
struct Layout {
  static constexpr int kSize = BF16 ? 2 : 4;
  static constexpr int kPer = 16 / kSize;
};

template <int BF16, int C>
__device__ __forceinline__ int first_of(int wave, int lane) {
  return (wave * C * 64 + lane) * Layout<BF16>::kPer;
}

template <int BF16, int C, bool STREAM>
__device__ __forceinline__ void load_tile(const void* src, int n, int first, u4* w) {
  constexpr int kPer = Layout<BF16>::kPer;
  const char* p = static_cast<const char*>(src) + (int64_t)first * Layout<BF16>::kSize;
  if (n == 4 * C * 64 * kPer) {  // a whole tile (uniform)
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = load16<STREAM>(p + c * 1024);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      w[c] = u4{0, 0, 0, 0};
      if (first + c * 64 * kPer + kPer <= n) w[c] = *global<const u4_2>(p + c * 1024);
    }
  }
}

// The fold of the squares of a tile's part, by one wave.
template <int BF16, int C, bool STREAM>
__device__ __forceinline__ float wave_squares(const void* src, int n, int wave, int lane) {
  constexpr int kPer = Layout<BF16>::kPer;
  const int first = first_of<BF16, C>(wave, lane);
  u4 w[C];
  load_tile<BF16, C, STREAM>(src, n, first, w);
  float v[C];
#pragma unroll
  for (int c = 0; c < C; ++c) v[c] = fold_load<BF16>(w[c]);
  const int rest = n % kPer;
  if (rest != 0) {
    // The tensor's end lies inside one lane's load, of which nothing was
    // read: its terms, padded with +0, fold the same way.
    const int at = n - rest;
    const int c = (at - first) / (64 * kPer);
    if (at >= first && first + c * 64 * kPer == at && c < C) {
      float q[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        q[i] = 0.0f;
        if (i < rest) {
          if constexpr (BF16)
            q[i] = square(__uint_as_float((uint32_t)global<const uint16_t>(src)[at + i] << 16));
          else
            q[i] = square(global<const float>(src)[at + i]);
        }
      }
#pragma unroll
      for (int k = kPer; k > 1; k >>= 1)
#pragma unroll
        for (int i = 0; i < k / 2; ++i) q[i] = add_c(q[2 * i], q[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = i == c ? q[0] : v[i];
    }
  }
  return fold_chunks<C>(v, lane);
}

template <int C, bool STREAM>
__global__ __launch_bounds__(256) void k_list_squares(const ListTile* __restrict__ tiles, float* __restrict__ sums) {
  const ListTile tile = tiles[blockIdx.x];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const float s = tile.bf16 ? wave_squares<1, C, STREAM>(tile.src, tile.n, wave, lane)
                            : wave_squares<0, C, STREAM>(tile.src, tile.n, wave, lane);
  __shared__ float waves[4];
  if (lane == 0) waves[wave] = s;
  __syncthreads();
  if (threadIdx.x == 0) sums[blockIdx.x] = add_c(add_c(waves[0], waves[1]), add_c(waves[2], waves[3]));
}

// The perfect tree over at(0) .. at(count - 1), count <= 1024, by one wave:
// lane l holds 4l .. 4l+3 of each 256.  Every lane returns it.
template <typename At>
__device__ __forceinline__ float wave_fold_of(At at, int count, int lane) {
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c * 256 >= count) break;
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = c * 256 + 4 * lane + i;
      q[i] = k < count ? at(k) : 0.0f;
    }
    v[c] = add_c(add_c(q[0], q[1]), add_c(q[2], q[3]));
  }
  return count <= 256 ? fold_chunks<1>(v, lane) : fold_chunks<4>(v, lane);
}
__device__ __forceinline__ float wave_fold(const float* p, int count, int lane) {
  return wave_fold_of([p](int k) { return p[k]; }, count, lane);
}

// What the norm is folded from.
struct Sums {
  const float* values;   // the tensors' sums; NESTED: their tiles'
  const ListTile* tiles;
  const int64_t* first;  // of each tensor, among the tiles
  int count, tile_count, most;
};

// The fold over all tensors, by a workgroup of 256; every lane returns it.
// NESTED: the tensors' own trees first, level by level in LDS, for up to
// kNested tiles in all.
template <bool NESTED>
__device__ __forceinline__ float list_sum(const Sums& s) {
  const int lane = threadIdx.x & 63;
  if constexpr (!NESTED) return wave_fold(s.values, s.count, lane);
  constexpr int kPer = kNested / 256;
  __shared__ float v[kNested];
  int index[kPer], count[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int t = i * 256 + threadIdx.x;
    const bool in = t < s.tile_count;
    index[i] = in ? s.tiles[t].index : 0;
    count[i] = in ? s.tiles[t].count : 0;
    v[t] = in ? s.values[t] : 0.0f;
  }
  for (int n = 1; n < s.most; n <<= 1) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      // What is read here has an odd multiple of n as its index, and is not
      // written at this level.
      const int t = i * 256 + threadIdx.x;
      if ((index[i] & (2 * n - 1)) == 0 && index[i] + n < count[i]) v[t] = add_c(v[t], v[t + n]);
    }
  }
  __syncthreads();
  const float* p = v;
  const int64_t* first = s.first;
  return wave_fold_of([p, first](int k) { return p[first[k]]; }, s.count, lane);
}

// sums[t] = the perfect tree over values[first[t] .. first[t+1]), at most
// 2^24 of them, in blocks of 4096; first == nullptr: one tree over `count`.
__global__ __launch_bounds__(256) void k_list_fold(const float* __restrict__ values, const int64_t* __restrict__ first,
                                                   int64_t count, float* __restrict__ sums) {
  const int64_t begin = first != nullptr ? first[blockIdx.x] : 0;
  const int64_t len = first != nullptr ? first[blockIdx.x + 1] - begin : count;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int blocks = (int)((len + 4095) / 4096);
  __shared__ float block_sums[4096];
  __shared__ float waves[2][4];
  for (int b = 0; b < blocks; ++b) {
    const int64_t at = (int64_t)b * 4096 + wave * 1024;
    const int64_t left = len - at;
    const float s = wave_fold(values + begin + (left > 0 ? at : 0),  // a wave past the end adds +0
                              (int)(left < 0 ? 0 : (left < kWaveFold ? left : kWaveFold)), lane);
    if (lane == 0) waves[b & 1][wave] = s;
    __syncthreads();  // the other half of `waves` is free again after it
    if (threadIdx.x == 0) {
      const float* w = waves[b & 1];
      block_sums[b] = add_c(add_c(w[0], w[1]), add_c(w[2], w[3]));
    }
  }
  __syncthreads();
  if (blocks <= 1) {
    if (threadIdx.x == 0) sums[blockIdx.x] = blocks == 1 ? block_sums[0] : 0.0f;
    return;
  }
  const int left = blocks - wave * kWaveFold;
  const float s = wave_fold(block_sums + (left > 0 ? wave * kWaveFold : 0),
                            left < 0 ? 0 : (left < kWaveFold ? left : kWaveFold), lane);
  if (lane == 0) waves[0][wave] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    sums[blockIdx.x] = add_c(add_c(waves[0][0], waves[0][1]), add_c(waves[0][2], waves[0][3]));
}

// coef of a norm: max_norm / (norm + 1e-6) below 1, else 1; NaN for a NaN.
__device__ __forceinline__ float coef_of(float norm, float max_norm) {
  if (!(max_norm > 0.0f)) return 1.0f;
  const float c = div_c(max_norm, add_c(norm, 1e-6f));
  return c >= 1.0f ? 1.0f : c;
}

__device__ __forceinline__ void write3(float* out3, float norm, float S, float coef) {
  out3[0] = norm;
  out3[1] = S;
  out3[2] = coef;
}

template <bool NESTED>
__global__ __launch_bounds__(256) void k_list_finish(Sums sums, float max_norm, float* __restrict__ out3) {
  const float S = list_sum<NESTED>(sums);
  const float norm = sqrt_c(S);
  if (threadIdx.x == 0) write3(out3, norm, S, coef_of(norm, max_norm));
}

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef float fl2 __attribute__((ext_vector_type(2)));

template <int BF16>
__device__ __forceinline__ u4 scale_load(u4 w, float coef) {
  u4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16)  // to nearest, ties to even, once
      r[i] = __builtin_bit_cast(
          uint32_t, __builtin_convertvector((fl2{mul_c(low(w[i]), coef), mul_c(high(w[i]), coef)}), bf2));
    else
      r[i] = __float_as_uint(mul_c(__uint_as_float(w[i]), coef));
  }
  return r;
}

// Elements at .. n-1 of a tile, fewer than a 16-byte vector holds.
template <int BF16>
__device__ __forceinline__ void scale_rest(const ListTile& tile, int at, float coef, bool same) {
  for (int i = at; i < tile.n; ++i) {
    if constexpr (BF16) {
      const uint16_t h = global<const uint16_t>(tile.src)[i];
      global<uint16_t>(tile.dst)[i] = same ? h : (uint16_t)scale_load<1>(u4{h, 0, 0, 0}, coef)[0];
    } else {
      const uint32_t h = global<const uint32_t>(tile.src)[i];
      global<uint32_t>(tile.dst)[i] = same ? h : __float_as_uint(mul_c(__uint_as_float(h), coef));
    }
  }
}

// Small lists: a workgroup scales a tile, and folds the norm itself while its
// loads travel (in place they wait: an unclipped list then needs none).
template <int BF16, int C, bool NESTED>
__device__ __forceinline__ void scale_tile(const ListTile& tile, const Sums& sums, float max_norm, float* out3) {
  constexpr int kPer = Layout<BF16>::kPer, kSize = Layout<BF16>::kSize;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int first = first_of<BF16, C>(wave, lane);
  const bool in_place = tile.src == tile.dst;
  u4 w[C];
  if (!in_place) load_tile<BF16, C, false>(tile.src, tile.n, first, w);
  const float S = list_sum<NESTED>(sums);
  const float norm = sqrt_c(S);
  const float coef = coef_of(norm, max_norm);
  if (out3 != nullptr && threadIdx.x == 0) write3(out3, norm, S, coef);
  const bool same = coef == 1.0f;  // the bits are copied
  if (in_place) {
    if (same) return;
    load_tile<BF16, C, false>(tile.src, tile.n, first, w);
  }
  char* q = static_cast<char*>(tile.dst) + (int64_t)first * kSize;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = first + c * 64 * kPer;
    if (at + kPer <= tile.n)
      store16<false>(same ? w[c] : scale_load<BF16>(w[c], coef), q + c * 1024);
    else if (at < tile.n)
      scale_rest<BF16>(tile, at, coef, same);
  }
}

template <int C, bool NESTED>
__global__ __launch_bounds__(256) void k_list_scale(Sums sums, float max_norm, float* __restrict__ out3) {
  const ListTile tile = sums.tiles[blockIdx.x];
  float* const out = blockIdx.x == 0 ? out3 : nullptr;
  if (tile.bf16)
    scale_tile<1, C, NESTED>(tile, sums, max_norm, out);
  else
    scale_tile<0, C, NESTED>(tile, sums, max_norm, out);
}

// Large lists: one wave for each 1 KB, PARTS in a tile, one 16-byte vector a
// lane, past the caches; the coefficient is in memory already.
template <int BF16>
__device__ __forceinline__ void stream_vector(const ListTile& tile, int at, float coef) {
  constexpr int kPer = Layout<BF16>::kPer, kSize = Layout<BF16>::kSize;
  const bool same = coef == 1.0f;
  if (same && tile.src == tile.dst) return;
  if (at + kPer <= tile.n) {
    const u4 w = load16<true>(static_cast<const char*>(tile.src) + (int64_t)at * kSize);
    store16<true>(same ? w : scale_load<BF16>(w, coef), static_cast<char*>(tile.dst) + (int64_t)at * kSize);
  } else if (at < tile.n) {
    scale_rest<BF16>(tile, at, coef, same);
  }
}

template <int PARTS>
__global__ __launch_bounds__(64) void k_list_stream(const ListTile* __restrict__ tiles,
                                                    const float* __restrict__ out3) {
  const ListTile tile = tiles[blockIdx.x / PARTS];
  const int lane = (blockIdx.x % PARTS) * 64 + threadIdx.x;
  const float coef = out3[2];
  if (tile.bf16)
    stream_vector<1>(tile, lane * 8, coef);
  else
    stream_vector<0>(tile, lane * 4, coef);
}

int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }

int64_t tile_elements(int32_t dtype, int32_t chunks) { return 4096 * (int64_t)chunks / (dtype == REPRO_BF16 ? 2 : 4); }

// Whether the last kernel folds the tensors' tiles as well, in every
// workgroup, which saves a launch.  Measured, us a call with and without:
// 211 tiles 9.6 and 12.0, 533 tiles 11.0 and 12.0, 816 tiles 14.5 and 12.4.
bool nested(const ListHeader& h) { return h.chunks == 4 && h.most > 1 && h.tiles <= kNested; }

// The launches up to the sums that a workgroup can fold.
hipError_t launch_sums(const ListHeader& h, uint8_t* plan, Sums* out, hipStream_t stream) {
  const ListTile* tiles = reinterpret_cast<const ListTile*>(plan + sizeof(ListHeader));
  const int64_t* first = reinterpret_cast<const int64_t*>(plan + h.first_offset);
  float* block_sums = reinterpret_cast<float*>(plan + h.sums_offset);
  float* tensor_sums = block_sums + h.tiles;
  *out = {block_sums, tiles, first, (int)h.tensors, (int)h.tiles, (int)h.most};
  if (h.tensors == 0) return hipSuccess;
  if (h.chunks == 16)
    hipLaunchKernelGGL((k_list_squares<16, true>), dim3((unsigned)h.tiles), dim3(256), 0, stream, tiles, block_sums);
  else
    hipLaunchKernelGGL((k_list_squares<4, false>), dim3((unsigned)h.tiles), dim3(256), 0, stream, tiles, block_sums);
  if (h.most > 1 && !nested(h)) {
    hipLaunchKernelGGL(k_list_fold, dim3((unsigned)h.tensors), dim3(256), 0, stream, block_sums, first, (int64_t)0,
                       tensor_sums);
    out->values = tensor_sums;
  }
  if (h.tensors > kWaveFold) {
    float* total = tensor_sums + h.tensors;
    hipLaunchKernelGGL(k_list_fold, dim3(1), dim3(256), 0, stream, out->values, (const int64_t*)nullptr, h.tensors,
                       total);
    out->values = total;
    out->count = 1;
  }
  return hipGetLastError();
}

}  // namespace

bool size_list(const int64_t* sizes, const int32_t* dtypes, int64_t count, ListHeader* h) {
  *h = {};
  h->magic = kMagic;
  h->tensors = count;
  int64_t bytes = 0;
  for (int64_t t = 0; t < count; ++t) {
    if (sizes[t] > (int64_t(1) << 44)) return false;
    bytes += sizes[t] * (dtypes[t] == REPRO_BF16 ? 2 : 4);
    if (bytes > (int64_t(1) << 46)) return false;
  }
  h->chunks = bytes >= kLargeList ? 16 : 4;
  for (int64_t t = 0; t < count; ++t) {
    const int64_t per = tile_elements(dtypes[t], h->chunks);
    const int64_t tiles = sizes[t] > 0 ? (sizes[t] + per - 1) / per : 1;  // an empty tensor has an empty tile
    if (tiles > h->most) h->most = tiles;
    h->tiles += tiles;
    if (h->tiles > kMaxTiles) return false;
  }
  h->first_offset = sizeof(ListHeader) + h->tiles * (int64_t)sizeof(ListTile);
  h->sums_offset = up16(h->first_offset + (count + 1) * 8);
  h->bytes = up16(h->sums_offset + (h->tiles + count + 1) * 4);
  return true;
}

void fill_list(const ListHeader& h, const void* const* grads, void* const* outs, const int64_t* sizes,
               const int32_t* dtypes, void* host_plan) {
  uint8_t* plan = static_cast<uint8_t*>(host_plan);
  __builtin_memset(plan, 0, (size_t)h.bytes);
  ListTile* tile = reinterpret_cast<ListTile*>(plan + sizeof(ListHeader));
  int64_t* first = reinterpret_cast<int64_t*>(plan + h.first_offset);
  int64_t k = 0;
  for (int64_t t = 0; t < h.tensors; ++t) {
    const int64_t per = tile_elements(dtypes[t], h.chunks);
    const int64_t size = dtypes[t] == REPRO_BF16 ? 2 : 4;
    const char* src = static_cast<const char*>(grads[t]);
    char* dst = outs != nullptr && outs[t] != nullptr ? static_cast<char*>(outs[t]) : const_cast<char*>(src);
    first[t] = k;
    int64_t at = 0;
    do {
      const int64_t n = sizes[t] - at < per ? sizes[t] - at : per;
      tile[k] = {src + at * size, dst + at * size, (int32_t)n, dtypes[t] == REPRO_BF16, (int32_t)(k - first[t]), 0};
      ++k;
      at += per;
    } while (at < sizes[t]);
    for (int64_t i = first[t]; i < k; ++i) tile[i].count = (int32_t)(k - first[t]);
  }
  first[h.tensors] = k;
  *reinterpret_cast<ListHeader*>(plan) = h;
}

hipError_t launch_list_norm(const ListHeader& h, uint8_t* plan, float max_norm, float* out3, hipStream_t stream) {
  Sums sums;
  const hipError_t e = launch_sums(h, plan, &sums, stream);
  if (e != hipSuccess) return e;
  if (nested(h))
    hipLaunchKernelGGL(k_list_finish<true>, dim3(1), dim3(256), 0, stream, sums, max_norm, out3);
  else
    hipLaunchKernelGGL(k_list_finish<false>, dim3(1), dim3(64), 0, stream, sums, max_norm, out3);
  return hipGetLastError();
}

hipError_t launch_list_clip(const ListHeader& h, uint8_t* plan, float max_norm, float* out3, hipStream_t stream) {
  if (h.chunks == 16 || h.tensors == 0) {
    const hipError_t e = launch_list_norm(h, plan, max_norm, out3, stream);
    if (e != hipSuccess || h.tensors == 0) return e;
    const ListTile* tiles = reinterpret_cast<const ListTile*>(plan + sizeof(ListHeader));
    // A launch holds fewer than 2^32 threads, 4096 for each tile.
    constexpr int64_t kTiles = int64_t(1) << 19;
    for (int64_t t = 0; t < h.tiles; t += kTiles) {
      const int64_t n = h.tiles - t < kTiles ? h.tiles - t : kTiles;
      hipLaunchKernelGGL(k_list_stream<64>, dim3((unsigned)n * 64), dim3(64), 0, stream, tiles + t, out3);
    }
    return hipGetLastError();
  }
  Sums sums;
  const hipError_t e = launch_sums(h, plan, &sums, stream);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)h.tiles), block(256);
  if (nested(h))
    hipLaunchKernelGGL((k_list_scale<4, true>), grid, block, 0, stream, sums, max_norm, out3);
  else
    hipLaunchKernelGGL((k_list_scale<4, false>), grid, block, 0, stream, sums, max_norm, out3);
  return hipGetLastError();
}

}  // namespace repro
