// Block products on the matrix cores: one workgroup's tile of C[m][n] = the sum
// over k of A[m][k] B[n][k], the building block of the vocabulary loss
// (loss.hip).
//
// Mathematics.  A and B are bf16, stored either way; each C[m][n] is one chain
// over k in ascending groups of eight, as the matrix instructions with bf16
// operands compute it (repro.h declares one step of it, so that a CPU finds
// the same words).  A binary32 matrix is three bf16 ones whose sum it is, and for
// each 32 k six products of them, the smallest first, continue one chain.
//
// Design for gfx950.  A tile of 256 x 256 is held in the accumulators of four
// waves, 128 x 128 each, so a stage of 32 k reads 128 KB of fragments for
// 64 KB of new data and 1024 cycles of matrix instructions: the most
// arithmetic for each byte that the LDS can give.  Stages go from memory to
// the LDS without registers, four of them in a ring: three are under way while
// one is read, and one barrier a stage orders both.  A matrix whose k is not
// contiguous (its rows are the k) keeps its rows in the LDS, and the LDS turns
// 4 x 16 elements on the way to the registers.  Tiles of 8192 x 2048 over 16384
// k: 1272 TFLOP/s with random numbers, which the card's power bounds (a library
// product of 8192^3 reaches 1211; zeros run at 1500 to 1740 here).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace repro {
namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kStageK = 32;   // k of a stage: 64 bytes of a row
constexpr int kParts = 6;     // products of a binary32 pair

// One side of a tile.  Rows along k: from the tile's first row and first k on.
// K rows: from the first k's row and the tile's first column on.
struct Side16 {
  const uint16_t* at;  // plane 0
  int64_t plane;       // elements from one plane to the next
  uint32_t pitch;      // bytes of a row
  uint32_t bytes;      // rows along k: from the first byte to the last row's end; k rows: of a row, to its end
  int64_t k_rows;      // k rows: that there are; the k behind them are zeros
};

// The planes of part p (0 high, 1 middle, 2 low).
__device__ __forceinline__ constexpr int plane_a(int p) { return p == 0 ? 2 : p == 2 || p == 3 ? 1 : 0; }
__device__ __forceinline__ constexpr int plane_b(int p) { return p == 1 ? 2 : p == 2 || p == 4 ? 1 : 0; }

__device__ __forceinline__ i32x4 buffer_of(const uint16_t* p, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)at), __builtin_amdgcn_readfirstlane((int)(at >> 32)),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

// 64 lanes' 16 bytes at `voffset` + `soffset` of a buffer to 1 KB of the LDS.
// The bound is that of a raw buffer in the chip's published instruction set: a
// dword is out of range where voffset, with its place among the four, is not
// below the buffer's bytes less soffset, each dword for itself; it arrives as a
// zero, and nothing is read.  (Checked inside a larger allocation, with buffers
// of 0, 64, 100, 102 and 512 bytes and soffsets of 0 to 1024: the difference does not
// wrap below zero, and of 100 bytes at soffset 64 nine dwords arrive.)  Not
// tracked by the compiler (which holds nothing in m0): wait_stage orders it.
__device__ __forceinline__ void to_lds(uint32_t lds, uint32_t voffset, const i32x4& buffer, uint32_t soffset) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voffset), "s"(buffer), "s"(soffset));
}

// Waits until at most `pending` of this wave's transfers are under way and its
// LDS reads have arrived, then for the other waves.
template <int pending>
__device__ __forceinline__ void wait_stage() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(pending) : "memory");
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

// One side's stages: EDGE rows or columns of the tile, moved by WAVES waves;
// a wave reads FRAGS fragments of 32.  K: the matrix's rows are the k.
template <bool K, int EDGE, int WAVES, int FRAGS>
struct Stages {
  static constexpr int kLoads = EDGE / 16 / WAVES;  // transfers of a wave
  static constexpr int kReads = K ? 2 : 1;          // of a fragment
  static constexpr uint32_t kBytes = EDGE * 64, kRow = K ? EDGE * 2 : 64;  // of a stage, of its rows in the LDS
  static_assert(kLoads * 16 * WAVES == EDGE, "whole loads");
  static_assert(!K || EDGE == 256 || EDGE == 128, "turn_of knows these rows");

  const Side16& side;
  uint32_t voff[kLoads];
  uint32_t first[K ? FRAGS : 2];
  int64_t left;       // k rows from this stage on
  const uint16_t* at;  // of this stage
  uint32_t soffset;

  // Where a row's parts lie in the LDS turns with the row, so that the lanes of
  // one read meet different banks.  Rows along k: four pieces of 16 bytes, read
  // by eight or sixteen neighbouring rows at once.  K rows: pieces of 64 bytes,
  // read by rows 0..3 and 8..11 (or 4..7, 12..15) at once.
  static __device__ __forceinline__ uint32_t turn_of(uint32_t row) {
    if constexpr (!K) return ((row >> 1) & 3) ^ ((row >> 3) & 1);
    if constexpr (EDGE == 256) return (row & 3) | ((row >> 3) & 1) << 2;
    return ((row >> 1) & 1) | ((row >> 3) & 1) << 1;
  }

  __device__ __forceinline__ Stages(const Side16& s, int wave, int lane, int part)
      : side(s), left(s.k_rows), at(s.at), soffset(0) {
    constexpr int kLanes = kRow / 16;  // of a row
    const uint32_t in = lane / kLanes, piece = lane % kLanes;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t row = (wave * kLoads + i) * (64 / kLanes) + in;
      if constexpr (K)
        voff[i] = row * side.pitch + ((piece >> 2) ^ turn_of(row)) * 64 + (piece & 3) * 16;
      else
        voff[i] = row * side.pitch + (piece ^ turn_of(row)) * 16;
    }
    if constexpr (K) {
      const uint32_t row = ((lane & 15) >> 2) + 8 * (lane >> 5);
#pragma unroll
      for (int f = 0; f < FRAGS; ++f)
        first[f] = row * kRow + ((part * FRAGS + f) ^ turn_of(row)) * 64 + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    } else {
      // Lane (row r, half h) reads pieces h and 2 + h of its rows.
      const uint32_t r = lane & 31, h = lane >> 5;
      first[0] = (part * FRAGS * 32 + r) * 64 + (h ^ turn_of(r)) * 16;
      first[1] = first[0] ^ 32;
    }
  }

  // This stage of one plane, as its transfers take it.
  __device__ __forceinline__ i32x4 buffer(int plane) const {
    uint32_t bytes = side.bytes;
    if constexpr (K) bytes = left > 0 ? (left < kStageK ? (uint32_t)left - 1 : kStageK - 1) * side.pitch + side.bytes : 0;
    return buffer_of(at + plane * side.plane, bytes);
  }
  // Transfers [from, to) of it to the stage at `lds`.
  __device__ __forceinline__ void issue(const i32x4& buffer, uint32_t lds, int wave, int from, int to) const {
#pragma unroll
    for (int i = from; i < to; ++i) to_lds(lds + (wave * kLoads + i) * 1024, voff[i], buffer, soffset);
  }
  __device__ __forceinline__ void advance() {
    if constexpr (K) {
      at += kStageK / 2 * (int64_t)side.pitch;
      left -= kStageK;
    } else {
      soffset += 64;
    }
  }
  // Read q of fragment f for the k half `set` of the stage at `lds`.
  __device__ __forceinline__ void read(const char* lds, int set, int f, int q, s16x4 (&to)[2]) const {
    if constexpr (K) {
      to[q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)(lds + first[f] + (set * 16 + q * 4) * kRow));
    } else {
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      const s16x8 v = *reinterpret_cast<const s16x8*>(lds + first[set] + f * 2048);
      to[0] = __builtin_shufflevector(v, v, 0, 1, 2, 3);
      to[1] = __builtin_shufflevector(v, v, 4, 5, 6, 7);
    }
  }
};

// WM x WN waves of TM x TN matrix tiles of 32 x 32; KA, KB: the sides whose
// rows are the k.
template <int WM, int WN, int TM, int TN, int PARTS, bool KA = false, bool KB = false,
          int STAGES = 4>
struct Product {
  static constexpr int kWaves = WM * WN, kBlockM = WM * TM * 32, kBlockN = WN * TN * 32, kStages = STAGES;
  typedef Stages<KA, kBlockM, kWaves, TM> A;
  typedef Stages<KB, kBlockN, kWaves, TN> B;
  static constexpr int kLoads = A::kLoads + B::kLoads, kFirstLoads = kLoads / 2;
  static constexpr uint32_t kStageBytes = A::kBytes + B::kBytes, kLdsBytes = kStages * kStageBytes;
  static constexpr int kProducts = TM * TN, kReads = TM * A::kReads + TN * B::kReads;
  // How many of `count` stand before step t of half a set's products.
  static constexpr __device__ int share(int count, int t) { return count * t / (kProducts / 2); }
  static_assert(TM == 4, "a wave's rows are a block of the statistics");

  // Read q of a set: whose it is, in the order in which the products need them.
  struct Which {
    bool a;
    int f, q;
  };
  static constexpr __device__ Which which(int q) {
    for (int o = 0; o < TM + TN; ++o) {
      const bool a = o == 1 || o > TN;
      const int each = a ? A::kReads : B::kReads;
      if (q < each) return {a, a ? (o == 1 ? 0 : o - TN) : (o == 0 ? 0 : o - 1), q};
      q -= each;
    }
    return {};
  }

  // acc[i][j] = the wave's tile rows 32 i, columns 32 j over k_stages (one at
  // least) stages, from +0.  All waves of the workgroup call it; the ring is
  // free afterwards.
  static __device__ __forceinline__ void run(const Side16& sa, const Side16& sb, int k_stages, char* ring,
                                             f32x16 (&acc)[TM][TN]) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)ring;
    A a(sa, wave, lane, wave % WM);
    B b(sb, wave, lane, wave / WM);
    const int total = PARTS * k_stages;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};

    // The transfers [from, to) of the stage to come, of part `part`, into slot
    // `slot` of the ring.
    struct Next {
      i32x4 a, b;
    };
    const auto following = [&](int part) {
      return Next{a.buffer(PARTS == 1 ? 0 : plane_a(part)), b.buffer(PARTS == 1 ? 0 : plane_b(part))};
    };
    const auto issue = [&](const Next& next, int slot, int from, int to) {
      const uint32_t at = base + slot * kStageBytes;
      const int to_a = to < A::kLoads ? to : A::kLoads, from_b = from > A::kLoads ? from - A::kLoads : 0;
      if (from < to_a) a.issue(next.a, at, wave, from, to_a);
      if (from_b < to - A::kLoads) b.issue(next.b, at + A::kBytes, wave, from_b, to - A::kLoads);
    };
    const auto advance = [&](int part) {
      if (part + 1 < PARTS) return;
      a.advance();
      b.advance();
    };
    s16x4 fa[2][TM][2], fb[2][TN][2];
    const auto read = [&](int set, uint32_t at, int q) {
      const Which w = which(q);
      if (w.a)
        a.read(ring + at, set, w.f, w.q, fa[set][w.f]);
      else
        b.read(ring + at + A::kBytes, set, w.f, w.q, fb[set][w.f]);
    };
    const auto whole = [](const s16x4 (&h)[2]) {
      return __builtin_bit_cast(bf8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    };
    // A set's products.  Behind each one stands its share of the other set's
    // reads (in the first half) and of the transfers (in the second), as the
    // LDS and memory take them while the matrix pipe runs; more at once would
    // hold up the next product.
    const auto multiply = [&](int set, uint32_t at, auto&& transfers) {
#pragma unroll
      for (int t = 0; t < kProducts; ++t) {
        const int i = t / TN, j = t % TN;
        acc[i][j] =
            __builtin_amdgcn_mfma_f32_32x32x16_bf16(whole(fa[set][i]), whole(fb[set][j]), acc[i][j], 0, 0, 0);
        if (t < kProducts / 2) {
#pragma unroll
          for (int q = share(kReads, t); q < share(kReads, t + 1); ++q) read(set ^ 1, at, q);
        } else {
          transfers(t - kProducts / 2);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };

#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i >= total) continue;
      issue(following(i % PARTS), i, 0, kLoads);
      advance(i % PARTS);
    }
    if (total >= kStages - 1)
      wait_stage<(kStages - 2) * kLoads>();
    else
      wait_stage<0>();
#pragma unroll
    for (int q = 0; q < kReads; ++q) read(0, 0, q);
    // Stage s, of part `part`.
    const auto stage = [&](int s, int part, auto more) {
      constexpr bool kMore = decltype(more)::value;
      const uint32_t at = (s % kStages) * kStageBytes, next = ((s + 1) % kStages) * kStageBytes;
      const int slot = (s + kStages - 1) % kStages, coming = (part + kStages - 1) % PARTS;
      Next to_come = {};
      if (kMore) to_come = following(coming);
      multiply(0, at, [&](int t) {
        if (kMore) issue(to_come, slot, share(kFirstLoads, t), share(kFirstLoads, t + 1));
      });
      // The next stage has landed, and every wave has read this one.
      wait_stage<kMore ? (kStages - 3) * kLoads + kFirstLoads : 0>();
      // Past the last stage the reads find an old one, which nothing uses.
      multiply(1, next, [&](int t) {
        if (kMore)
          issue(to_come, slot, kFirstLoads + share(kLoads - kFirstLoads, t),
                kFirstLoads + share(kLoads - kFirstLoads, t + 1));
      });
      if (kMore) advance(coming);
    };
    int s = 0;
    if constexpr (PARTS == 1) {
      for (; s + kStages - 1 < total; ++s) stage(s, 0, std::true_type{});
      for (; s < total; ++s) stage(s, 0, std::false_type{});
    } else {
      for (; s < total - PARTS; s += PARTS)
#pragma unroll
        for (int part = 0; part < PARTS; ++part) stage(s + part, part, std::true_type{});
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        if (part + kStages - 1 < PARTS)
          stage(s + part, part, std::true_type{});
        else
          stage(s + part, part, std::false_type{});
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
};

}  // namespace
}  // namespace repro
