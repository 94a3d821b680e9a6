// Block products on the matrix cores: one workgroup's tile of C = A B^T, the
// building block of the vocabulary loss (loss.hip).
//
// Mathematics.  A and B are bf16, with k contiguous; each C[m][n] is one chain
// over k in ascending groups of eight, as the matrix instructions with bf16
// operands compute it (repro.h declares one step of it, so that a CPU finds
// the same words; tests/product_oracle.c).  A binary32 matrix is three bf16 ones whose
// sum it is, and for each 32 k six products of them, the smallest first, continue
// one chain.
//
// Design for gfx950.  A tile of 256 x 256 is held in the accumulators of four
// waves, 128 x 128 each, so a stage of 32 k reads 128 KB of fragments for
// 64 KB of new data and 1024 cycles of matrix instructions: the most
// arithmetic for each byte that the LDS can give.  Stages go from memory to
// the LDS without registers, four of them in a ring: three are under way while
// one is read, and one barrier a stage orders both.
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

// One side's rows of a tile, from the first k on.
struct Rows16 {
  const uint16_t* at;  // plane 0
  int64_t plane;       // elements from one plane to the next
  uint32_t pitch;      // bytes of a row
  uint32_t bytes;      // from the first row's first byte to the last row's end
};

// The planes of part p (0 high, 1 middle, 2 low).
__device__ __forceinline__ constexpr int plane_a(int p) { return p == 0 ? 2 : p == 2 || p == 3 ? 1 : 0; }
__device__ __forceinline__ constexpr int plane_b(int p) { return p == 1 ? 2 : p == 2 || p == 4 ? 1 : 0; }

__device__ __forceinline__ i32x4 buffer_of(const Rows16& r, int plane) {
  const uint64_t at = reinterpret_cast<uint64_t>(r.at + plane * r.plane);
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)at), __builtin_amdgcn_readfirstlane((int)(at >> 32)),
               __builtin_amdgcn_readfirstlane((int)r.bytes), 0x00020000};
}

// 64 lanes' 16 bytes at `voffset` + `soffset` of a buffer to 1 KB of the LDS;
// lanes past the buffer's bytes read nothing from memory.  Not tracked by the
// compiler (which holds nothing in m0): wait_stage orders it.
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

// A row's four 16-byte pieces of a stage lie in the LDS in an order that turns
// with the row, so that eight or sixteen rows' reads of one piece meet
// different banks.
__device__ __forceinline__ uint32_t turn_of(uint32_t row) { return ((row >> 1) & 3) ^ ((row >> 3) & 1); }

// WM x WN waves of TM x TN matrix tiles of 32 x 32.
template <int WM, int WN, int TM, int TN, int PARTS, int kStages = 4>
struct Product {
  static constexpr int kWaves = WM * WN, kBlockM = WM * TM * 32, kBlockN = WN * TN * 32;
  static constexpr int kLoadsA = kBlockM / 16 / kWaves, kLoadsB = kBlockN / 16 / kWaves, kLoads = kLoadsA + kLoadsB;
  static constexpr uint32_t kBytesA = kBlockM * 64, kBytesB = kBlockN * 64, kStageBytes = kBytesA + kBytesB;
  static constexpr uint32_t kLdsBytes = kStages * kStageBytes;
  static constexpr int kProducts = TM * TN, kReads = TM + TN, kFirstLoads = kLoads / 2;
  // How many of `count` stand before step t of half a set's products.
  static constexpr __device__ int share(int count, int t) { return count * t / (kProducts / 2); }
  static_assert(TM == 4, "a wave's rows are a block of the statistics");
  static_assert(kLoadsA * 16 * kWaves == kBlockM && kLoadsB * 16 * kWaves == kBlockN, "whole loads");

  struct Feed {
    const Rows16 &a, &b;
    uint32_t voff_a[kLoadsA], voff_b[kLoadsB];
    uint32_t lds, soffset;
    int part;

    __device__ Feed(const Rows16& a_, const Rows16& b_, uint32_t base, int wave, int lane)
        : a(a_), b(b_), lds(base), soffset(0), part(0) {
      const uint32_t row = lane >> 2, piece = ((lane & 3) ^ turn_of(row)) * 16;
#pragma unroll
      for (int i = 0; i < kLoadsA; ++i) voff_a[i] = ((wave * kLoadsA + i) * 16 + row) * a.pitch + piece;
#pragma unroll
      for (int i = 0; i < kLoadsB; ++i) voff_b[i] = ((wave * kLoadsB + i) * 16 + row) * b.pitch + piece;
    }
    // Transfers [from, to) of the next stage into slot `slot` of the ring.
    __device__ __forceinline__ void issue(int wave, int slot, int from, int to) {
      const uint32_t at = lds + slot * kStageBytes;
      const i32x4 buffer_a = buffer_of(a, PARTS == 1 ? 0 : plane_a(part));
      const i32x4 buffer_b = buffer_of(b, PARTS == 1 ? 0 : plane_b(part));
#pragma unroll
      for (int i = from; i < to; ++i) {
        if (i < kLoadsA)
          to_lds(at + (wave * kLoadsA + i) * 1024, voff_a[i], buffer_a, soffset);
        else
          to_lds(at + kBytesA + (wave * kLoadsB + i - kLoadsA) * 1024, voff_b[i - kLoadsA], buffer_b, soffset);
      }
    }
    __device__ __forceinline__ void advance() {
      if (PARTS == 1 || ++part == PARTS) {
        part = 0;
        soffset += 64;
      }
    }
  };

  // acc[i][j] = the wave's tile rows 32 i, columns 32 j of A B^T over
  // k_stages (one at least) stages, from +0.  All waves of the workgroup call
  // it; the ring is free afterwards.
  static __device__ __forceinline__ void run(const Rows16& a, const Rows16& b, int k_stages, char* ring,
                                             f32x16 (&acc)[TM][TN]) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave % WM, wn = wave / WM;
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)ring;
    Feed feed(a, b, base, wave, lane);
    const int total = PARTS * k_stages;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};

    // Lane (row r, half h) reads pieces h and 2 + h of its rows.
    const uint32_t r = lane & 31, h = lane >> 5;
    const uint32_t first = r * 64 + (h ^ turn_of(r)) * 16;
    const char* pa[2] = {ring + wm * (TM * 2048) + first, ring + wm * (TM * 2048) + (first ^ 32)};
    const char* pb[2] = {ring + kBytesA + wn * (TN * 2048) + first, ring + kBytesA + wn * (TN * 2048) + (first ^ 32)};
    bf8 fa[2][TM], fb[2][TN];
    // Fragment q of a set, in the order in which the products need them.
    const auto read = [&](int set, uint32_t at, int q) {
      if (q == 1 || q > TN) {
        const int i = q == 1 ? 0 : q - TN;
        fa[set][i] = *reinterpret_cast<const bf8*>(pa[set] + at + i * 2048);
      } else {
        const int j = q == 0 ? 0 : q - 1;
        fb[set][j] = *reinterpret_cast<const bf8*>(pb[set] + at + j * 2048);
      }
    };
    // A set's products.  Behind each one stands its share of the other set's
    // reads (in the first half) and of the transfers (in the second), as the
    // LDS and memory take them while the matrix pipe runs; more at once would
    // hold up the next product.
    const auto multiply = [&](int set, uint32_t at, auto&& transfers) {
#pragma unroll
      for (int t = 0; t < kProducts; ++t) {
        const int i = t / TN, j = t % TN;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[set][i], fb[set][j], acc[i][j], 0, 0, 0);
        if (t < kProducts / 2) {
#pragma unroll
          for (int q = share(kReads, t); q < share(kReads, t + 1); ++q) read(set ^ 1, at, q);
        } else {
          transfers(t - kProducts / 2);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    int issued = 0;
    for (; issued < kStages - 1 && issued < total; ++issued) {
      feed.issue(wave, issued, 0, kLoads);
      feed.advance();
    }
    if (issued == kStages - 1)
      wait_stage<(kStages - 2) * kLoads>();
    else
      wait_stage<0>();
#pragma unroll
    for (int q = 0; q < kReads; ++q) read(0, 0, q);
    const auto stage = [&](int s, auto more) {
      constexpr bool kMore = decltype(more)::value;
      const uint32_t at = (s % kStages) * kStageBytes, next = ((s + 1) % kStages) * kStageBytes;
      const int slot = (s + kStages - 1) % kStages;
      multiply(0, at, [&](int t) {
        if (kMore) feed.issue(wave, slot, share(kFirstLoads, t), share(kFirstLoads, t + 1));
      });
      // The next stage has landed, and every wave has read this one.
      wait_stage<kMore ? (kStages - 3) * kLoads + kFirstLoads : 0>();
      // Past the last stage the reads find an old one, which nothing uses.
      multiply(1, next, [&](int t) {
        if (kMore)
          feed.issue(wave, slot, kFirstLoads + share(kLoads - kFirstLoads, t),
                     kFirstLoads + share(kLoads - kFirstLoads, t + 1));
      });
      if (kMore) feed.advance();
    };
    int s = 0;
    for (; s + kStages - 1 < total; ++s) stage(s, std::true_type{});
    for (; s < total; ++s) stage(s, std::false_type{});
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
};

}  // namespace
}  // namespace repro
