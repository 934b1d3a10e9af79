// q8_tile.hpp -- what the two tiled products share: direct loads to LDS, barriers, the order
// of tiles over the chip and the sum of partial results (internal to libs2r).
#pragma once

#include "q8_device.hpp"
#include "s2r_device.hpp"

namespace s2r {

constexpr uint32_t kTileCus = 256;   // compute units of an MI355X
constexpr uint32_t kTileGroup = 8;   // rows of tiles that are walked together

typedef __attribute__((address_space(3))) void lds_void;

// A bounds-checked view of global memory: reads at or beyond `bytes` give zeros.
__device__ inline __amdgpu_buffer_rsrc_t rsrc_of(uint64_t base, uint64_t bytes) {
  // offsets of a tile stay below 2^31 + 2^30: what ends beyond may as well end there
  const uint32_t n = bytes > 0xc0000000ull ? 0xc0000000u : (uint32_t)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, (int)n, 0x00020000);
}

// 16 bytes per lane from `at` bytes into the view to LDS, lane i at `lds` + 16 i; `lds` is
// the same for the wave.
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t at) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, at, 0, 0, 0);
}

// Every load of this wave has arrived and every LDS access is done, for all waves.
__device__ inline void drain_and_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The same with the wave's newest LEFT loads still on their way.
template <int LEFT>
__device__ inline void sync_but() {
  static_assert(LEFT >= 0 && LEFT < 64, "six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (LEFT & 15) | (LEFT >> 4) << 14);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Every LDS access of all waves is done; loads may be on their way.
__device__ inline void sync_reads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Item b of `total` to a tile and a part of the sum.  Consecutive workgroups go to the eight
// accelerator dies in turn, so the items are cut into eight stretches, one for each die and
// its L2; within a stretch kTileGroup rows of tiles are walked column by column, so that the
// workgroups that run together on a die share rows and columns of both operands.
struct TileAt {
  uint32_t row, col, part;
};
__device__ inline TileAt tile_at(uint32_t b, uint32_t rows, uint32_t cols, uint32_t total) {
  const uint32_t die = b % kXcds, per = total / kXcds, rem = total % kXcds;
  uint32_t lin = die * per + min(die, rem) + b / kXcds;
  TileAt t;
  t.part = lin / (rows * cols);
  lin -= t.part * (rows * cols);
  const uint32_t span = kTileGroup * cols, g = lin / span, first = g * kTileGroup;
  const uint32_t height = min(rows - first, kTileGroup), in = lin - g * span;
  t.row = first + in % height;
  t.col = in / height;
  // divisions run in vector registers: back to scalar ones
  t.row = __builtin_amdgcn_readfirstlane(t.row);
  t.col = __builtin_amdgcn_readfirstlane(t.col);
  t.part = __builtin_amdgcn_readfirstlane(t.part);
  return t;
}

// Results turn in LDS, 64 fp32 columns to a row: where 16-byte piece s of row p lies.  The lanes
// that write together, one piece of 16 rows, and those that read a row meet every bank once.
__device__ inline uint32_t turned(uint32_t p, uint32_t s) {
  return p * 256 + (s ^ (p % 8 | (p / 8 ^ p / 16) % 2 * 8)) * 16;
}

// 32 x 64 results from LDS to rows n0 .., columns k0 .. of dw, or added to what is there.  Four
// columns per lane, 16 lanes a row; dw is only known to be 4-byte aligned.
__device__ inline void add_turned(float* dw, uint64_t ld, const uint8_t* lds, uint32_t n0, uint32_t N,
                                  uint32_t k0, uint32_t K, bool accumulate) {
  if (n0 >= N || k0 >= K) return;
  typedef f32x4 __attribute__((aligned(4))) f32x4_a4;
  const uint32_t lane = threadIdx.x % 64, s = lane % 16, k = k0 + 4 * s;
  f32x4 v[8];
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e) {
    v[e] = *reinterpret_cast<const f32x4*>(lds + turned(lane / 16 + 4 * e, s));
  }
  float* const at = dw + (uint64_t)(n0 + lane / 16) * ld + k;
  if (n0 + 32 <= N && k0 + 64 <= K) {
    if (accumulate) {
      f32x4 old[8];
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) old[e] = *reinterpret_cast<const f32x4_a4*>(at + 4 * e * ld);
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) v[e] += old[e];
    }
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) *reinterpret_cast<f32x4_a4*>(at + 4 * e * ld) = v[e];
    return;
  }
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e) {
    if (n0 + lane / 16 + 4 * e >= N) continue;
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c) {
      float* const p = at + 4 * e * ld + c;
      if (k + c < K) *p = accumulate ? *p + v[e][c] : v[e][c];
    }
  }
}

// A sum cut into parts of whole blocks, each with its own partial results.
struct Cut {
  uint32_t parts, blocks;  // blocks of a part
};
inline Cut cut_evenly(uint32_t blocks, uint32_t parts) {
  if (blocks == 0) return {1, 0};
  const uint32_t each = (blocks + parts - 1) / parts;
  return {(blocks + each - 1) / each, each};
}

}  // namespace s2r
