// q8_tile.hpp -- what the tiled products share: direct loads to LDS, barriers, the order
// of tiles over the chip and the sum of partial results (internal to libs2r).
#pragma once

#include <type_traits>
#include <utility>

#include "q8_device.hpp"
#include "s2r_device.hpp"

namespace s2r {

// f(first), ..., f(end - 1) with constants: the compiler gives up unrolling long bodies.
template <int FIRST, class F, int... I>
__device__ inline void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, FIRST + I>()), ...);
}
template <int FIRST, int END, class F>
__device__ inline void each(F&& f) {
  each_of<FIRST>(f, std::make_integer_sequence<int, END - FIRST>());
}

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
// workgroups that run together on a die share rows and columns of both operands.  Each kTileGroup rows begin
// an eighth of the columns further on, so that the lines that the dies write at a time lie on different memory channels
// (4-bit product 16384 x 8192 x 4096: to bf16 280 us, 290 without; to fp32 347 and 402).
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
  t.col = in / height + g % kXcds * cols / kXcds;  // the same for all of these rows
  t.col = t.col < cols ? t.col : t.col - cols;
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
  // ragged: what is there is read at once, then added to; four columns together where the row has them
  const bool four = k + 4 <= K;
  if (accumulate) {
    f32x4 old[8] = {};
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) {
      if (n0 + lane / 16 + 4 * e >= N) continue;
      if (four) {
        old[e] = *reinterpret_cast<const f32x4_a4*>(at + 4 * e * ld);
      } else {
#pragma unroll
        for (uint32_t c = 0; c < 3; ++c)
          if (k + c < K) old[e][c] = at[4 * e * ld + c];
      }
    }
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) v[e] += old[e];
  }
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e) {
    if (n0 + lane / 16 + 4 * e >= N) continue;
    if (four) {
      *reinterpret_cast<f32x4_a4*>(at + 4 * e * ld) = v[e];
    } else {
#pragma unroll
      for (uint32_t c = 0; c < 3; ++c)
        if (k + c < K) at[4 * e * ld + c] = v[e][c];
    }
  }
}

// 16-byte piece s of a 128-byte LDS row p lies at s ^ spread(p): the 32 lanes that read one piece of
// 32 rows meet every bank once.
__host__ __device__ constexpr int lesser(int a, int b) { return a < b ? a : b; }
__device__ inline uint32_t spread(uint32_t p) { return p / 2 % 4 | p / 16 % 2 << 2; }

// ROWS x 64 results from LDS: rows m0, m0 + step, ..., columns n0 .. n0 + 63; lane l takes eight
// columns of rows l / 8 + 8 k.  They leave through a view that ends with row M - 1; lanes
// without eight columns aim beyond its end.
template <int DT, int ROWS>
__device__ inline void store_rows(const s2r_mat& c, const f32x4 (&v)[ROWS / 8][2], uint32_t m0, uint32_t step,
                                  uint32_t M, uint32_t n0, uint32_t N) {
  constexpr uint32_t size = elem_bytes<DT>(), kNowhere = 0xffff0000u;
  const uint64_t first = (uint64_t)m0 * c.ld + n0, last = (uint64_t)(M - 1) * c.ld + N;
  const auto view = rsrc_of((uint64_t)c.data + first * size, (last - first) * size);
  const uint32_t lane = threadIdx.x % 64, n = lane % 8 * 8;
  const uint32_t ld = step * (uint32_t)c.ld * size;
  const uint32_t at = n0 + n < N ? lane / 8 * ld + n * size : kNowhere;
#pragma unroll
  for (uint32_t k = 0; k < ROWS / 8; ++k) {
    const uint32_t to = n0 + n < N ? at + 8 * k * ld : kNowhere;
    const f32x4 lo = v[k][0], hi = v[k][1];
    if (DT == S2R_F32) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, lo), view, to, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, hi), view, to + 16, 0, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b128(
          u32x4{pack2<DT>(lo[0], lo[1]), pack2<DT>(lo[2], lo[3]), pack2<DT>(hi[0], hi[1]),
                pack2<DT>(hi[2], hi[3])}, view, to, 0, 0);
    }
  }
}

template <int ROWS>
__device__ inline void store_turned(const s2r_mat& c, const uint8_t* lds, uint32_t m0, uint32_t step,
                                    uint32_t M, uint32_t n0, uint32_t N) {
  if (m0 >= M || n0 >= N) return;
  const uint32_t lane = threadIdx.x % 64, s = lane % 8 * 2;
  if (n0 + 64 > N && N % 8 != 0) {  // a lane may have fewer than eight columns
#pragma unroll 1
    for (uint32_t row = lane / 8; row < ROWS; row += 8) {
      const uint32_t m = m0 + step * row, n = n0 + lane % 8 * 8;
      const f32x4 lo = *reinterpret_cast<const f32x4*>(lds + turned(row, s));
      const f32x4 hi = *reinterpret_cast<const f32x4*>(lds + turned(row, s + 1));
      if (m < M && n < N) store8(c, m, n, N, lo, hi);
    }
    return;
  }
  f32x4 v[ROWS / 8][2];
#pragma unroll
  for (uint32_t k = 0; k < ROWS / 8; ++k) {
    v[k][0] = *reinterpret_cast<const f32x4*>(lds + turned(lane / 8 + 8 * k, s));
    v[k][1] = *reinterpret_cast<const f32x4*>(lds + turned(lane / 8 + 8 * k, s + 1));
  }
  if (c.dtype == S2R_BF16) {
    store_rows<S2R_BF16, ROWS>(c, v, m0, step, M, n0, N);
  } else if (c.dtype == S2R_F16) {
    store_rows<S2R_F16, ROWS>(c, v, m0, step, M, n0, N);
  } else {
    store_rows<S2R_F32, ROWS>(c, v, m0, step, M, n0, N);
  }
}

// One 32 x 32 fragment of results from registers to rows m0 .., columns n0 .. of c: lane (r, g) holds row r,
// columns 8 (q / 4) + 4 g + q % 4.  Of 16-bit results the lane halves swap four columns each, so that every lane
// has eight side by side; a row's 32 bytes leave together and meet the rest of their line in L2.
// `view` begins with row m0, column n0 of the wave and ends with row M - 1: rows beyond it leave nothing.
template <int DT>
__device__ inline void store_fragment(const f32x16& x, __amdgpu_buffer_rsrc_t view, uint32_t at) {
  if (DT == S2R_F32) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      __builtin_amdgcn_raw_buffer_store_b128(
          u32x4{__float_as_uint(x[4 * q]), __float_as_uint(x[4 * q + 1]), __float_as_uint(x[4 * q + 2]),
                __float_as_uint(x[4 * q + 3])}, view, at + 32 * q, 0, 0);
    return;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t v[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) v[w] = pack2<DT == S2R_F32 ? S2R_BF16 : DT>(x[8 * p + 2 * w], x[8 * p + 2 * w + 1]);
    // the upper lanes' first four columns for the lower lanes' next four
    const auto lo = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{lo[0], hi[0], lo[1], hi[1]}, view, at + 32 * p, 0, 0);
  }
}

// All FM x FN fragments of a wave: lane r of fragment i has row m0 + 32 i + r, or with TURNS
// m0 + FM r + i.
template <int FM, int FN, bool TURNS = false>
__device__ inline void store_wave(const s2r_mat& c, const f32x16 (&acc)[FM][FN], uint32_t m0, uint32_t M, uint32_t n0,
                                  uint32_t N) {
  const uint32_t lane = threadIdx.x % 64, r = lane % 32, g = lane / 32;
  const uint32_t size = c.dtype == S2R_F32 ? 4 : 2, ld = (uint32_t)c.ld * size;
  const bool ragged = n0 + 32 * FN > N && N % 8 != 0;  // a lane may have fewer columns than it stores
  const uint64_t first = (uint64_t)m0 * c.ld + n0, last = (uint64_t)(M - 1) * c.ld + N;
  const auto view = rsrc_of((uint64_t)c.data + first * size, (last - first) * size);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const uint32_t n = n0 + 32 * j;
      if (n >= N) continue;
      f32x16 x = acc[i][j];
      // stays where the matrix instruction left it until here: all of them would not fit beside each other
      asm volatile("" : "+a"(x));
      const uint32_t row = TURNS ? FM * r + i : 32 * i + r;
      if (ragged || n + 32 > N) {
        const uint32_t m = m0 + row;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (m < M && n + 8 * q + 4 * g < N)
            store4(c, m, n + 8 * q + 4 * g, N, f32x4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]});
      } else if (c.dtype == S2R_BF16) {
        store_fragment<S2R_BF16>(x, view, row * ld + 64 * j + 16 * g);
      } else if (c.dtype == S2R_F16) {
        store_fragment<S2R_F16>(x, view, row * ld + 64 * j + 16 * g);
      } else {
        store_fragment<S2R_F32>(x, view, row * ld + 128 * j + 16 * g);
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
