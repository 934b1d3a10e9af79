// q8_gemm.hpp -- the tiled product of 8-bit matrices, for q8_gemm.hip and q8_experts.hip (internal to
// libs2r).  q8_gemm.hip has the mathematics and what it measured.
#pragma once

#include "moe_launch.hpp"
#include "q8_tile.hpp"

namespace s2r {

// ---- fragments ----------------------------------------------------------------------------
__device__ inline i32x8 join(u32x4 lo, u32x4 hi) {
  i32x8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = (int)lo[i];
    v[4 + i] = (int)hi[i];
  }
  return v;
}

// Codes 8 part .. + 7 of a lane's 32, as bf16.
template <int FMT>
__device__ inline bf16x8 widen8(const i32x8& c, int part, uint32_t sb) {
  const u32x2 lo = to_bf16<FMT>(c[2 * part], scale_value(sb)), hi = to_bf16<FMT>(c[2 * part + 1], scale_value(sb));
  return __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], hi[0], hi[1]});
}

__device__ inline void clear_from(i32x8& v, int left) {  // `left` bytes stay
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const int l = left - 4 * w;
    v[w] = l <= 0 ? 0 : l < 4 ? v[w] & (int)((1u << (8 * l)) - 1) : v[w];
  }
}

// `at` is the byte of `sa` that holds this fragment's scale.
template <int FA, int FB>
__device__ inline f32x16 mma32(const i32x8& b, const i32x8& a, const f32x16& c, uint32_t sb,
                               uint32_t sa, int at) {
  switch (at) {
    case 0:
      return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, FB, FA, 0, (int)sb, 0, (int)sa);
    case 1:
      return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, FB, FA, 0, (int)sb, 1, (int)sa);
    case 2:
      return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, FB, FA, 0, (int)sb, 2, (int)sa);
    default:
      return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, FB, FA, 0, (int)sb, 3, (int)sa);
  }
}

// ---- tiles --------------------------------------------------------------------------------
// WM x WN waves, each 32 FM rows of A by 32 FN rows of B; a block is 128 of the sum, one scale
// of every row.  LDS holds two blocks, 128 bytes of every row of both operands: one is
// multiplied while the next arrives straight from global memory, a whole line of each row.
// A block is multiplied in two halves of 64, and the fragments of a half are read into
// registers while the half before is multiplied: its LDS is free again after the first half.
// 16-byte piece s of LDS row p lies at s ^ spread(p): the lanes that read together meet every
// bank once.  Rows of A are taken in the order m = FM r + i (fragment i, lane r), so that the
// scales of a lane's fragments are one load.
// A workgroup stays for several tiles, and the blocks of all of them are one stream: the next
// tile's first blocks arrive while the last ones of this are multiplied and its results leave.
// With EXPERTS the rows of tiles are those of the experts, one after the other: LDS holds how many
// there are up to each expert, and a row of tiles ends where its expert does.
struct ExpertTiles {
  s2r_experts of;
  ExpertSteps steps;
};
// Tiles up to and with each expert, and those of each wave's experts: LDS that is there only where it is asked for, for
// the plain 256 x 256 form takes all there is.
template <int WAVES>
struct ExpertLds {
  uint32_t upto[S2R_MAX_EXPERTS], wave[WAVES];
};
template <int WAVES>
__device__ inline ExpertLds<WAVES>& expert_lds() {
  __shared__ ExpertLds<WAVES> x;
  return x;
}
constexpr int kLdsBytes = 160 * 1024;  // of a compute unit
template <int FA, int FB, int WM, int WN, int FM, int FN, bool TAIL, bool WIDE, bool EXPERTS>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_q8_gemm(
    s2r_q8_mat a, s2r_q8_mat b, s2r_mat c, uint64_t part_bytes, uint32_t M, uint32_t N, uint32_t K,
    uint32_t m_tiles, uint32_t n_tiles, uint32_t total, uint32_t part_blocks, ExpertTiles experts) {
  constexpr int kWaves = WM * WN, TM = 32 * FM * WM, TN = 32 * FN * WN;
  constexpr int kLoadsA = TM / 8 / kWaves, kLoads = (TM + TN) / 8 / kWaves;
  constexpr int kBytes = (TM + TN) * kQ8Block;
  static_assert(kLoads - kLoads * 5 / 8 <= FM * FN, "late loads have a slot each");
  constexpr int kTurnRows = kWaves > 4 ? 16 : 32, kTurn = kTurnRows * 64 * 4;  // a wave's results in LDS
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kBytes + (EXPERTS ? 0 : kWaves * kTurn)];
  static_assert(sizeof(lds) + (EXPERTS ? sizeof(ExpertLds<kWaves>) : 0) <= kLdsBytes, "");

  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, r = lane % 32, g = lane / 32;
  const uint32_t wm = wave / WN * (32 * FM), wn = wave % WN * (32 * FN);
  const uint32_t blocks = (K + kQ8Block - 1) / kQ8Block;

  if constexpr (EXPERTS) {
    ExpertLds<kWaves>& tiles = expert_lds<kWaves>();
    constexpr uint32_t kEach = S2R_MAX_EXPERTS / (64 * kWaves);  // experts of a thread
    uint32_t mine[kEach], sum = 0;
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
      const uint32_t e = threadIdx.x * kEach + i;
      const uint32_t first = e < experts.of.experts ? min(experts.of.first[e], M) : M;
      const uint32_t rows = e < experts.of.experts ? min(experts.of.rows[e], M - first) : 0;
      sum += (rows + TM - 1) / TM;
      mine[i] = sum;
    }
    uint32_t upto = sum;  // of the wave's threads
#pragma unroll
    for (uint32_t o = 1; o < 64; o <<= 1) {
      const uint32_t v = (uint32_t)__shfl_up((int)upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 63) tiles.wave[wave] = upto;
    __syncthreads();
    m_tiles = 0;
    uint32_t before = upto - sum;
    for (uint32_t w = 0; w < kWaves; ++w) {
      if (w < wave) before += tiles.wave[w];
      m_tiles += tiles.wave[w];
    }
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) tiles.upto[threadIdx.x * kEach + i] = before + mine[i];
    m_tiles = __builtin_amdgcn_readfirstlane(m_tiles);
    total = m_tiles * n_tiles;
    __syncthreads();
    if (blockIdx.x >= total) return;
  }
  // a row of tiles: its first row of A and C, the end of its rows, and its expert
  struct RowOf {
    uint32_t m0, end, expert;
  };
  auto row_of = [&](uint32_t tile) {
    if constexpr (EXPERTS) {
      const uint32_t* const upto = expert_lds<kWaves>().upto;
      uint32_t e = 0;  // experts whose tiles end at or before this one
      for (uint32_t i = 0; i < experts.of.experts; i += 64)
        e += (uint32_t)__popcll(__ballot(i + lane < experts.of.experts && upto[i + lane] <= tile));
      e = __builtin_amdgcn_readfirstlane(e);
      const uint32_t first = min(experts.of.first[e], M), rows = min(experts.of.rows[e], M - first);
      const uint32_t m0 = first + (tile - (e ? upto[e - 1] : 0)) * TM;
      return RowOf{(uint32_t)__builtin_amdgcn_readfirstlane(m0), (uint32_t)__builtin_amdgcn_readfirstlane(first + rows), e};
    } else {
      return RowOf{tile * TM, M, 0};
    }
  };

  // where this lane's pieces of a block come from, relative to the tile's first row
  uint32_t from[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const bool is_a = j < kLoadsA;
    const uint32_t p = (is_a ? wave * kLoadsA + j : wave * (kLoads - kLoadsA) + j - kLoadsA) * 8 + lane / 8;
    const uint32_t row = is_a ? p / (32 * FM) * (32 * FM) + FM * (p % 32) + p / 32 % FM : p;
    from[j] = row * (uint32_t)(is_a ? a.ld : b.ld) + (lane % 8 ^ spread(p)) * 16;
  }

  // The stream of blocks: the newest that is loaded, and the first one of the item after its
  // own.  The views end with the last row's last 16-byte piece.
  const uint32_t row_end = (K + 15) / 16 * 16;
  struct At {
    uint32_t item, left;  // blocks of the item after this one
    uint64_t a, b, len_a, len_b, scale_a;
    uint64_t scale_b;
    uint32_t lane_scale;
  };
  auto start_of = [&](uint32_t item) {
    At x = {};
    x.item = item;
    x.left = ~0u;  // nothing more: loads of zeros, and some scales or other
    x.scale_a = (uint64_t)a.scale;
    x.scale_b = (uint64_t)b.scale;
    if (item >= total) return x;
    const TileAt t = tile_at(item, m_tiles, n_tiles, total);
    const RowOf row = row_of(t.row);
    const uint32_t m0 = row.m0, n0 = t.col * TN, block = t.part * part_blocks;
    const uint64_t k = (uint64_t)block * kQ8Block;
    x.left = __builtin_amdgcn_readfirstlane(min(block + part_blocks, blocks) - block - 1);
    x.a = (uint64_t)a.q + (uint64_t)m0 * a.ld + k;
    x.b = (uint64_t)b.q + (uint64_t)n0 * b.ld + k;
    if (EXPERTS) {
      x.b += row.expert * experts.steps.step;
      x.scale_b += row.expert * experts.steps.scale_step;
    }
    x.len_a = (uint64_t)(row.end - m0 - 1) * a.ld + row_end - k;
    x.len_b = (uint64_t)(N - n0 - 1) * b.ld + row_end - k;
    x.scale_a += block * a.lds;
    x.scale_b += block * b.lds + min(n0 + wn, N - 1) / kQ8Block;
    x.lane_scale = min(m0 + wm + FM * r, (uint32_t)a.lds - FM);
    return x;
  };
  At in = {}, after = {};
  auto advance = [&] {  // without a branch: it runs between matrix instructions
    in.left = __builtin_amdgcn_readfirstlane(in.left);
    const bool go = in.left == 0, on = in.left + 1 > 1;
    in.item = go ? after.item : in.item;
    in.a = go ? after.a : in.a + kQ8Block;
    in.b = go ? after.b : in.b + kQ8Block;
    in.len_a = go ? after.len_a : on ? in.len_a - kQ8Block : 0;
    in.len_b = go ? after.len_b : on ? in.len_b - kQ8Block : 0;
    in.scale_a = go ? after.scale_a : on ? in.scale_a + a.lds : in.scale_a;
    in.scale_b = go ? after.scale_b : on ? in.scale_b + b.lds : in.scale_b;
    in.lane_scale = go ? after.lane_scale : in.lane_scale;
    in.left = go ? after.left : on ? in.left - 1 : ~0u;
  };
  struct Views {
    __amdgpu_buffer_rsrc_t a, b;
  };
  auto views = [&] { return Views{rsrc_of(in.a, in.len_a), rsrc_of(in.b, in.len_b)}; };
  auto load = [&](uint8_t* to, const Views& v, int j) {
    if (j < kLoadsA) load_to_lds(v.a, to + (wave * kLoadsA + j) * 1024, from[j]);
    else load_to_lds(v.b, to + TM * kQ8Block + (wave * (kLoads - kLoadsA) + j - kLoadsA) * 1024, from[j]);
  };
  auto load_scales = [&](uint32_t& sa, uint32_t& sb) {
    const uint8_t* at = reinterpret_cast<const uint8_t*>(in.scale_a) + in.lane_scale;
    sa = FM == 4 ? *reinterpret_cast<const uint32_t*>(at)
                 : FM == 2 ? *reinterpret_cast<const uint16_t*>(at) : *at;
    sb = *reinterpret_cast<const uint8_t*>(in.scale_b);
  };

  struct Frags {
    i32x8 a[FM], b[FN];
  };
  uint32_t at[2][2];  // where in a fragment's rows this lane's pieces of a half lie
#pragma unroll
  for (int h = 0; h < 4; ++h)
    at[h / 2][h % 2] = r * kQ8Block + ((h / 2 * 4 + 2 * g + h % 2) ^ spread(r)) * 16;
  // read e of a half's 2 (FM + FN)
  auto read = [&](Frags& f, const uint8_t* from_lds, int h, int e) {
    const int i = e / 2;
    const uint32_t row = i < FN ? TM + wn + 32 * i : wm + 32 * (i - FN);
    const u32x4 v = *reinterpret_cast<const u32x4*>(from_lds + row * kQ8Block + at[h][e % 2]);
    i32x8& to = i < FN ? f.b[i] : f.a[i - FN];
#pragma unroll
    for (int w = 0; w < 4; ++w) to[e % 2 * 4 + w] = (int)v[w];
  };
  auto clear_tail = [&](Frags& f, int left) {  // codes at or beyond K
#pragma unroll
    for (int i = 0; i < FM; ++i) clear_from(f.a[i], left - 32 * (int)g);
#pragma unroll
    for (int j = 0; j < FN; ++j) clear_from(f.b[j], left - 32 * (int)g);
  };
  // A half is multiplied in kSlots instructions: one for each pair of fragments, or four where codes
  // become bf16 (WIDE), eight of a lane's 32 at a time.  kRead of them cover the next half's
  // reads, loads begin after that.
  constexpr int kMma = FM * FN, kReads = 2 * (FM + FN), kSlots = WIDE ? 4 * kMma : kMma;
  constexpr int kRead = kSlots * 5 / 16, kEarly = kLoads * 5 / 8;
  struct Wide {
    bf16x8 a[FM], b[FN];
  };
  Wide wide[2];
  // fragment i of FN + FM, its eight codes number `part`
  auto widen = [&](Wide& to, const Frags& f, int part, int i, uint32_t sa, uint32_t sb) {
    if (i < FN) to.b[i] = widen8<FB>(f.b[i], part, sb);
    else to.a[i - FN] = widen8<FA>(f.a[i - FN], part, sa >> 8 * (i - FN) & 0xff);
  };

  uint8_t *here = lds, *there = lds + kBytes;
  uint32_t sa = 0, sb = 0, sa_ahead = 0, sb_ahead = 0;  // of this block and of the next
  Frags f0, f1;
  if (blocks > 0) {
    in = start_of(blockIdx.x);
    after = start_of(blockIdx.x + gridDim.x);
    Views v = views();
#pragma unroll
    for (int j = 0; j < kLoads; ++j) load(here, v, j);
    load_scales(sa, sb);
    advance();
    v = views();
#pragma unroll
    for (int j = 0; j < kLoads; ++j) load(there, v, j);
    load_scales(sa_ahead, sb_ahead);
    sync_but<kLoads>();
#pragma unroll
    for (int e = 0; e < kReads; ++e) read(f0, here, 0, e);
#pragma unroll
    for (int i = 0; i < (WIDE ? FM + FN : 0); ++i) widen(wide[0], f0, 0, i, sa, sb);
  }

  for (uint32_t item = blockIdx.x; item < total; item += gridDim.x) {
    const TileAt t = tile_at(item, m_tiles, n_tiles, total);
    const uint32_t b0 = t.part * part_blocks, b1 = min(b0 + part_blocks, blocks);
    after = start_of(in.item + gridDim.x);
    f32x16 acc[FM][FN] = {};
    auto multiply = [&](const Frags& f, int slot) {
      const int e = slot % kMma;
      f32x16& to = acc[e / FN][e % FN];
      if (WIDE) {
        const Wide& w = wide[slot / kMma % 2];
        to = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w.b[e % FN], w.a[e / FN], to, 0, 0, 0);
      } else {
        to = mma32<FA, FB>(f.b[e % FN], f.a[e / FN], to, sb, sa, e / FN);
      }
    };
    // beside the products of one part: the next part's codes, or the next half's first ones
    auto widen_ahead = [&](const Frags& f, const Frags& next, int slot, uint32_t sa_next, uint32_t sb_next) {
      if (!WIDE) return;
      const int part = slot / kMma, e = slot % kMma;
#pragma unroll
      for (int i = e * (FM + FN) / kMma; i < (e + 1) * (FM + FN) / kMma; ++i) {
        if (part < 3) widen(wide[(part + 1) % 2], f, part + 1, i, sa, sb);
        else widen(wide[0], next, 0, i, sa_next, sb_next);
      }
    };
    auto run = [&](auto clear, uint32_t block) {  // one block, without the codes at or beyond K
      if (clear) {
        clear_tail(f0, (int)(K - block * kQ8Block));
#pragma unroll
        for (int i = 0; i < (WIDE ? FM + FN : 0); ++i) widen(wide[0], f0, 0, i, sa, sb);
      }
      each<0, kRead>([&](auto e) {
        multiply(f0, e);
#pragma unroll
        for (int q = e * kReads / kRead; q < (e + 1) * kReads / kRead; ++q) read(f1, here, 1, q);
        if (e == 0) advance();
        widen_ahead(f0, f1, e, sa, sb);
        __builtin_amdgcn_sched_barrier(0);
      });
      multiply(f0, kRead);
      widen_ahead(f0, f1, kRead, sa, sb);
      sync_reads();  // this block's LDS is free
      const Views v = views();
      each<kRead + 1, kSlots>([&](auto e) {
        constexpr int kAt = e - kRead - 1, kOf = kSlots - kRead - 1;
        multiply(f0, e);
#pragma unroll
        for (int q = kAt * kEarly / kOf; q < (kAt + 1) * kEarly / kOf; ++q) load(here, v, q);
        if (!(clear && e / kMma == 3)) widen_ahead(f0, f1, e, sa, sb);
        __builtin_amdgcn_sched_barrier(0);
      });
      sync_but<kEarly>();  // the next block is there
      // moved here, where their loads are known to be done, and not by the compiler further up
      uint32_t sa_next, sb_next;
      asm volatile("v_mov_b32 %0, %1" : "=v"(sa_next) : "v"(sa_ahead));
      asm volatile("v_mov_b32 %0, %1" : "=v"(sb_next) : "v"(sb_ahead));
      load_scales(sa_ahead, sb_ahead);
      if (clear) {
        clear_tail(f1, (int)(K - block * kQ8Block) - 64);
#pragma unroll
        for (int i = 0; i < (WIDE ? FM + FN : 0); ++i) widen(wide[0], f1, 0, i, sa, sb);
      }
      constexpr int kReadLate = WIDE ? 3 * kMma : kMma;  // its first codes are widened after that
      each<0, kSlots>([&](auto e) {
        multiply(f1, e);
#pragma unroll
        for (int q = e * kReads / kReadLate; q < lesser((e + 1) * kReads / kReadLate, kReads); ++q)
          read(f0, there, 0, q);
#pragma unroll
        for (int q = kEarly + e * kMma / kSlots; q < lesser(kEarly + (e + 1) * kMma / kSlots, kLoads); ++q)
          load(here, v, q);
        widen_ahead(f1, f0, e, sa_next, sb_next);
        __builtin_amdgcn_sched_barrier(0);
      });
      uint8_t* const x = here;
      here = there;
      there = x;
      sa = sa_next;
      sb = sb_next;
    };
    const uint32_t whole = TAIL && b1 == blocks ? b1 - 1 : b1;
    for (uint32_t block = b0; block < whole; ++block) run(std::false_type(), block);
    if (TAIL && b1 == blocks) run(std::true_type(), b1 - 1);
    if (EXPERTS) {  // no room to turn in LDS
      const RowOf row = row_of(t.row);
      const uint32_t m0 = row.m0 + wm, n0 = t.col * TN + wn;
      if (m0 < row.end && n0 < N) store_wave<FM, FN, true>(c, acc, m0, row.end, n0, N);
      continue;
    }
    // kTurnRows x 64 results at a time turn in LDS, so that whole lines leave
    const uint32_t m0 = t.row * TM + wm, n0 = t.col * TN + wn;  // of this wave
    if (m0 >= M || n0 >= N) continue;
    uint8_t* const mine = lds + 2 * kBytes + wave * kTurn;
    s2r_mat out = c;
    out.data = static_cast<uint8_t*>(c.data) + t.part * part_bytes;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; j += 2)
#pragma unroll
        for (int h = 0; h < 32 / kTurnRows; ++h) {
          if (kTurnRows == 32 || r / kTurnRows == h) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const f32x16& x = acc[i][j + e / 4];
              const int q = e % 4 * 4;
              *reinterpret_cast<f32x4*>(mine + turned(r % kTurnRows, 2 * e + g)) =
                  f32x4{x[q], x[q + 1], x[q + 2], x[q + 3]};
            }
          }
          __builtin_amdgcn_wave_barrier();
          store_turned<kTurnRows>(out, mine, m0 + i + FM * kTurnRows * h, FM, M, n0 + 32 * j, N);
          __builtin_amdgcn_wave_barrier();
        }
  }
  drain_and_sync();
}

__device__ inline i32x8 load_frag(const uint8_t* row, uint32_t k, uint32_t K) {
  return join(load_codes16(row, k, K), load_codes16(row, k + 64, K));
}

}  // namespace s2r
