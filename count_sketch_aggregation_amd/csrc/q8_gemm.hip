// q8_gemm.hip -- C = A B^T of 8-bit matrices with a power-of-two scale for each block of 128:
//   c[m][n] = sum_k a[m][k] sa[k / 128][m] b[n][k] sb[k / 128][n / 128].
// The first operand of every matrix instruction is B, so that a lane's results are consecutive
// columns of C; one fp32 accumulator runs over the whole sum.
//
// Two ways through the matrix cores.  s2r_q8_gemm and the few-row form, which memory bounds, decode to
// bf16, exact for every stored value, and use the bf16 instruction, whose sums are fp32.
// s2r_q8_gemm_fast gives the codes to the scaled 8-bit instruction, which multiplies both
// operands by their scales itself and runs at twice the rate, but cuts products: of eight
// neighbouring k (aligned to eight) each is cut toward zero at 2^-13 of the largest one's power of two
// before they are added (2^16 - 2^16 + 2^3 gives 2^3, 2^16 - 2^16 + 2^2 gives 0; a subnormal code
// counts as the format's least normal); these sums and the accumulator are added as fp32.  Where
// nothing cancels a 16-bit result hides that (root mean square 2.4e-5 of its size, rounding costs
// 2e-4 in fp16), but a sum that cancels does not, whatever type it is rounded to: so the caller
// chooses.
//
// Measured on MI355X, 16384 x 8192 x 4096 e4m3 to bf16, many passes in turn over three sets of inputs:
// s2r_q8_gemm 763 us, 1.44 PFLOP/s (a library's product of bf16 matrices 704), its matrix cores busy for
// 77% of the cycles; s2r_q8_gemm_fast 429 us, 2.56 PFLOP/s (a library's with one scale for a whole
// matrix 367), 68%.  There a block of the sum of a 256 x 256 tile takes 2400 to 2700 cycles where its
// matrix instructions alone take 2048; zeros run 18% faster than random codes, so the rest is
// mostly power.
#include <algorithm>

#include "moe_launch.hpp"
#include "q8_launch.hpp"
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
template <int FA, int FB, int WM, int WN, int FM, int FN, bool TAIL, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_q8_gemm(
    s2r_q8_mat a, s2r_q8_mat b, s2r_mat c, uint64_t part_bytes, uint32_t M, uint32_t N, uint32_t K,
    uint32_t m_tiles, uint32_t n_tiles, uint32_t total, uint32_t part_blocks) {
  constexpr int kWaves = WM * WN, TM = 32 * FM * WM, TN = 32 * FN * WN;
  constexpr int kLoadsA = TM / 8 / kWaves, kLoads = (TM + TN) / 8 / kWaves;
  constexpr int kBytes = (TM + TN) * kQ8Block;
  static_assert(kLoads - kLoads * 5 / 8 <= FM * FN, "late loads have a slot each");
  constexpr int kTurnRows = kWaves > 4 ? 16 : 32, kTurn = kTurnRows * 64 * 4;  // a wave's results in LDS
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kBytes + kWaves * kTurn];

  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, r = lane % 32, g = lane / 32;
  const uint32_t wm = wave / WN * (32 * FM), wn = wave % WN * (32 * FN);
  const uint32_t blocks = (K + kQ8Block - 1) / kQ8Block;

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
    const uint32_t m0 = t.row * TM, n0 = t.col * TN, block = t.part * part_blocks;
    const uint64_t k = (uint64_t)block * kQ8Block;
    x.left = __builtin_amdgcn_readfirstlane(min(block + part_blocks, blocks) - block - 1);
    x.a = (uint64_t)a.q + (uint64_t)m0 * a.ld + k;
    x.b = (uint64_t)b.q + (uint64_t)n0 * b.ld + k;
    x.len_a = (uint64_t)(M - m0 - 1) * a.ld + row_end - k;
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

// ---- few rows -----------------------------------------------------------------------------
// Up to 16 FM rows of A: the rows of B are read once, straight into registers, and bound the
// call.  A workgroup takes 16 of them and cuts the sum among its waves, block by block in
// turn; the partial sums meet in LDS and are added in the order of the waves.
constexpr int kFewBatch = 2;  // blocks of the sum a wave has in flight

__device__ inline i32x8 load_frag(const uint8_t* row, uint32_t k, uint32_t K) {
  return join(load_codes16(row, k, K), load_codes16(row, k + 64, K));
}

template <int FA, int FB, int FM, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_q8_gemm_few(s2r_q8_mat a, s2r_q8_mat b, s2r_mat c,
                                                            uint32_t M, uint32_t N, uint32_t K) {
  __shared__ f32x4 part[WAVES][FM][64];
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
  const uint32_t n0 = blockIdx.x * 16;
  const uint32_t n = min(n0 + r, N - 1);
  const uint8_t* rows_a[FM];
  uint32_t ms[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    ms[i] = min(16 * i + r, M - 1);
    rows_a[i] = a.q + (uint64_t)ms[i] * a.ld;
  }
  const uint8_t* row_b = b.q + (uint64_t)n * b.ld;
  const uint8_t* scale_b = b.scale + n0 / kQ8Block;
  f32x4 acc[FM] = {};
  const uint32_t steps = (K + kQ8Block - 1) / kQ8Block;
  for (uint32_t s = wave; s < steps; s += WAVES * kFewBatch) {
    i32x8 fb[kFewBatch], fa[kFewBatch][FM];
    uint32_t sb[kFewBatch], sa[kFewBatch][FM];
#pragma unroll
    for (int e = 0; e < kFewBatch; ++e) {
      const uint32_t at = s + e * WAVES, k = at * kQ8Block + 16 * g;  // and 64 further on: lines in whole halves
      if (at >= steps) continue;
      fb[e] = load_frag(row_b, k, K);
      sb[e] = scale_b[(uint64_t)at * b.lds];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        fa[e][i] = load_frag(rows_a[i], k, K);
        sa[e][i] = a.scale[(uint64_t)at * a.lds + ms[i]];
      }
    }
#pragma unroll
    for (int e = 0; e < kFewBatch; ++e) {
      if (s + e * WAVES >= steps) continue;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const bf16x8 wb = widen8<FB>(fb[e], p, sb[e]);
#pragma unroll
        for (int i = 0; i < FM; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, widen8<FA>(fa[e][i], p, sa[e][i]), acc[i], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < FM * 64; e += 64 * WAVES) {
    f32x4 v = part[0][e / 64][e % 64];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += part[w][e / 64][e % 64];
    const uint32_t m = e / 64 * 16 + e % 16, at = n0 + e % 64 / 16 * 4;
    if (m < M) store4(c, m, at, N, v);
  }
}

// ---- few rows of an expert ------------------------------------------------------------------
// The same for the rows of experts, 16 at a time: a workgroup takes 16 columns of the experts with
// rows, gridDim.y apart in their order.  first and rows are cut at M.
struct ExpertRows {
  uint32_t expert, first, end;
};
// The `nth` expert with rows, found by the lanes of every wave; expert ~0 where there are fewer.
__device__ inline ExpertRows nth_expert(const s2r_experts& e, uint32_t M, uint32_t nth) {
  const uint32_t lane = threadIdx.x % 64;
  for (uint32_t base = 0; base < e.experts; base += 64) {
    const bool there = base + lane < e.experts;
    const uint32_t first = there ? min(e.first[base + lane], M) : 0;
    const uint32_t rows = there ? min(e.rows[base + lane], M - first) : 0;
    const uint64_t some = __ballot(rows > 0);
    const uint32_t n = (uint32_t)__popcll(some);
    if (nth < n) {
      const bool is = rows > 0 && (uint32_t)__popcll(some & ((1ull << lane) - 1)) == nth;
      const uint32_t at = (uint32_t)__builtin_ctzll(__ballot(is));
      const uint32_t f = __builtin_amdgcn_readlane(first, at);
      return {base + at, f, f + (uint32_t)__builtin_amdgcn_readlane(rows, at)};
    }
    nth -= n;
  }
  return {~0u, 0, 0};
}

template <int FA, int FB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_q8_gemm_few_experts(s2r_q8_mat a, s2r_q8_mat b, ExpertSteps steps,
                                                                    s2r_mat c, s2r_experts experts, uint32_t M,
                                                                    uint32_t N, uint32_t K) {
  __shared__ f32x4 part[WAVES][64];
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
  const uint32_t n0 = blockIdx.x * 16, n = min(n0 + r, N - 1);
  const uint32_t blocks = (K + kQ8Block - 1) / kQ8Block;
  for (uint32_t nth = blockIdx.y;; nth += gridDim.y) {
    const ExpertRows x = nth_expert(experts, M, nth);
    if (x.expert == ~0u) return;
    const uint8_t* row_b = b.q + x.expert * steps.step + (uint64_t)n * b.ld;
    const uint8_t* scale_b = b.scale + x.expert * steps.scale_step + n0 / kQ8Block;
    for (uint32_t m0 = x.first; m0 < x.end; m0 += 16) {
      const uint32_t m = min(m0 + r, x.end - 1);
      const uint8_t* row_a = a.q + (uint64_t)m * a.ld;
      f32x4 acc = {};
      for (uint32_t s = wave; s < blocks; s += WAVES) {
        const uint32_t k = s * kQ8Block + 16 * g;
        const i32x8 fb = load_frag(row_b, k, K), fa = load_frag(row_a, k, K);
        const uint32_t sb = scale_b[(uint64_t)s * b.lds], sa = a.scale[(uint64_t)s * a.lds + m];
#pragma unroll
        for (int p = 0; p < 4; ++p)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<FB>(fb, p, sb), widen8<FA>(fa, p, sa), acc, 0, 0, 0);
      }
      part[wave][lane] = acc;
      __syncthreads();
      if (wave == 0) {
        f32x4 v = part[0][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += part[w][lane];
        if (m0 + r < x.end && n0 + 4 * g < N) store4(c, m0 + r, n0 + 4 * g, N, v);
      }
      __syncthreads();
    }
  }
}

// The parts of a sum, added in their order.
constexpr int kSumThreads = 256;
__global__ __launch_bounds__(kSumThreads) void k_q8_gemm_sum(const float* __restrict__ part,
                                                             uint64_t part_floats, uint32_t parts,
                                                             s2r_mat c, uint32_t M, uint32_t N) {
  const uint32_t quads = (N + 3) / 4;
  const uint64_t e = (uint64_t)blockIdx.x * kSumThreads + threadIdx.x;
  const uint32_t m = (uint32_t)(e / quads), n = (uint32_t)(e % quads) * 4;
  if (m >= M) return;
  const float* p = part + (uint64_t)m * (4 * quads) + n;
  f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll 4
  for (uint32_t i = 1; i < parts; ++i) v += *reinterpret_cast<const f32x4*>(p + i * part_floats);
  store4(c, m, n, N, v);
}

namespace {

// Tiles and parts of the sum with the least estimated time, in nanoseconds.  A tile of 256 x 256
// takes 1350 for a block of the sum (2700 by way of bf16) and 8000 to begin and to leave, one of
// 256 x 128 900 (1500) and 6000, one of 128 x 128 680 (900) and 5000 (measured at K = 4096 with one
// tile on every compute unit), and the compute units take them in rounds.  Parts are written and read again, at 4
// bytes a picosecond, by a launch of 3000.
struct GemmPlan {
  uint32_t tm, tn, mt, nt, blocks;
  Cut cut;
};
GemmPlan gemm_plan(uint64_t M, uint64_t N, uint64_t K, bool wide) {
  static constexpr uint32_t kTiles[][5] = {
      {256, 256, 1350, 2700, 8000}, {256, 128, 900, 1500, 6000}, {128, 128, 680, 900, 5000}};
  const uint32_t blocks = (uint32_t)((K + kQ8Block - 1) / kQ8Block);
  GemmPlan best = {};
  uint64_t least = ~0ull;
  for (const auto& t : kTiles) {
    GemmPlan p = {t[0], t[1], (uint32_t)((M + t[0] - 1) / t[0]), (uint32_t)((N + t[1] - 1) / t[1]),
                  blocks, {1, blocks}};
    const uint64_t tiles = (uint64_t)p.mt * p.nt;
    for (uint32_t parts = 1; parts <= 16; ++parts) {
      p.cut = cut_evenly(blocks, parts);
      if (parts > 1 && (p.cut.parts != parts || p.cut.blocks < 2 || blocks % p.cut.blocks == 1 ||
                        tiles * parts > kTileCus))
        continue;  // as few parts give the same, or one has a single block beside longer ones
      const uint64_t rounds = (tiles * parts + kTileCus - 1) / kTileCus;
      uint64_t ns = rounds * ((uint64_t)p.cut.blocks * t[wide ? 3 : 2] + t[4]);
      if (parts > 1) ns += 3000 + M * N * 4 * (2 * parts + 1) / 4000;
      if (ns < least) least = ns, best = p;
    }
  }
  return best;
}

// More than 32 rows of A are read so often that a large B is better off in tiles, if their sum can
// be cut: 64 x 8192 x 4096 16.1 us in tiles (13.8 s2r_q8_gemm_fast), 23.7 without, 40 rows 15.3 (12.6)
// and 19.9; 64 x 4096 x 4096 (13.6) and 12.8; 64 x 2000 x 2000 (10.4) and 6.4.
bool few_rows(uint64_t M, uint64_t N, uint64_t K, bool workspace) {
  return M <= 32 || (M <= 64 && (N * K < 1ull << 25 || !workspace));
}

template <int FA, int FB>
void go_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q8_mat& a, const s2r_q8_mat& b,
             const s2r_mat& c, bool fast, void* workspace, hipStream_t s) {
  const uint32_t m = (uint32_t)M, n = (uint32_t)N, k = (uint32_t)K;
  if (few_rows(M, N, K, workspace != nullptr)) {
    trace_mark(s, "k_q8_gemm_few");
    const dim3 grid((n + 15) / 16);
    // One workgroup for every compute unit or fewer: more waves each (4096 rows of B, one of A: 7.0
    // us with 16, 8.3 with 8; 8192 rows: 11.9 and 10.7).
    const bool sparse = grid.x <= kTileCus;
#define S2R_FEW(FM, WAVES) \
  hipLaunchKernelGGL((k_q8_gemm_few<FA, FB, FM, WAVES>), grid, dim3(64 * WAVES), 0, s, a, b, c, m, n, k)
    if (M <= 16) {
      if (sparse) S2R_FEW(1, 16);
      else S2R_FEW(1, 8);
    } else if (M <= 32) {
      S2R_FEW(2, 8);
    } else {
      S2R_FEW(4, 8);
    }
#undef S2R_FEW
    return;
  }
  const bool wide = !fast;
  GemmPlan p = gemm_plan(M, N, K, wide);
  if (!workspace) p.cut = {1, p.blocks};
  const bool cut = p.cut.parts > 1;
  s2r_mat out = c;
  if (cut) out = {workspace, (N + 3) / 4 * 4, S2R_F32};
  const uint64_t part_bytes = M * out.ld * sizeof(float);
  const uint32_t total = p.mt * p.nt * p.cut.parts;
  const dim3 grid(std::min(total, kTileCus));
#define S2R_TILE(FM, FN, TAIL, WIDE)                                                               \
  hipLaunchKernelGGL((k_q8_gemm<FA, FB, 2, 2, FM, FN, TAIL, WIDE>), grid, dim3(256), 0, s, a, b,    \
                     out, part_bytes, m, n, k, p.mt, p.nt, total, p.cut.blocks)
#define S2R_TILE_TAIL(FM, FN, WIDE)                          \
  do {                                                       \
    if (k % kQ8Block == 0) S2R_TILE(FM, FN, false, WIDE);    \
    else S2R_TILE(FM, FN, true, WIDE);                       \
  } while (0)
  trace_mark(s, "k_q8_gemm");
  if (p.tn == 256) {
    if (wide) S2R_TILE_TAIL(4, 4, true);
    else S2R_TILE_TAIL(4, 4, false);
  } else if (p.tm == 256) {
    if (wide) S2R_TILE_TAIL(4, 2, true);
    else S2R_TILE_TAIL(4, 2, false);
  } else {
    if (wide) S2R_TILE_TAIL(2, 2, true);
    else S2R_TILE_TAIL(2, 2, false);
  }
#undef S2R_TILE_TAIL
#undef S2R_TILE
  if (!cut) return;
  trace_mark(s, "k_q8_gemm_sum");
  const uint64_t quads = M * ((N + 3) / 4);
  hipLaunchKernelGGL(k_q8_gemm_sum, dim3((uint32_t)((quads + kSumThreads - 1) / kSumThreads)),
                     dim3(kSumThreads), 0, s, static_cast<const float*>(workspace), part_bytes / 4,
                     p.cut.parts, c, m, n);
}

}  // namespace

size_t q8_gemm_workspace(uint64_t M, uint64_t N, uint64_t K) {
  if (few_rows(M, N, K, true)) return 0;
  // for s2r_q8_gemm and s2r_q8_gemm_fast
  const uint32_t parts = std::max(gemm_plan(M, N, K, false).cut.parts, gemm_plan(M, N, K, true).cut.parts);
  return parts > 1 ? parts * M * ((N + 3) / 4 * 4) * sizeof(float) : 0;
}

hipError_t launch_q8_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q8_mat& a,
                          const s2r_q8_mat& b, const s2r_mat& c, bool fast, void* workspace,
                          hipStream_t s) {
  if (a.format == S2R_E4M3) {
    if (b.format == S2R_E4M3) go_gemm<S2R_E4M3, S2R_E4M3>(M, N, K, a, b, c, fast, workspace, s);
    else go_gemm<S2R_E4M3, S2R_E5M2>(M, N, K, a, b, c, fast, workspace, s);
  } else {
    if (b.format == S2R_E4M3) go_gemm<S2R_E5M2, S2R_E4M3>(M, N, K, a, b, c, fast, workspace, s);
    else go_gemm<S2R_E5M2, S2R_E5M2>(M, N, K, a, b, c, fast, workspace, s);
  }
  return hipGetLastError();
}

hipError_t launch_q8_gemm_experts(uint64_t M, uint64_t N, uint64_t K, const s2r_experts& e,
                                  const s2r_q8_mat& a, const s2r_q8_mat& b, ExpertSteps steps,
                                  const s2r_mat& c, hipStream_t s) {
  // experts with rows are at least 4 rows apart
  const dim3 grid((uint32_t)((N + 15) / 16), (uint32_t)std::min<uint64_t>(e.experts, (M + 3) / 4));
  trace_mark(s, "k_q8_gemm_few_experts");
#define S2R_FEW(FA, FB)                                                                                  \
  hipLaunchKernelGGL((k_q8_gemm_few_experts<FA, FB, 8>), grid, dim3(512), 0, s, a, b, steps, c, e, (uint32_t)M, \
                     (uint32_t)N, (uint32_t)K)
  if (a.format == S2R_E4M3) {
    if (b.format == S2R_E4M3) S2R_FEW(S2R_E4M3, S2R_E4M3);
    else S2R_FEW(S2R_E4M3, S2R_E5M2);
  } else {
    if (b.format == S2R_E4M3) S2R_FEW(S2R_E5M2, S2R_E4M3);
    else S2R_FEW(S2R_E5M2, S2R_E5M2);
  }
#undef S2R_FEW
  return hipGetLastError();
}

}  // namespace s2r
