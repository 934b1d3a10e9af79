// q4_gemm.hip -- C = A B^T of 4-bit matrices with a power-of-two scale for 32 elements of a row:
//   c[m][n] = sum_k a[m][k] sa[m][k / 32] b[n][k] sb[n][k / 32].
// The scaled matrix instruction takes the codes and the scales as they are stored: a lane's 32 codes
// of a fragment are one block.  Its first operand is B, so that a lane's results are consecutive columns of
// C; one fp32 accumulator runs over the whole sum.  Unlike in 8 bits it cuts nothing that fp32 would hold:
// products of codes are multiples of 1/4 up to 36, and the eight neighbours that it adds first share
// their scales.
//
// Measured on MI355X, 16384 x 8192 x 4096 to bf16: 272 to 298 us by card and values, 3.7 to 4.0 PFLOP/s (a
// library's product of as many 4-bit codes 481, of 8-bit ones 359, of bf16 697); 4.5 with a sum of 8192, 6.0 if all
// codes are zeros.  A chunk of 512 of a 256 x 256 tile takes 3.3 us, 2.6 for zeros, where its matrix
// instructions take 4096 cycles: mostly power.  Results take 9 us a tile, in which all compute units write
// at once: 268 MB, 45 us in all at the rate of a large fill.
#include <algorithm>

#include "q4_device.hpp"
#include "q4_launch.hpp"
#include "q8_tile.hpp"

namespace s2r {

constexpr int kQ4Step = 256;  // elements of the sum in 128 bytes of a row, one block of 8 scales

__device__ inline i32x8 q4_frag(u32x4 v) {
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// 32 codes of a row from k on, those at or beyond K zero.
__device__ inline u32x4 q4_piece(const uint8_t* row, uint32_t k, uint32_t K) {
  u32x4 v = {0, 0, 0, 0};
  if (k < K) v = *reinterpret_cast<const u32x4*>(row + k / 2);
  if (k + 32 > K) {
#pragma unroll
    for (int w = 0; w < 4; ++w) v[w] = q4_keep(v[w], (int)K - (int)k - 8 * w);
  }
  return v;
}

// ---- few rows -----------------------------------------------------------------------------
// 16 rows of A and 16 of B to a workgroup, whose waves take 256 of the sum in turn; the partial sums
// meet in LDS and are added in the order of the waves.
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_q4_gemm_few(s2r_q4_mat a, s2r_q4_mat b, s2r_mat c, uint32_t M,
                                                            uint32_t N, uint32_t K, uint32_t n_tiles) {
  constexpr int kBatch = 2;  // steps of the sum a wave has in flight
  __shared__ f32x4 part[WAVES][64];
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
  const uint32_t n0 = blockIdx.x % n_tiles * 16, m0 = blockIdx.x / n_tiles * 16;
  const uint64_t n = min(n0 + r, N - 1), m = min(m0 + r, M - 1);
  const uint8_t *row_a = a.q + m * a.ld, *row_b = b.q + n * b.ld;
  const uint8_t *scale_a = a.scale + m * a.lds, *scale_b = b.scale + n * b.lds;
  f32x4 acc = {};
  const uint32_t steps = (K + kQ4Step - 1) / kQ4Step;
  for (uint32_t s = wave; s < steps; s += WAVES * kBatch) {
    u32x4 fa[kBatch][2], fb[kBatch][2];
    u32x2 sa[kBatch], sb[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const uint32_t at = s + e * WAVES;
      if (at >= steps) continue;
      sa[e] = *reinterpret_cast<const u32x2*>(scale_a + 8 * at);
      sb[e] = *reinterpret_cast<const u32x2*>(scale_b + 8 * at);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t k = at * kQ4Step + 128 * h + 32 * g;
        fa[e][h] = q4_piece(row_a, k, K), fb[e][h] = q4_piece(row_b, k, K);
      }
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const uint32_t at = s + e * WAVES;
      if (at >= steps) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // codes beyond K are zeros, under whatever scale
        const bool in = at * kQ4Step + 128 * h + 32 * g < K;
        const uint32_t xa = in ? sa[e][h] >> 8 * g : 127, xb = in ? sb[e][h] >> 8 * g : 127;
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q4_frag(fb[e][h]), q4_frag(fa[e][h]), acc, 4, 4, 0,
                                                               (int)xb, 0, (int)xa);
      }
    }
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  f32x4 v = part[0][lane];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) v += part[w][lane];
  if (m0 + r < M && n0 + 4 * g < N) store4(c, m0 + r, n0 + 4 * g, N, v);
}

// ---- tiles --------------------------------------------------------------------------------
// WM x WN waves, each 32 FM rows of A by 32 FN rows of B; a block is 256 of the sum, 128 bytes of
// every row.  LDS holds two blocks of both operands: one is multiplied while the next arrives straight from
// global memory, a whole line of each row.  A block is multiplied in two halves, and the
// fragments of a half are read into registers while the half before is multiplied: its LDS is free again
// after the first half.  Lane group g takes pieces 4 g .. 4 g + 3 of a row, so that its four scales are
// one register.  Scales come by chunks of two blocks, 16 bytes of every row, a chunk ahead: a
// row's scales lie together, and as few as a block's 8 would cost a request for each row as often as
// the codes do.  Sums have an even number of blocks, the last one of zeros where need be.
// A workgroup stays for several tiles, and the blocks of all of them are one stream: the next
// tile's first blocks arrive while the last ones of this are multiplied and its results leave.
constexpr uint32_t kQ4Chunk = 2 * kQ4Step;

template <int AT>
__device__ inline f32x16 q4_mma(u32x4 b, u32x4 a, const f32x16& c, uint32_t sb, uint32_t sa) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(q4_frag(b), q4_frag(a), c, 4, 4, AT, (int)sb, AT, (int)sa);
}

template <int WM, int WN, int FM, int FN, bool TAIL>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_q4_gemm(
    s2r_q4_mat a, s2r_q4_mat b, s2r_mat c, uint64_t part_bytes, uint32_t M, uint32_t N, uint32_t K,
    uint32_t m_tiles, uint32_t n_tiles, uint32_t total, uint32_t part_blocks) {
  constexpr int kWaves = WM * WN, TM = 32 * FM * WM, TN = 32 * FN * WN;
  constexpr int kLoadsA = TM / 8 / kWaves, kLoads = (TM + TN) / 8 / kWaves;
  constexpr int kScaleLoads = ((TM + TN) / 64 + kWaves - 1) / kWaves;
  constexpr int kBytes = (TM + TN) * 128, kScaleBytes = kWaves * kScaleLoads * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kBytes + 2 * kScaleBytes];
  uint8_t* const scales = lds + 2 * kBytes;

  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, r = lane % 32, g = lane / 32;
  const uint32_t wm = wave / WN * (32 * FM), wn = wave % WN * (32 * FN);
  const uint32_t blocks = (K + kQ4Chunk - 1) / kQ4Chunk * 2;

  // Where this lane's pieces of a block come from, relative to the tile's first row: load j takes 8 rows, of which
  // those of j % 4 = 2, 3 are spread differently.  The rest is added at each load: 16 offsets would
  // not fit the registers.
  auto from_of = [&](int j, uint32_t ld, int loads) {
    const uint32_t p = (wave * loads + j) * 8 + lane / 8;
    return p * ld + (lane % 8 ^ spread(p)) * 16;
  };
  static_assert(kLoadsA % 4 == 0 && (kLoads - kLoadsA) % 4 == 0, "");
  const uint32_t from_a[2] = {from_of(0, (uint32_t)a.ld, kLoadsA), from_of(2, (uint32_t)a.ld, kLoadsA)};
  const uint32_t from_b[2] = {from_of(0, (uint32_t)b.ld, kLoads - kLoadsA), from_of(2, (uint32_t)b.ld, kLoads - kLoadsA)};

  // The stream of blocks: the newest that is loaded, and the first one of the item after its
  // own.  The views end with the last row's last 16-byte piece and its last 8 scales.
  const uint32_t row_end = (K + 31) / 32 * 16, scale_end = (K + 255) / 256 * 8;
  struct At {
    uint32_t item, left;  // blocks of the item after this one
    uint64_t a, b, scale_a, scale_b;
    int len_a, len_b, len_sa, len_sb;  // cut at 1.5 2^30: a tile's rows span less than 2^30 and 2^22 bytes
  };
  // 64-bit products and comparisons run in vector registers: back to scalar ones
  auto uniform = [](uint64_t x) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(x >> 32)) << 32 |
           (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)x);
  };
  auto cut = [](uint64_t len) { return (int)__builtin_amdgcn_readfirstlane(len > 0x60000000ull ? 0x60000000u : (uint32_t)len); };
  auto start_of = [&](uint32_t item) {
    At x = {};
    x.item = item;
    x.left = ~0u;  // nothing more: loads of zeros
    if (item >= total) return x;
    const TileAt t = tile_at(item, m_tiles, n_tiles, total);
    const uint32_t m0 = t.row * TM, n0 = t.col * TN, block = t.part * part_blocks;
    const uint64_t k = (uint64_t)block * 128, ks = (uint64_t)block * 8;
    x.left = __builtin_amdgcn_readfirstlane(min(block + part_blocks, blocks) - block - 1);
    x.a = uniform((uint64_t)a.q + (uint64_t)m0 * a.ld + k);
    x.b = uniform((uint64_t)b.q + (uint64_t)n0 * b.ld + k);
    x.scale_a = uniform((uint64_t)a.scale + (uint64_t)m0 * a.lds + ks);
    x.scale_b = uniform((uint64_t)b.scale + (uint64_t)n0 * b.lds + ks);
    x.len_a = cut((uint64_t)(M - m0 - 1) * a.ld + row_end - k);
    x.len_b = cut((uint64_t)(N - n0 - 1) * b.ld + row_end - k);
    x.len_sa = cut((uint64_t)(M - m0 - 1) * a.lds + scale_end - ks);
    x.len_sb = cut((uint64_t)(N - n0 - 1) * b.lds + scale_end - ks);
    return x;
  };
  At in = {}, after = {};
  auto less = [](int len, int by) { return max(len - by, 0); };
  // Without a branch and in nine steps, for it runs between matrix instructions: one of them covers few
  // scalar instructions.
  bool go = false, on = false;
  auto advance = [&](int step) {
    switch (step) {
      case 0:
        in.left = __builtin_amdgcn_readfirstlane(in.left);
        go = in.left == 0, on = in.left + 1 > 1;
        in.item = go ? after.item : in.item;
        break;
      case 1: in.a = go ? after.a : in.a + 128; break;
      case 2: in.len_a = go ? after.len_a : on ? less(in.len_a, 128) : 0; break;
      case 3: in.b = go ? after.b : in.b + 128; break;
      case 4: in.len_b = go ? after.len_b : on ? less(in.len_b, 128) : 0; break;
      case 5: in.scale_a = go ? after.scale_a : in.scale_a + 8; break;
      case 6: in.len_sa = go ? after.len_sa : on ? less(in.len_sa, 8) : 0; break;
      case 7: in.scale_b = go ? after.scale_b : in.scale_b + 8; break;
      case 8:
        in.len_sb = go ? after.len_sb : on ? less(in.len_sb, 8) : 0;
        in.left = go ? after.left : on ? in.left - 1 : ~0u;
        break;
    }
  };
  struct Views {
    __amdgpu_buffer_rsrc_t a, b;
  };
  // rsrc_of's 64-bit comparison would take the whole stream to vector registers
  auto view = [](uint64_t base, int len) {
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, len, 0x00020000);
  };
  auto views = [&] { return Views{view(in.a, in.len_a), view(in.b, in.len_b)}; };
  auto load = [&](uint8_t* to, const Views& v, int j) {
    const bool is_a = j < kLoadsA;
    const int i = is_a ? j : j - kLoadsA;
    uint32_t ld = (uint32_t)(is_a ? a.ld : b.ld) * 8;
    asm volatile("" : "+s"(ld));  // not moved out of the loop
    const uint32_t from = (is_a ? from_a : from_b)[i / 2 % 2] + (i - i / 2 % 2 * 2) * ld;
    if (is_a) load_to_lds(v.a, to + (wave * kLoadsA + i) * 1024, from);
    else load_to_lds(v.b, to + TM * 128 + (wave * (kLoads - kLoadsA) + i) * 1024, from);
  };
  // the chunk that begins with block `in`: 64 rows to a load, also beyond B's where there are too few
  auto load_scales = [&](uint8_t* to) {
#pragma unroll
    for (int j = 0; j < kScaleLoads; ++j) {
      const uint32_t p = (wave * kScaleLoads + j) * 64;
      const bool is_a = p < TM;
      const auto v = view(is_a ? in.scale_a : in.scale_b, is_a ? in.len_sa : in.len_sb);
      load_to_lds(v, to + p * 16, ((is_a ? p : p - TM) + lane) * (uint32_t)(is_a ? a.lds : b.lds));
    }
  };

  struct Frags {
    u32x4 a[2][FM], b[2][FN];
  };
  uint32_t at[2][2];  // where in a fragment's rows this lane's pieces of a half lie
#pragma unroll
  for (int h = 0; h < 4; ++h) at[h / 2][h % 2] = r * 128 + ((4 * g + h) ^ spread(r)) * 16;
  auto row_of = [&](int i) { return i < FN ? TM + wn + 32 * i : wm + 32 * (i - FN); };
  // read e of a half's 2 (FM + FN)
  auto read = [&](Frags& f, const uint8_t* from_lds, int h, int e) {
    const int i = e / 2;
    const u32x4 v = *reinterpret_cast<const u32x4*>(from_lds + row_of(i) * 128 + at[h][e % 2]);
    (i < FN ? f.b[e % 2][i] : f.a[e % 2][i - FN]) = v;
  };
  struct Scales {
    uint32_t of[FN + FM];
  };
  const uint32_t scale_at = r * 16 + g * 4;
  auto read_scale = [&](Scales& s, const uint8_t* chunk, uint32_t odd, int i) {
    s.of[i] = *reinterpret_cast<const uint32_t*>(chunk + row_of(i) * 16 + scale_at + odd * 8);
  };
  auto clear_tail = [&](Frags& f, int h, int left) {  // codes at or beyond K
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int l = left - 32 * (int)(4 * g + 2 * h + t) - 8 * w;
#pragma unroll
        for (int i = 0; i < FM; ++i) f.a[t][i][w] = q4_keep(f.a[t][i][w], l);
#pragma unroll
        for (int j = 0; j < FN; ++j) f.b[t][j][w] = q4_keep(f.b[t][j][w], l);
      }
  };
  auto clear_scales = [&](Scales& s, int left) {  // scales of blocks at or beyond K: 1, whatever is there
    const int n = (left + 31) / 32 - 4 * (int)g;
    const uint32_t keep = n <= 0 ? 0 : n < 4 ? (1u << (8 * n)) - 1 : ~0u;
#pragma unroll
    for (int i = 0; i < FN + FM; ++i) s.of[i] = (s.of[i] & keep) | (0x7f7f7f7fu & ~keep);
  };
  constexpr int kMma = FM * FN, kReads = 2 * (FM + FN), kSlots = 2 * kMma;
  constexpr int kRead = kSlots * 5 / 16, kEarly = kLoads * 5 / 8;

  uint8_t *here = lds, *there = lds + kBytes;
  uint32_t chunk = 0;  // where the scales of the blocks that are multiplied lie
  Frags f0, f1;
  Scales s, s_next;
  if (blocks > 0) {
    in = start_of(blockIdx.x);
    after = start_of(blockIdx.x + gridDim.x);
    load_scales(scales);
    Views v = views();
#pragma unroll
    for (int j = 0; j < kLoads; ++j) load(here, v, j);
#pragma unroll
    for (int step = 0; step < 9; ++step) advance(step);
    v = views();
#pragma unroll
    for (int j = 0; j < kLoads; ++j) load(there, v, j);
    sync_but<kLoads>();
#pragma unroll
    for (int e = 0; e < kReads; ++e) read(f0, here, 0, e);
#pragma unroll
    for (int i = 0; i < FN + FM; ++i) read_scale(s, scales, 0, i);
  }

  for (uint32_t item = blockIdx.x; item < total; item += gridDim.x) {
    const TileAt t = tile_at(item, m_tiles, n_tiles, total);
    const uint32_t b0 = t.part * part_blocks, b1 = min(b0 + part_blocks, blocks);
    after = start_of(in.item + gridDim.x);
    f32x16 acc[FM][FN] = {};
    auto multiply = [&](const Frags& f, auto half, auto slot) {
      constexpr int kHalf = half, kT = slot / kMma, kI = slot % kMma / FN, kJ = slot % FN;
      acc[kI][kJ] = q4_mma<2 * kHalf + kT>(f.b[kT][kJ], f.a[kT][kI], acc[kI][kJ], s.of[kJ], s.of[FN + kI]);
    };
    // the first or the second block of a chunk, without the codes at or beyond K
    auto run = [&](auto clear, auto odd, uint32_t block) {
      const std::integral_constant<int, 0> first;
      const std::integral_constant<int, 1> second;
      const int left = (int)K - (int)(block * kQ4Step);
      if (clear) {
        clear_scales(s, left);
        clear_tail(f0, 0, left);
      }
      each<0, kRead>([&](auto e) {
        multiply(f0, first, e);
#pragma unroll
        for (int q = e * kReads / kRead; q < (e + 1) * kReads / kRead; ++q) read(f1, here, 1, q);
#pragma unroll
        for (int step = e * 9 / kRead; step < (e + 1) * 9 / kRead; ++step) advance(step);
        __builtin_amdgcn_sched_barrier(0);
      });
      multiply(f0, first, std::integral_constant<int, kRead>());
      sync_reads();  // this block's LDS is free
      const Views v = views();
      each<kRead + 1, kSlots>([&](auto e) {
        constexpr int kAt = e - kRead - 1, kOf = kSlots - kRead - 1;
        multiply(f0, first, e);
#pragma unroll
        for (int q = kAt * kEarly / kOf; q < (kAt + 1) * kEarly / kOf; ++q) load(here, v, q);
        __builtin_amdgcn_sched_barrier(0);
      });
      sync_but<kEarly>();  // the next block is there, and its scales
      if (clear) clear_tail(f1, 1, left);
      const uint8_t* const chunk_next = scales + (odd ? chunk ^ 1 : chunk) * kScaleBytes;
      each<0, kSlots>([&](auto e) {
        multiply(f1, second, e);
        constexpr int kReadEnd = kSlots * 3 / 4;
#pragma unroll
        for (int q = e * kReads / kReadEnd; q < lesser((e + 1) * kReads / kReadEnd, kReads); ++q) read(f0, there, 0, q);
#pragma unroll
        for (int q = e * (FM + FN) / kSlots; q < (e + 1) * (FM + FN) / kSlots; ++q) read_scale(s_next, chunk_next, odd ? 0 : 1, q);
        if (kEarly + e < kLoads) load(here, v, kEarly + e);
        if (e == kLoads - kEarly && !odd) load_scales(scales + (chunk ^ 1) * kScaleBytes);
        __builtin_amdgcn_sched_barrier(0);
      });
      uint8_t* const x = here;
      here = there;
      there = x;
      if (odd) chunk ^= 1;
      s = s_next;
    };
    const uint32_t whole = TAIL ? min(b1, K / kQ4Chunk * 2) : b1;
    for (uint32_t block = b0; block < whole; block += 2) {
      run(std::false_type(), std::false_type(), block);
      run(std::false_type(), std::true_type(), block + 1);
    }
    if (TAIL && whole < b1) {
      run(std::true_type(), std::false_type(), whole);
      run(std::true_type(), std::true_type(), whole + 1);
    }
    const uint32_t m0 = t.row * TM + wm, n0 = t.col * TN + wn;  // of this wave
    if (m0 >= M || n0 >= N) continue;
    s2r_mat out = c;
    out.data = static_cast<uint8_t*>(c.data) + t.part * part_bytes;
    store_wave(out, acc, m0, M, n0, N);
  }
  drain_and_sync();
}

// The parts of a sum, added in their order.
constexpr int kQ4SumThreads = 256;
__global__ __launch_bounds__(kQ4SumThreads) void k_q4_gemm_sum(const float* __restrict__ part,
                                                               uint64_t part_floats, uint32_t parts,
                                                               s2r_mat c, uint32_t M, uint32_t N) {
  const uint32_t quads = (N + 3) / 4;
  const uint64_t e = (uint64_t)blockIdx.x * kQ4SumThreads + threadIdx.x;
  const uint32_t m = (uint32_t)(e / quads), n = (uint32_t)(e % quads) * 4;
  if (m >= M) return;
  const float* p = part + (uint64_t)m * (4 * quads) + n;
  f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll 4
  for (uint32_t i = 1; i < parts; ++i) v += *reinterpret_cast<const f32x4*>(p + i * part_floats);
  store4(c, m, n, N, v);
}

namespace {

// Tiles and parts of the sum with the least estimated time, in nanoseconds: of 256 x 256 a compute unit takes one,
// 3400 for a chunk of the sum and 12000 to begin and to leave (results leave all compute units at once); of 128 x
// 128 it takes one in 1380 and 3500 or two beside each other in 2520 and 4400.  Parts are written and read again,
// at 4 bytes a picosecond, by a launch of 3000.  Measured, tiles of 256 and of 128: 4096 x 4096 x 4096 41 us and
// 51, 5001 x 1000 x 4100 39 and 29, 2048 x 2048 x 4096 28 and 16; tiles of 256 x 128 were best nowhere.
struct Q4Plan {
  uint32_t side, mt, nt, chunks;
  Cut cut;  // in chunks
};
Q4Plan q4_plan(uint64_t M, uint64_t N, uint64_t K) {
  const uint32_t chunks = (uint32_t)((K + kQ4Chunk - 1) / kQ4Chunk);
  Q4Plan best = {};
  uint64_t least = ~0ull;
  for (const uint32_t side : {256u, 128u}) {
    Q4Plan p = {side, (uint32_t)((M + side - 1) / side), (uint32_t)((N + side - 1) / side), chunks, {1, chunks}};
    const uint64_t tiles = (uint64_t)p.mt * p.nt;
    for (uint32_t parts = 1; parts <= 16; ++parts) {
      p.cut = cut_evenly(chunks, parts);
      const uint64_t all = tiles * parts, each = p.cut.blocks;
      if (parts > 1 && (p.cut.parts != parts || all > kTileCus)) continue;
      uint64_t ns = side == 256         ? (all + kTileCus - 1) / kTileCus * (each * 3400 + 12000)
                    : all <= kTileCus ? each * 1380 + 3500
                                        : (all + 2 * kTileCus - 1) / (2 * kTileCus) * (each * 2520 + 4400);
      if (parts > 1) ns += 3000 + M * N * 4 * (2 * parts + 1) / 4000;
      if (ns < least) least = ns, best = p;
    }
  }
  return best;
}

// 33 x 4096 x 4096 takes 9.5 us as few rows and 10.2 in tiles, 64 13.0 and 11.1.
bool q4_few_rows(uint64_t M) { return M <= 32; }

}  // namespace

size_t q4_gemm_workspace(uint64_t M, uint64_t N, uint64_t K) {
  if (q4_few_rows(M)) return 0;
  const uint32_t parts = q4_plan(M, N, K).cut.parts;
  return parts > 1 ? parts * M * ((N + 3) / 4 * 4) * sizeof(float) : 0;
}

hipError_t launch_q4_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q4_mat& a, const s2r_q4_mat& b,
                          const s2r_mat& c, void* workspace, hipStream_t s) {
  const uint32_t m = (uint32_t)M, n = (uint32_t)N, k = (uint32_t)K;
  if (q4_few_rows(M)) {
    const uint32_t nt = (n + 15) / 16;
    trace_mark(s, "k_q4_gemm_few");
    hipLaunchKernelGGL((k_q4_gemm_few<8>), dim3(nt * ((m + 15) / 16)), dim3(512), 0, s, a, b, c, m, n, k, nt);
    return hipGetLastError();
  }
  Q4Plan p = q4_plan(M, N, K);
  if (!workspace) p.cut = {1, p.chunks};
  const bool cut = p.cut.parts > 1;
  s2r_mat out = c;
  if (cut) out = {workspace, (N + 3) / 4 * 4, S2R_F32};
  const uint64_t part_bytes = M * out.ld * sizeof(float);
  const uint32_t total = p.mt * p.nt * p.cut.parts;
  const dim3 grid(std::min(total, p.side == 128 ? 2 * kTileCus : kTileCus));
#define S2R_TILE(F, TAIL)                                                                                      \
  hipLaunchKernelGGL((k_q4_gemm<2, 2, F, F, TAIL>), grid, dim3(256), 0, s, a, b, out, part_bytes, m, n, k, p.mt, \
                     p.nt, total, 2 * p.cut.blocks)
  trace_mark(s, p.side == 256 ? "k_q4_gemm<256>" : "k_q4_gemm<128>");
  const bool tail = k % kQ4Chunk != 0;
  if (p.side == 256 && tail) S2R_TILE(4, true);
  else if (p.side == 256) S2R_TILE(4, false);
  else if (tail) S2R_TILE(2, true);
  else S2R_TILE(2, false);
#undef S2R_TILE
  if (cut) {
    trace_mark(s, "k_q4_gemm_sum");
    const uint64_t quads = M * ((N + 3) / 4);
    hipLaunchKernelGGL(k_q4_gemm_sum, dim3((uint32_t)((quads + kQ4SumThreads - 1) / kQ4SumThreads)), dim3(kQ4SumThreads),
                       0, s, static_cast<const float*>(workspace), part_bytes / 4, p.cut.parts, c, m, n);
  }
  return hipGetLastError();
}

}  // namespace s2r
