// q8_wgrad.hip -- the weight gradient from an 8-bit checkpoint:
//   dw[n][k] (+)= sum_m dy[m][n] x[m][k],  x[m][k] = code * scale[k / 128][m].
// The checkpoint's scale changes along m, the summed index, so the scaled matrix instruction
// cannot apply it: both operands become bf16, which holds every stored value exactly, and
// the products are summed in fp32 by the bf16 matrix instruction.
//
// Measured on MI355X: 16384 x 4096 x 4096 from bf16 gradients 467 us, 1.18 PFLOP/s, as a library's
// bf16 product of the same layout (464; 347 where the sum's index is the contiguous one), from e5m2
// gradients 453.  Its LDS is
// busy for half of the cycles (read 768, written 512 of about 3400 a block) and zeros run 20%
// faster than random values.
#include <algorithm>

#include "q8_launch.hpp"
#include "q8_tile.hpp"

namespace s2r {

constexpr int kWgradRows = 64;  // rows m of a block of the sum
constexpr int kBf16 = 2;        // kind of an operand that is bf16 already (else its q8 format)

// An operand on its way to LDS, a block of 64 rows x COLS columns at a time, bf16 there: 64-byte
// piece s of row p lies at s ^ (p % 4).  What is bf16 already goes there directly; codes come
// to registers first and are decoded from there.  Rows at or beyond the end give zeros.
template <int KIND, int COLS, int WAVES>
struct Feed {
  static constexpr bool kDirect = KIND == kBf16;
  static constexpr int kRowBytes = 2 * COLS, kBytes = kWgradRows * kRowBytes;
  static constexpr int kSource = kDirect ? kRowBytes : COLS;  // bytes of a row where it comes from
  static constexpr int kLoads = kWgradRows * kSource / 1024 / WAVES, kRows = 1024 / kSource;
  static_assert(kLoads > 0 && kLoads * kRows % 4 == 0, "");

  uint64_t base, left, step;  // the next block: address, bytes to the operand's end, its own bytes
  uint32_t at[kLoads];        // of this lane in each load
  uint32_t wave, row, last;
  const uint8_t* scale;
  uint32_t to;                // LDS place of this lane's first codes
  static constexpr int kUnits = kDirect ? 0 : 4 * kLoads;  // four codes of every lane each
  u32x4 next[kLoads], code[kLoads];  // a block's codes: on their way, and being decoded
  uint32_t next_sb[kLoads], sb[kLoads];
  u32x4 half;

  __device__ void start(const s2r_mat& m, const s2r_q8_mat& q, uint32_t c0, uint32_t cols,
                        uint32_t first, uint32_t end, uint32_t w) {
    const uint32_t lane = threadIdx.x % 64, s = lane % (kSource / 16), r = lane / (kSource / 16);
    const uint32_t ld = kDirect ? (uint32_t)m.ld * 2 : (uint32_t)q.ld;
    const uint64_t skip = kDirect ? 2 * (uint64_t)c0 : c0;
    wave = w;
    base = (kDirect ? (uint64_t)m.data : (uint64_t)q.q) + (uint64_t)first * ld + skip;
    const uint32_t row_end = (cols * (kDirect ? 2 : 1) + 15) / 16 * 16;  // of the last row's last piece
    left = (uint64_t)(end - first - 1) * ld + row_end - skip;
    step = (uint64_t)kWgradRows * ld;
    const uint32_t p0 = wave * (kLoads * kRows) + r;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const uint32_t p = p0 + j * kRows;
      at[j] = p * ld + (kDirect ? (s / 4 ^ p % 4) * 64 + s % 4 * 16 : s * 16);
    }
    if (!kDirect) {
      row = first + p0;
      last = end - 1;
      scale = q.scale + (uint64_t)(min(c0 + 16 * s, cols - 1) / kQ8Block) * q.lds;
      to = p0 * kRowBytes + (s / 2 ^ p0 % 4) * 64 + s % 2 * 32;
    }
  }
  __device__ void advance() {
    base += step;
    left = left > step ? left - step : 0;
  }
  __device__ __amdgpu_buffer_rsrc_t view() const { return rsrc_of(base, left); }
  // The compiler would have every transposing load of LDS wait for every load that is on its
  // way there: it is not told of these, and the loop waits for them itself.  Nothing comes back
  // to a register; m0, the place in LDS, is an input, so that the compiler knows what it holds; the
  // pause covers it and scalar registers that a vector instruction has just written.
  __device__ void load(uint32_t lds, u32x4 v, int j) const {
    const uint32_t to = lds + (wave * kLoads + j) * 1024;
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :: "v"(at[j]), "s"(v), "{m0}"(__builtin_amdgcn_readfirstlane(to)) : "memory");
  }
  __device__ u32x4 words() const {
    const uint32_t n = left > 0xc0000000ull ? 0xc0000000u : (uint32_t)left;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)base),
                 (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(base >> 32) & 0xffffu),
                 (uint32_t)__builtin_amdgcn_readfirstlane(n), 0x00020000u};
  }
  // codes of the next block, with their scales (of a row beyond the end: any finite one, its codes
  // are 0; kWgradRows and kRows are multiples of 4, and so is `first`)
  __device__ void fetch(u32x4 (&c)[kLoads], uint32_t (&b)[kLoads]) {
    const auto v = view();
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      c[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(v, at[j], 0, 0));
      b[j] = *reinterpret_cast<const uint32_t*>(scale + min(row + j * kRows, last) / 4 * 4);
    }
    row += kWgradRows;
    advance();
  }
  __device__ void fetch() { fetch(next, next_sb); }
  __device__ void fetch_first() { fetch(code, sb); }
  __device__ uint32_t own_scale(uint32_t b) const {  // of four rows; a lane's is the same in every block
    return min(b >> row % 4 * 8 & 0xff, 254u) << 23;
  }
  // Half of the lanes decode and write their upper 16 bytes first: together the lanes of a write
  // then meet every bank.
  __device__ bool upper_first() const { return (threadIdx.x / 4 ^ threadIdx.x / 8) % 2; }
  __device__ void put_code(int j, u32x4 c, uint32_t b) {
    const bool swap = upper_first();
    const uint32_t c0 = c[0], c1 = c[1], c2 = c[2], c3 = c[3];
    code[j] = u32x4{swap ? c2 : c0, swap ? c3 : c1, swap ? c0 : c2, swap ? c1 : c3};
    sb[j] = own_scale(b);
  }
  __device__ void settle_first() {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) put_code(j, code[j], sb[j]);
  }
  // The fetched codes become those that are decoded: moved here, where they are known to have
  // come, and not by the compiler further up.
  __device__ void take() {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      u32x4 c;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t x;
        asm volatile("v_mov_b32 %0, %1" : "=v"(x) : "v"(next[j][w]));
        c[w] = x;
      }
      uint32_t b;
      asm volatile("v_mov_b32 %0, %1" : "=v"(b) : "v"(next_sb[j]));
      put_code(j, c, b);
    }
  }
  // unit u decoded
  __device__ void decode(uint8_t* lds, int u) {
    const int j = u / 4, w = u % 4;
    const u32x2 v = to_bf16<KIND == S2R_E5M2 ? S2R_E5M2 : S2R_E4M3>(code[j][w], __uint_as_float(sb[j]));
    half[w % 2 * 2] = v[0];
    half[w % 2 * 2 + 1] = v[1];
    if (w % 2)
      *reinterpret_cast<u32x4*>(lds + to + j * (kRows * kRowBytes) + ((w == 3) != upper_first() ? 16 : 0)) = half;
  }
};

// WM x WN waves, each 32 FM columns n by 32 FN columns k of dw; a block is 64 rows m, summed in
// four steps of 16.  The matrix instruction wants eight rows m of one column in a lane, and
// memory has columns side by side: LDS is read with the transposing load, four rows of 16
// columns to a lane each.  LDS holds two blocks of both operands; the fragments of a step are
// read while the step before is multiplied, so a block's LDS is free before its last step:
// there the block after the next begins to arrive.  Codes come to registers a block before, and
// are decoded all along the next one's steps.
template <int KY, int FX, int WM, int WN, int FM, int FN>
__global__ __launch_bounds__(64 * WM * WN, FM * FN == 16 ? 1 : 2) void k_q8_wgrad(
    s2r_mat dy16, s2r_q8_mat dy8, s2r_q8_mat xq, float* dw, uint64_t lddw, uint64_t part_floats,
    uint32_t M, uint32_t N, uint32_t K, bool accumulate, uint32_t n_tiles, uint32_t k_tiles,
    uint32_t part_rows) {
  constexpr int kWaves = WM * WN, TM = 32 * FM * WM, TN = 32 * FN * WN;
  using Y = Feed<KY, TM, kWaves>;
  using X = Feed<FX, TN, kWaves>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * (Y::kBytes + X::kBytes)];

  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, r = lane % 32, g = lane / 32;
  const TileAt t = tile_at(blockIdx.x, n_tiles, k_tiles, gridDim.x);
  const uint32_t n0 = t.row * TM, k0 = t.col * TN;
  const uint32_t wm = wave / WN * (32 * FM), wn = wave % WN * (32 * FN);
  const uint32_t m0 = t.part * part_rows, m1 = min(m0 + part_rows, M);

  struct Frags {
    bf16x8 y[FM], x[FN];
  };
  // read e of a step's 2 (FM + FN), two for a fragment
  const uint32_t q = lane % 16;
  uint32_t at_y[FM], at_x[FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
    at_y[i] = (8 * g + q / 4) * Y::kRowBytes + ((wm / 32 + i) ^ q / 4) * 64 + lane / 16 % 2 * 32 + q % 4 * 8;
#pragma unroll
  for (int j = 0; j < FN; ++j)
    at_x[j] = (8 * g + q / 4) * X::kRowBytes + ((wn / 32 + j) ^ q / 4) * 64 + lane / 16 % 2 * 32 + q % 4 * 8;
  auto read = [&](Frags& f, const uint8_t* ly, const uint8_t* lx, int step, int e) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const int i = e / 2;
    const uint8_t* p = i < FN ? lx + at_x[i] + (16 * step + e % 2 * 4) * X::kRowBytes
                              : ly + at_y[i - FN] + (16 * step + e % 2 * 4) * Y::kRowBytes;
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    bf16x8& to = i < FN ? f.x[i] : f.y[i - FN];
#pragma unroll
    for (int w = 0; w < 4; ++w) to[e % 2 * 4 + w] = __builtin_bit_cast(__bf16, (short)v[w]);
  };
  constexpr int kMma = FM * FN, kReads = 2 * (FM + FN);
  f32x16 acc[FM][FN] = {};

  if (m0 < m1) {
    Y y;
    X x;
    y.start(dy16, dy8, n0, N, m0, m1, wave);
    x.start(dy16, xq, k0, K, m0, m1, wave);
    constexpr uint32_t kBytes = Y::kBytes + X::kBytes;
    const uint32_t lds_at = (uint32_t)(uintptr_t)(lds_void*)lds;
    uint32_t here = 0, there = kBytes;
    auto load_y = [&](uint32_t to, int e, int of) {  // share e of a block
      const u32x4 v = y.words();
#pragma unroll
      for (int j = e * Y::kLoads / of; j < (e + 1) * Y::kLoads / of; ++j) y.load(lds_at + to, v, j);
    };
    auto fetch = [&] {
      x.fetch();
      if (!Y::kDirect) y.fetch();
    };
    auto take = [&] {
      x.take();
      if (!Y::kDirect) y.take();
    };
    constexpr int kUnits = X::kUnits + Y::kUnits, kSlots = 4 * kMma;
    auto decode = [&](uint32_t to, int first, int end) {
#pragma unroll
      for (int u = first; u < end; ++u) {
        if (u < X::kUnits) x.decode(lds + to + Y::kBytes, u);
        else if (!Y::kDirect) y.decode(lds + to, u - X::kUnits);
      }
    };
    x.fetch_first();
    if (!Y::kDirect) y.fetch_first();
    fetch();
    if (Y::kDirect) {
      load_y(here, 0, 1);
      y.advance();
      load_y(there, 0, 1);
      y.advance();
    }
    drain_and_sync();
    x.settle_first();
    if (!Y::kDirect) y.settle_first();
    decode(here, 0, kUnits);
    take();
    fetch();
    decode(there, 0, kUnits / 4);
    sync_reads();
    Frags f0, f1;
#pragma unroll
    for (int e = 0; e < kReads; ++e) read(f0, lds + here, lds + here + Y::kBytes, 0, e);

    auto multiply = [&](const Frags& f, int e) {
      acc[e / FN][e % FN] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.x[e % FN], f.y[e / FN], acc[e / FN][e % FN], 0, 0, 0);
    };
    // step s of a block: the next one's fragments are read, the next block's codes decoded
    auto step = [&](const Frags& f, Frags& next, int s) {
#pragma unroll
      for (int e = 0; e < kMma; ++e) {
        multiply(f, e);
#pragma unroll
        for (int i = e * kReads / kMma; i < (e + 1) * kReads / kMma; ++i)
          read(next, lds + here, lds + here + Y::kBytes, s + 1, i);
        const int slot = (s + 1) * kMma + e;
        decode(there, slot * kUnits / kSlots, (slot + 1) * kUnits / kSlots);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (uint32_t m = m0; m < m1; m += kWgradRows) {
      step(f0, f1, 0);
      step(f1, f0, 1);
      step(f0, f1, 2);
      drain_and_sync();  // the next block is there, codes are in registers, this LDS is free
      take();
      fetch();
#pragma unroll
      for (int e = 0; e < kMma; ++e) {
        multiply(f1, e);
#pragma unroll
        for (int i = e * kReads / kMma; i < (e + 1) * kReads / kMma; ++i)
          read(f0, lds + there, lds + there + Y::kBytes, 0, i);
        if (Y::kDirect) load_y(here, e, kMma);
        decode(here, e * kUnits / kSlots, (e + 1) * kUnits / kSlots);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (Y::kDirect) y.advance();
      const uint32_t t = here;
      here = there;
      there = t;
    }
  }
  drain_and_sync();

  // Lane (r, g) of a fragment holds column n = r, columns k = 8 (i / 4) + 4 g + i % 4; 32 x 64 at a
  // time turn in LDS, so that whole lines leave.
  constexpr int kTurn = 32 * 64 * 4;
  static_assert(kWaves * kTurn <= (int)sizeof(lds), "");
  uint8_t* const mine = lds + wave * kTurn;
  float* const out = dw + t.part * part_floats;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; j += 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const f32x16& v = acc[i][j + e / 4];
        const int w = e % 4 * 4;
        *reinterpret_cast<f32x4*>(mine + turned(r, 2 * e + g)) = f32x4{v[w], v[w + 1], v[w + 2], v[w + 3]};
      }
      __builtin_amdgcn_wave_barrier();
      add_turned(out, lddw, mine, n0 + wm + 32 * i, N, k0 + wn + 32 * j, K, accumulate);
      __builtin_amdgcn_wave_barrier();
    }
}

// The partial sums of a row, added in their order.
constexpr int kSumThreads = 256;
__global__ __launch_bounds__(kSumThreads) void k_q8_wgrad_sum(const float* __restrict__ part,
                                                              uint64_t part_floats, uint32_t parts,
                                                              float* __restrict__ dw, uint64_t lddw,
                                                              uint32_t N, uint32_t K, bool accumulate) {
  typedef f32x4 __attribute__((aligned(4))) f32x4_a4;
  const uint32_t quads = (K + 3) / 4;
  const uint64_t e = (uint64_t)blockIdx.x * kSumThreads + threadIdx.x;
  const uint32_t n = (uint32_t)(e / quads), k = (uint32_t)(e % quads) * 4;
  if (n >= N) return;
  const float* p = part + (uint64_t)n * (4 * quads) + k;
  f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll 4
  for (uint32_t i = 1; i < parts; ++i) v += *reinterpret_cast<const f32x4*>(p + i * part_floats);
  float* const to = dw + (uint64_t)n * lddw + k;
  if (k + 4 <= K) {
    if (accumulate) v += *reinterpret_cast<const f32x4_a4*>(to);
    *reinterpret_cast<f32x4_a4*>(to) = v;
  } else {
#pragma unroll
    for (uint32_t c = 0; c < 3; ++c)
      if (k + c < K) to[c] = accumulate ? to[c] + v[c] : v[c];
  }
}

namespace {

// Tiles and parts of the sum with the least estimated time, in nanoseconds.  A tile of 256 x 256
// takes 1600 for a block of 64 rows and 9000 to begin and to leave, one of 128 x 128 1100 and 6000
// (loads' latency: two of them on a compute unit take hardly longer than one).  Parts are written and read
// again, at 5 bytes a picosecond, by a launch of 2000.  Measured: 8192 x 2048 x 2048 88 us in tiles
// of 256 and 4 parts, 95 in tiles of 128 and 2; 4096 x 2048 x 2048 60 and 56; 700 x 2000 x 2000 28 in
// 2 parts, 19 in one.
struct WgradPlan {
  uint32_t side, nt, kt;  // of the tiles
  Cut cut;
  uint64_t part_floats;
};
WgradPlan wgrad_plan(uint64_t M, uint64_t N, uint64_t K) {
  static constexpr uint32_t kTiles[][4] = {{256, kTileCus, 1600, 9000}, {128, 2 * kTileCus, 1100, 6000}};
  const uint32_t blocks = (uint32_t)((M + kWgradRows - 1) / kWgradRows);
  const uint64_t part_floats = N * ((K + 3) / 4 * 4);
  WgradPlan best = {};
  uint64_t least = ~0ull;
  for (const auto& t : kTiles) {
    WgradPlan p = {t[0], (uint32_t)((N + t[0] - 1) / t[0]), (uint32_t)((K + t[0] - 1) / t[0]), {1, blocks},
                   part_floats};
    const uint64_t tiles = (uint64_t)p.nt * p.kt;
    for (uint32_t parts = 1; parts <= 64; ++parts) {
      p.cut = cut_evenly(blocks, parts);
      if (parts > 1 && (p.cut.parts != parts || tiles * parts > t[1])) continue;
      const uint64_t rounds = (tiles * parts + t[1] - 1) / t[1];
      uint64_t ns = rounds * ((uint64_t)p.cut.blocks * t[2] + t[3]);
      if (parts > 1) ns += 2000 + part_floats * 4 * (2 * parts + 1) / 5000;
      if (ns < least) least = ns, best = p;
    }
  }
  return best;
}

template <int KY, int FX>
void go_wgrad(uint64_t M, uint64_t N, uint64_t K, const s2r_mat& d, const s2r_q8_mat& q,
              const s2r_q8_mat& x, float* dw, uint64_t lddw, bool accumulate, float* workspace,
              hipStream_t s) {
  WgradPlan p = wgrad_plan(M, N, K);
  if (!workspace) p.cut = {1, (uint32_t)((M + kWgradRows - 1) / kWgradRows)};
  const bool cut = p.cut.parts > 1;
  const uint32_t grid = p.nt * p.kt * p.cut.parts, rows = p.cut.blocks * kWgradRows;
  float* const to = cut ? workspace : dw;
  const uint64_t ld = cut ? (K + 3) / 4 * 4 : lddw;
  const bool add = accumulate && !cut;
  trace_mark(s, "k_q8_wgrad");
  if (p.side == 256)
    hipLaunchKernelGGL((k_q8_wgrad<KY, FX, 2, 4, 4, 2>), dim3(grid), dim3(512), 0, s, d, q, x, to, ld,
                       p.part_floats, (uint32_t)M, (uint32_t)N, (uint32_t)K, add, p.nt, p.kt, rows);
  else
    hipLaunchKernelGGL((k_q8_wgrad<KY, FX, 2, 2, 2, 2>), dim3(grid), dim3(256), 0, s, d, q, x, to, ld,
                       p.part_floats, (uint32_t)M, (uint32_t)N, (uint32_t)K, add, p.nt, p.kt, rows);
  if (!cut) return;
  trace_mark(s, "k_q8_wgrad_sum");
  const uint64_t quads = N * ((K + 3) / 4);
  hipLaunchKernelGGL(k_q8_wgrad_sum, dim3((uint32_t)((quads + kSumThreads - 1) / kSumThreads)),
                     dim3(kSumThreads), 0, s, workspace, p.part_floats, p.cut.parts, dw, lddw,
                     (uint32_t)N, (uint32_t)K, accumulate);
}

}  // namespace

size_t q8_wgrad_workspace(uint64_t M, uint64_t N, uint64_t K) {
  const WgradPlan p = wgrad_plan(M, N, K);
  return p.cut.parts > 1 ? p.cut.parts * p.part_floats * sizeof(float) : 0;
}

hipError_t launch_q8_wgrad(uint64_t M, uint64_t N, uint64_t K, const s2r_mat* dy16,
                           const s2r_q8_mat* dy8, const s2r_q8_mat& x, float* dw, uint64_t lddw,
                           bool accumulate, void* workspace, hipStream_t s) {
  const s2r_mat d = dy16 ? *dy16 : s2r_mat{};
  const s2r_q8_mat q = dy8 ? *dy8 : s2r_q8_mat{};
  float* const ws = static_cast<float*>(workspace);
#define S2R_WGRAD(KY, FX) go_wgrad<KY, FX>(M, N, K, d, q, x, dw, lddw, accumulate, ws, s)
  const int ky = dy16 ? kBf16 : (int)dy8->format;
  if (x.format == S2R_E4M3) {
    if (ky == kBf16) S2R_WGRAD(kBf16, S2R_E4M3);
    else if (ky == S2R_E4M3) S2R_WGRAD(S2R_E4M3, S2R_E4M3);
    else S2R_WGRAD(S2R_E5M2, S2R_E4M3);
  } else {
    if (ky == kBf16) S2R_WGRAD(kBf16, S2R_E5M2);
    else if (ky == S2R_E4M3) S2R_WGRAD(S2R_E4M3, S2R_E5M2);
    else S2R_WGRAD(S2R_E5M2, S2R_E5M2);
  }
#undef S2R_WGRAD
  return hipGetLastError();
}

}  // namespace s2r
