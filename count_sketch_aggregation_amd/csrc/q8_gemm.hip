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

#include "q8_gemm.hpp"
#include "q8_launch.hpp"

namespace s2r {

// ---- few rows -----------------------------------------------------------------------------
// Up to 16 FM rows of A: the rows of B are read once, straight into registers, and bound the
// call.  A workgroup takes 16 of them and cuts the sum among its waves, block by block in
// turn; the partial sums meet in LDS and are added in the order of the waves.
constexpr int kFewBatch = 2;  // blocks of the sum a wave has in flight

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
  hipLaunchKernelGGL((k_q8_gemm<FA, FB, 2, 2, FM, FN, TAIL, WIDE, false>), grid, dim3(256), 0, s, a, b,    \
                     out, part_bytes, m, n, k, p.mt, p.nt, total, p.cut.blocks, ExpertTiles{})
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

}  // namespace s2r
