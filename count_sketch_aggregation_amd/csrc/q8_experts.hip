// q8_experts.hip -- the products of a layer of experts: c[m] = a[m] b_e^T for the rows m of every expert e,
// in one launch, wherever device memory says they are.  Decoded to bf16 and summed in fp32 as
// s2r_q8_gemm does.  Measured on MI355X: 8192 tokens of 4 choices, 16 experts of 4096 x 2048 to bf16 440 us,
// 1.25 PFLOP/s, matrix cores busy for 68% of the cycles (a library's bf16 product of 16384 x 8192 x 4096 reaches 1.58);
// the input gradient of as many rows, transposed weights side by side 449; 16 tokens of 4 choices, 32 experts of 2048 x
// 1024, 17 to 23 of them chosen, 13 us, 2.7 to 3.7 TB/s.
#include <algorithm>

#include "q8_gemm.hpp"

namespace s2r {

// ---- few rows of an expert ------------------------------------------------------------------
// As few rows of one matrix are summed in q8_gemm.hip, with one block of the sum in flight: a workgroup takes 16 NF
// columns of the experts with rows, gridDim.y apart in their order, and all rows of each, 32 at a time, one after
// the other.  So an expert with most of the rows is slow: 1000 tokens of one choice, 64 experts of 2048 x 1024, 39 us, and 99 if
// nine in ten choose the same one.  first and rows are cut at M.
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

// NF: fragments of 16 columns to a workgroup.  Rows go 32 at a time, the upper 16 where there are any.
template <int FA, int FB, int NF, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_q8_gemm_few_experts(s2r_q8_mat a, s2r_q8_mat b, ExpertSteps steps,
                                                                    s2r_mat c, s2r_experts experts, uint32_t M,
                                                                    uint32_t N, uint32_t K) {
  __shared__ f32x4 part[WAVES][2][NF][64];
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
  const uint32_t n0 = blockIdx.x * (16 * NF);
  const uint32_t blocks = (K + kQ8Block - 1) / kQ8Block;
  for (uint32_t nth = blockIdx.y;; nth += gridDim.y) {
    const ExpertRows x = nth_expert(experts, M, nth);
    if (x.expert == ~0u) return;
    const uint8_t* const expert_b = b.q + x.expert * steps.step;
    const uint8_t* const scale_b = b.scale + x.expert * steps.scale_step + n0 / kQ8Block;  // of all 16 NF columns
    static_assert(kQ8Block % (16 * NF) == 0, "");
    for (uint32_t m0 = x.first; m0 < x.end; m0 += 32) {
      const bool two = m0 + 16 < x.end;
      const uint32_t m[2] = {min(m0 + r, x.end - 1), min(m0 + 16 + r, x.end - 1)};
      f32x4 acc[2][NF] = {};
      for (uint32_t s = wave; s < blocks; s += WAVES) {
        const uint32_t k = s * kQ8Block + 16 * g;
        i32x8 fb[NF], fa[2];
        uint32_t sa[2];
#pragma unroll
        for (int f = 0; f < NF; ++f) fb[f] = load_frag(expert_b + (uint64_t)min(n0 + 16 * f + r, N - 1) * b.ld, k, K);
        const uint32_t sb = scale_b[(uint64_t)s * b.lds];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && !two) continue;
          fa[i] = load_frag(a.q + (uint64_t)m[i] * a.ld, k, K);
          sa[i] = a.scale[(uint64_t)s * a.lds + m[i]];
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          bf16x8 wb[NF];
#pragma unroll
          for (int f = 0; f < NF; ++f) wb[f] = widen8<FB>(fb[f], p, sb);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i == 1 && !two) continue;
            const bf16x8 wa = widen8<FA>(fa[i], p, sa[i]);
#pragma unroll
            for (int f = 0; f < NF; ++f) acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[f], wa, acc[i][f], 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f) part[wave][i][f][lane] = acc[i][f];
      __syncthreads();
      for (uint32_t e = threadIdx.x; e < (two ? 2 : 1) * NF * 64; e += 64 * WAVES) {
        const uint32_t i = e / (NF * 64), f = e / 64 % NF, l = e % 64;
        f32x4 v = part[0][i][f][l];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += part[w][i][f][l];
        const uint32_t row = m0 + 16 * i + l % 16, col = n0 + 16 * f + l / 16 * 4;
        if (row < x.end && col < N) store4(c, row, col, N, v);
      }
      __syncthreads();
    }
  }
}

namespace {

// A few rows to an expert are summed as few rows are, more go to tiles; the host knows only how many there are on
// average (M is at most 20 for each: 100 tokens of 4 choices, 32 experts of 2048 x 2048 38 us, 41 in tiles; 200
// tokens 57 and 38; or 64 for each where there would be few tiles: 100 tokens of 2 choices, 8 experts of 1024 x 1024 8.5
// us, 12.3 in tiles; 300 tokens, of 512 x 1024 18.0 and 12.0).
template <int FA, int FB>
void go_gemm_experts(uint64_t M, uint64_t N, uint64_t K, const s2r_experts& e, const s2r_q8_mat& a,
                     const s2r_q8_mat& b, ExpertSteps steps, const s2r_mat& c, hipStream_t s) {
  const uint32_t m = (uint32_t)M, n = (uint32_t)N, k = (uint32_t)K;
  const uint64_t some = std::min<uint64_t>(e.experts, (M + 3) / 4);  // experts with rows are at least 4 rows apart
  auto tiles = [&](uint64_t side) { return (M / side + some) * ((N + side - 1) / side); };
  const uint64_t few = tiles(128) <= kTileCus / 2 ? 64 : 20;
  if (M <= few * e.experts) {
    trace_mark(s, "k_q8_gemm_few_experts");
    const dim3 grid((n + 31) / 32, (uint32_t)some);
    // two workgroups for every compute unit or fewer: more waves each (2 experts of 4096 x 4096, one token: 10 us
    // with 8, 13 with 4; 60 of 2048 x 2048, 64 tokens: 65 and 56)
    if ((uint64_t)grid.x * some <= 2 * kTileCus)
      hipLaunchKernelGGL((k_q8_gemm_few_experts<FA, FB, 2, 8>), grid, dim3(512), 0, s, a, b, steps, c, e, m, n, k);
    else
      hipLaunchKernelGGL((k_q8_gemm_few_experts<FA, FB, 2, 4>), grid, dim3(256), 0, s, a, b, steps, c, e, m, n, k);
    return;
  }
  // Tiles by estimated time, in nanoseconds: of 256 x 256 one to a compute unit, 2700 for a block of the sum and
  // 8000 to begin and to leave; of 128 x 128 two beside each other, 1500 and 4500 (8192 tokens of 4 choices, 16
  // experts of 4096 x 2048: 456 us and 489; 2 choices, 8 of 2048 x 2048: 148 and 130).  As many
  // tiles are reckoned with as there can be, for some experts have many more rows than others (4000 tokens of one
  // choice, 32 experts of 2048 x 1024: 53 and 33).
  const uint32_t blocks = (k + kQ8Block - 1) / kQ8Block;
  auto rounds = [](uint64_t n, uint64_t width) { return (n + width - 1) / width; };
  const bool large = rounds(tiles(256), kTileCus) * (blocks * 2700 + 8000) < rounds(tiles(128), 2 * kTileCus) * (blocks * 1500 + 4500);
  const dim3 grid((uint32_t)(large ? std::min<uint64_t>(tiles(256), kTileCus) : std::min<uint64_t>(tiles(128), 2 * kTileCus)));
#define S2R_TILE(FM, FN, TAIL)                                                                                   \
  hipLaunchKernelGGL((k_q8_gemm<FA, FB, 2, 2, FM, FN, TAIL, true, true>), grid, dim3(256), 0, s, a, b, c, 0, m, n, k, 0, \
                     (n + 64 * FN - 1) / (64 * FN), 0, blocks, ExpertTiles{e, steps})
#define S2R_TILE_TAIL(FM, FN)                          \
  do {                                                 \
    if (k % kQ8Block == 0) S2R_TILE(FM, FN, false);    \
    else S2R_TILE(FM, FN, true);                       \
  } while (0)
  trace_mark(s, "k_q8_gemm_experts");
  if (large) S2R_TILE_TAIL(4, 4);
  else S2R_TILE_TAIL(2, 2);
#undef S2R_TILE_TAIL
#undef S2R_TILE
}

}  // namespace

hipError_t launch_q8_gemm_experts(uint64_t M, uint64_t N, uint64_t K, const s2r_experts& e,
                                  const s2r_q8_mat& a, const s2r_q8_mat& b, ExpertSteps steps,
                                  const s2r_mat& c, hipStream_t s) {
#define S2R_EXPERTS(FA, FB) go_gemm_experts<FA, FB>(M, N, K, e, a, b, steps, c, s)
  if (a.format == S2R_E4M3) {
    if (b.format == S2R_E4M3) S2R_EXPERTS(S2R_E4M3, S2R_E4M3);
    else S2R_EXPERTS(S2R_E4M3, S2R_E5M2);
  } else {
    if (b.format == S2R_E4M3) S2R_EXPERTS(S2R_E5M2, S2R_E4M3);
    else S2R_EXPERTS(S2R_E5M2, S2R_E5M2);
  }
#undef S2R_EXPERTS
  return hipGetLastError();
}

}  // namespace s2r
