// q8_experts.hip -- the products of a layer of experts: c[m] = a[m] b_e^T for the rows m of every expert e,
// in one launch, wherever device memory says they are.  Decoded to bf16 and summed in fp32 as
// s2r_q8_gemm does.
#include <algorithm>

#include "q8_gemm.hpp"

namespace s2r {

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

namespace {

// A few rows to an expert are summed as few rows are; more go to tiles, whose height the average tells
// (how many rows an expert has, the host does not know).
template <int FA, int FB>
void go_gemm_experts(uint64_t M, uint64_t N, uint64_t K, const s2r_experts& e, const s2r_q8_mat& a,
                     const s2r_q8_mat& b, ExpertSteps steps, const s2r_mat& c, hipStream_t s) {
  const uint32_t m = (uint32_t)M, n = (uint32_t)N, k = (uint32_t)K;
  if (M <= 32 * (uint64_t)e.experts) {
    // experts with rows are at least 4 rows apart
    const dim3 grid((n + 15) / 16, (uint32_t)std::min<uint64_t>(e.experts, (M + 3) / 4));
    trace_mark(s, "k_q8_gemm_few_experts");
    hipLaunchKernelGGL((k_q8_gemm_few_experts<FA, FB, 8>), grid, dim3(512), 0, s, a, b, steps, c, e, m, n, k);
    return;
  }
  const uint32_t blocks = (k + kQ8Block - 1) / kQ8Block;
  auto tiles = [&](uint64_t tm, uint64_t tn) { return (M / tm + std::min<uint64_t>(e.experts, M / 4)) * ((N + tn - 1) / tn); };
#define S2R_TILE(FM, FN, TAIL)                                                                                   \
  hipLaunchKernelGGL((k_q8_gemm<FA, FB, 2, 2, FM, FN, TAIL, true, true>),                                        \
                     dim3((uint32_t)std::min<uint64_t>(tiles(64 * FM, 64 * FN), kTileCus)), dim3(256), 0, s, a, b, c, 0, m, \
                     n, k, 0, (n + 64 * FN - 1) / (64 * FN), 0, blocks, ExpertTiles{e, steps})
#define S2R_TILE_TAIL(FM, FN)                          \
  do {                                                 \
    if (k % kQ8Block == 0) S2R_TILE(FM, FN, false);    \
    else S2R_TILE(FM, FN, true);                       \
  } while (0)
  trace_mark(s, "k_q8_gemm_experts");
  if (tiles(256, 256) >= kTileCus && M >= 192 * (uint64_t)e.experts) S2R_TILE_TAIL(4, 4);
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
