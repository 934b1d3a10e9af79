// q4_gemm.hip -- C = A B^T of 4-bit matrices with a power-of-two scale for 32 elements of a row:
//   c[m][n] = sum_k a[m][k] sa[m][k / 32] b[n][k] sb[n][k / 32].
// The scaled matrix instruction takes the codes and the scales as they are stored: a lane's 32 codes
// of a fragment are one block.  Its first operand is B, so that a lane's results are consecutive columns of
// C; one fp32 accumulator runs over the whole sum.
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
  __shared__ f32x4 part[WAVES][64];
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
  const uint32_t n0 = blockIdx.x % n_tiles * 16, m0 = blockIdx.x / n_tiles * 16;
  const uint64_t n = min(n0 + r, N - 1), m = min(m0 + r, M - 1);
  const uint8_t *row_a = a.q + m * a.ld, *row_b = b.q + n * b.ld;
  const uint8_t *scale_a = a.scale + m * a.lds, *scale_b = b.scale + n * b.lds;
  f32x4 acc = {};
  const uint32_t steps = (K + kQ4Step - 1) / kQ4Step;
  for (uint32_t s = wave; s < steps; s += WAVES) {
    const u32x2 sa = *reinterpret_cast<const u32x2*>(scale_a + 8 * s);
    const u32x2 sb = *reinterpret_cast<const u32x2*>(scale_b + 8 * s);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = s * kQ4Step + 128 * h + 32 * g;
      const u32x4 fa = q4_piece(row_a, k, K), fb = q4_piece(row_b, k, K);
      // codes beyond K are zeros, under whatever scale
      const uint32_t xa = k < K ? sa[h] >> 8 * g : 127, xb = k < K ? sb[h] >> 8 * g : 127;
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q4_frag(fb), q4_frag(fa), acc, 4, 4, 0, (int)xb, 0,
                                                             (int)xa);
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

size_t q4_gemm_workspace(uint64_t M, uint64_t N, uint64_t K) { return 0; }

hipError_t launch_q4_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q4_mat& a, const s2r_q4_mat& b,
                          const s2r_mat& c, void* workspace, hipStream_t s) {
  const uint64_t nt = (N + 15) / 16;
  trace_mark(s, "k_q4_gemm_few");
  by_rows(M, 16, 2 * nt, [&](uint64_t m, uint64_t rows) {
    const s2r_q4_mat f = from_row(a, m);
    const s2r_mat to = from_row(c, m);
    const dim3 grid((uint32_t)(nt * ((rows + 15) / 16)));
    hipLaunchKernelGGL((k_q4_gemm_few<8>), grid, dim3(512), 0, s, f, b, to, (uint32_t)rows, (uint32_t)N,
                       (uint32_t)K, (uint32_t)nt);
  });
  return hipGetLastError();
}

}  // namespace s2r
