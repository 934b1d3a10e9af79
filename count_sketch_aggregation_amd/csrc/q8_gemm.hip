// q8_gemm.hip -- C = A B^T of 8-bit matrices with a power-of-two scale for each block of 128:
//   c[m][n] = sum_k a[m][k] sa[k / 128][m] b[n][k] sb[k / 128][n / 128].
// The scaled matrix instruction multiplies both operands by their scales itself, so one fp32
// accumulator runs over the whole sum.  The first operand is B, so that a lane's four results
// are consecutive columns of C.
#include "q8_device.hpp"
#include "q8_launch.hpp"

namespace s2r {

constexpr int kGemmThreads = 256;  // 4 waves, each 32 x 32 of a 64 x 64 tile

__device__ inline i32x8 load_frag(const uint8_t* row, uint32_t k, uint32_t K) {
  const u32x4 lo = load_codes16(row, k, K), hi = load_codes16(row, k + 16, K);
  i32x8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = (int)lo[i];
    v[4 + i] = (int)hi[i];
  }
  return v;
}

template <int FA, int FB>
__global__ __launch_bounds__(kGemmThreads) void k_q8_gemm(s2r_q8_mat a, s2r_q8_mat b, s2r_mat c,
                                                          uint32_t M, uint32_t N, uint32_t K,
                                                          uint32_t n_tiles) {
  const uint32_t wave = threadIdx.x / 64, r = threadIdx.x % 16, g = threadIdx.x % 64 / 16;
  const uint32_t m0 = blockIdx.x / n_tiles * 64 + wave / 2 * 32;
  const uint32_t n0 = blockIdx.x % n_tiles * 64 + wave % 2 * 32;
  f32x4 acc[2][2] = {};
  for (uint32_t k = 0; k < K; k += kQ8Block) {
    i32x8 fa[2], fb[2];
    uint32_t sa[2], sb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t m = min(m0 + 16 * i + r, M - 1), n = min(n0 + 16 * i + r, N - 1);
      fa[i] = load_frag(a.q + (uint64_t)m * a.ld, k + 32 * g, K);
      fb[i] = load_frag(b.q + (uint64_t)n * b.ld, k + 32 * g, K);
      sa[i] = a.scale[(uint64_t)(k / kQ8Block) * a.lds + m];
      sb[i] = b.scale[(uint64_t)(k / kQ8Block) * b.lds + n / kQ8Block];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            fb[j], fa[i], acc[i][j], FB, FA, 0, (int)sb[j], 0, (int)sa[i]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t m = m0 + 16 * i + r;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t n = n0 + 16 * j + 4 * g + t;
        if (m >= M || n >= N) continue;
        const uint64_t at = (uint64_t)m * c.ld + n;
        if (c.dtype == S2R_F32) static_cast<float*>(c.data)[at] = acc[i][j][t];
        else if (c.dtype == S2R_BF16)
          static_cast<uint16_t*>(c.data)[at] = (uint16_t)pack2<S2R_BF16>(acc[i][j][t], 0.f);
        else static_cast<uint16_t*>(c.data)[at] = (uint16_t)pack2<S2R_F16>(acc[i][j][t], 0.f);
      }
    }
}

size_t q8_gemm_workspace(uint64_t, uint64_t, uint64_t) { return 0; }

hipError_t launch_q8_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q8_mat& a,
                          const s2r_q8_mat& b, const s2r_mat& c, void*, hipStream_t s) {
  const uint64_t nt = (N + 63) / 64, mt = (M + 63) / 64;
  trace_mark(s, "k_q8_gemm");
#define S2R_GEMM(FA, FB)                                                                  \
  hipLaunchKernelGGL((k_q8_gemm<FA, FB>), dim3((uint32_t)(nt * mt)), dim3(kGemmThreads), 0, s, \
                     a, b, c, (uint32_t)M, (uint32_t)N, (uint32_t)K, (uint32_t)nt)
  if (a.format == S2R_E4M3) {
    if (b.format == S2R_E4M3) S2R_GEMM(S2R_E4M3, S2R_E4M3);
    else S2R_GEMM(S2R_E4M3, S2R_E5M2);
  } else {
    if (b.format == S2R_E4M3) S2R_GEMM(S2R_E5M2, S2R_E4M3);
    else S2R_GEMM(S2R_E5M2, S2R_E5M2);
  }
#undef S2R_GEMM
  return hipGetLastError();
}

}  // namespace s2r
