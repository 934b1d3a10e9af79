// q8_wgrad.hip -- the weight gradient from an 8-bit checkpoint:
//   dw[n][k] (+)= sum_m dy[m][n] x[m][k],  x[m][k] = code * scale[k / 128][m].
// The checkpoint's scale changes along m, the summed index, so the scaled matrix instruction
// cannot apply it: both operands become bf16, which holds every stored value exactly, and
// the products are summed in fp32 by the bf16 matrix instruction.
#include "q8_device.hpp"
#include "q8_launch.hpp"

namespace s2r {

constexpr int kWgradThreads = 256;  // 4 waves, each 32 x 32 of a 64 x 64 tile

// element (m, c) of an operand as bf16 bits; zero at or beyond M
template <int KIND>  // 0, 1: row-block codes of that format; 2: bf16
__device__ inline uint16_t wgrad_elem(const s2r_mat& d, const s2r_q8_mat& q, uint32_t m, uint32_t c,
                                      uint32_t M) {
  if (m >= M) return 0;
  if (KIND == 2) return static_cast<const uint16_t*>(d.data)[(uint64_t)m * d.ld + c];
  const int code = q.q[(uint64_t)m * q.ld + c];
  const float s = scale_value(q.scale[(uint64_t)(c / kQ8Block) * q.lds + m]);
  const float v = (KIND == S2R_E4M3 ? __builtin_amdgcn_cvt_f32_fp8(code, 0)
                                    : __builtin_amdgcn_cvt_f32_bf8(code, 0)) * s;
  return (uint16_t)(__float_as_uint(v) >> 16);  // exact
}

template <int KY, int FX>
__global__ __launch_bounds__(kWgradThreads) void k_q8_wgrad(s2r_mat dy16, s2r_q8_mat dy8,
                                                            s2r_q8_mat x, float* dw, uint64_t lddw,
                                                            uint32_t M, uint32_t N, uint32_t K,
                                                            bool accumulate, uint32_t k_tiles) {
  const uint32_t wave = threadIdx.x / 64, r = threadIdx.x % 16, g = threadIdx.x % 64 / 16;
  const uint32_t n0 = blockIdx.x / k_tiles * 64 + wave / 2 * 32;
  const uint32_t k0 = blockIdx.x % k_tiles * 64 + wave % 2 * 32;
  f32x4 acc[2][2] = {};
  for (uint32_t m = 0; m < M; m += 32) {
    bf16x8 fy[2], fx[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t n = min(n0 + 16 * i + r, N - 1), k = min(k0 + 16 * i + r, K - 1);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t mm = m + 8 * g + e;
        fy[i][e] = __builtin_bit_cast(__bf16, wgrad_elem<KY>(dy16, dy8, mm, n, M));
        fx[i][e] = __builtin_bit_cast(__bf16, wgrad_elem<FX>(dy16, x, mm, k, M));
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[j], fy[i], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t n = n0 + 16 * i + r;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t k = k0 + 16 * j + 4 * g + t;
        if (n >= N || k >= K) continue;
        float* at = dw + (uint64_t)n * lddw + k;
        *at = accumulate ? *at + acc[i][j][t] : acc[i][j][t];
      }
    }
}

size_t q8_wgrad_workspace(uint64_t, uint64_t, uint64_t) { return 0; }

hipError_t launch_q8_wgrad(uint64_t M, uint64_t N, uint64_t K, const s2r_mat* dy16,
                           const s2r_q8_mat* dy8, const s2r_q8_mat& x, float* dw, uint64_t lddw,
                           bool accumulate, void*, hipStream_t s) {
  const uint64_t kt = (K + 63) / 64, nt = (N + 63) / 64;
  const s2r_mat d = dy16 ? *dy16 : s2r_mat{};
  const s2r_q8_mat q = dy8 ? *dy8 : s2r_q8_mat{};
  trace_mark(s, "k_q8_wgrad");
#define S2R_WGRAD(KY, FX)                                                               \
  hipLaunchKernelGGL((k_q8_wgrad<KY, FX>), dim3((uint32_t)(nt * kt)), dim3(kWgradThreads), 0, \
                     s, d, q, x, dw, lddw, (uint32_t)M, (uint32_t)N, (uint32_t)K, accumulate,  \
                     (uint32_t)kt)
  const int ky = dy16 ? 2 : (int)dy8->format;
  if (x.format == S2R_E4M3) {
    if (ky == 2) S2R_WGRAD(2, S2R_E4M3);
    else if (ky == S2R_E4M3) S2R_WGRAD(S2R_E4M3, S2R_E4M3);
    else S2R_WGRAD(S2R_E5M2, S2R_E4M3);
  } else {
    if (ky == 2) S2R_WGRAD(2, S2R_E5M2);
    else if (ky == S2R_E4M3) S2R_WGRAD(S2R_E4M3, S2R_E5M2);
    else S2R_WGRAD(S2R_E5M2, S2R_E5M2);
  }
#undef S2R_WGRAD
  return hipGetLastError();
}

}  // namespace s2r
