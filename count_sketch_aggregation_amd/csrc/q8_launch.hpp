// q8_launch.hpp -- host-side launchers of the 8-bit training kernels (internal to libs2r).
#pragma once

#include "s2r_launch.hpp"
#include "s2r_q8.h"

namespace s2r {

// A launch holds below 2^32 threads: `go(first row, rows)` for as few ranges of rows as that takes, with
// `rows_each` rows and 256 threads to a workgroup and col_tiles workgroups side by side.
template <class F>
inline void by_rows(uint64_t M, uint64_t rows_each, uint64_t col_tiles, F&& go) {
  const uint64_t most = ((1ull << 24) - 1) / col_tiles * rows_each;
  for (uint64_t m = 0; m < M; m += most) go(m, M - m < most ? M - m : most);
}
// The same matrix from row m on; what the caller left out stays so.
inline s2r_mat from_row(s2r_mat x, uint64_t m) {
  if (x.data) x.data = static_cast<uint8_t*>(x.data) + m * x.ld * (x.dtype == S2R_F32 ? 4 : 2);
  return x;
}
inline s2r_q8_mat from_row(s2r_q8_mat x, uint64_t m) {
  if (x.q) x.q += m * x.ld, x.scale += m;
  return x;
}

hipError_t launch_q8_save(uint64_t M, uint64_t K, const s2r_mat& x, const s2r_q8_mat& out,
                          hipStream_t s);
hipError_t launch_q8_load(uint64_t M, uint64_t K, const s2r_q8_mat& in, const s2r_mat& x,
                          hipStream_t s);
hipError_t launch_q8_weight(uint64_t N, uint64_t K, const s2r_mat& w, const s2r_q8_mat& out,
                            const s2r_q8_mat* out_t, hipStream_t s);

size_t q8_gemm_workspace(uint64_t M, uint64_t N, uint64_t K);
hipError_t launch_q8_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q8_mat& a,
                          const s2r_q8_mat& b, const s2r_mat& c, bool fast, void* workspace,
                          hipStream_t s);

size_t q8_wgrad_workspace(uint64_t M, uint64_t N, uint64_t K);
hipError_t launch_q8_wgrad(uint64_t M, uint64_t N, uint64_t K, const s2r_mat* dy16,
                           const s2r_q8_mat* dy8, const s2r_q8_mat& x, float* dw, uint64_t lddw,
                           bool accumulate, void* workspace, hipStream_t s);

hipError_t launch_q8_glu(uint64_t M, uint64_t F, s2r_act act, const s2r_mat& g, const s2r_mat* u,
                         const s2r_q8_mat* gq, const s2r_q8_mat* uq, const s2r_mat* y,
                         const s2r_q8_mat* yq, hipStream_t s);
hipError_t launch_q8_glu_grad(uint64_t M, uint64_t F, s2r_act act, const s2r_q8_mat& gq,
                              const s2r_q8_mat* uq, const s2r_mat& dy, const s2r_mat* dg,
                              const s2r_mat* du, const s2r_q8_mat* dgq, const s2r_q8_mat* duq,
                              hipStream_t s);

}  // namespace s2r
