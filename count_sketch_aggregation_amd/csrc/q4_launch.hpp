// q4_launch.hpp -- host-side launchers of the 4-bit kernels (internal to libs2r).
#pragma once

#include "q8_launch.hpp"
#include "s2r_q4.h"

namespace s2r {

inline s2r_q4_mat from_row(s2r_q4_mat x, uint64_t m) {
  if (x.q) x.q += m * x.ld, x.scale += m * x.lds;
  return x;
}

hipError_t launch_q4_save(uint64_t R, uint64_t C, const s2r_mat& x, const s2r_q4_mat* out,
                          const s2r_q4_mat* out_t, hipStream_t s);
hipError_t launch_q4_load(uint64_t R, uint64_t C, const s2r_q4_mat& in, const s2r_mat& x, hipStream_t s);

size_t q4_gemm_workspace(uint64_t M, uint64_t N, uint64_t K);
hipError_t launch_q4_gemm(uint64_t M, uint64_t N, uint64_t K, const s2r_q4_mat& a, const s2r_q4_mat& b,
                          const s2r_mat& c, void* workspace, hipStream_t s);

}  // namespace s2r
