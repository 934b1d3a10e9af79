// moe_launch.hpp -- host-side launchers of the kernels behind s2r_moe.h (internal to libs2r).
#pragma once

#include "q8_launch.hpp"
#include "s2r_moe.h"

namespace s2r {

size_t moe_route_workspace(uint64_t T, uint32_t K, uint32_t E);
hipError_t launch_moe_route(uint64_t T, uint32_t K, uint32_t E, const int32_t* expert,
                            uint32_t* first, uint32_t* rows, int32_t* place, void* workspace,
                            hipStream_t s);
hipError_t launch_moe_gather(uint64_t T, uint32_t K, uint64_t D, const s2r_mat& x,
                             const int32_t* place, uint64_t R, const s2r_mat* out,
                             const s2r_q8_mat* outq, hipStream_t s);
hipError_t launch_moe_combine(uint64_t T, uint32_t K, uint64_t D, const s2r_mat& rows, uint64_t R,
                              const int32_t* place, const float* weight, const s2r_mat& y,
                              hipStream_t s);
hipError_t launch_moe_combine_grad(uint64_t T, uint32_t K, uint64_t D, const s2r_mat& dy,
                                   const int32_t* place, uint64_t R, const float* weight,
                                   const s2r_mat* rows, const s2r_mat* drows,
                                   const s2r_q8_mat* drowsq, float* dweight, hipStream_t s);

// The experts' matrices of a product: expert e's is `step` and `scale_step` bytes after e - 1's.
struct ExpertSteps {
  uint64_t step, scale_step;
};
hipError_t launch_q8_gemm_experts(uint64_t M, uint64_t N, uint64_t K, const s2r_experts& e,
                                  const s2r_q8_mat& a, const s2r_q8_mat& b, ExpertSteps steps,
                                  const s2r_mat& c, hipStream_t s);
hipError_t launch_q8_wgrad_experts(uint64_t M, uint64_t N, uint64_t K, const s2r_experts& e,
                                   const s2r_mat* dy16, const s2r_q8_mat* dy8, const s2r_q8_mat& x,
                                   float* dw, uint64_t lddw, uint64_t dw_step, bool accumulate,
                                   hipStream_t s);

}  // namespace s2r
