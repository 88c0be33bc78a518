// delta_common.cuh -- what the kernels of the gated delta rule share.
//
// A value head has a state S of 128 value rows by 128 key columns, fp32.  With
// k and q a token's key and query of the head's key head, as they are, and
// r_k = 1 / sqrt(|k|^2 + eps), r_q likewise (1 for a negative eps):
//     u_t = b_t (v_t - r_k e^g_t S_p k_t)
//     S_t = e^g_t S_p + r_k u_t k_t'
//     o_t = scale r_q S_t q_t
// Products with k and q themselves are exact to start with; the factors go to
// the results.
#pragma once

#include "sdva_common.cuh"
#include "sdva_internal.cuh"

namespace sdva {
namespace delta {

constexpr size_t kStateElems = (size_t)kHeadDim * kHeadDim;  // of one value head

// 16-byte alignment and strides of token rows of `heads` heads.
inline bool rows_ok(const void* p, int64_t stride, int heads) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride >= (int64_t)heads * kHeadDim &&
         (stride & 7) == 0;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

__device__ __forceinline__ float norm_factor(float sum_sq, float eps) {
  return eps < 0.0f ? 1.0f : rsqrtf(sum_sq + eps);
}

}  // namespace delta
}  // namespace sdva
