// delta_common.cuh -- what the kernels of the gated delta rule share.
//
// A value head has a state S of 128 value rows by 128 key columns, fp32.  With
// k' = 2^-e k and q' = 2^-e q a token's key and query brought to a largest
// element in [1, 2) (exact), and r = 2^e / sqrt(|k|^2 + eps) their factor
// (2^e for a negative eps), so that kn = r k':
//     u_t = b_t (v_t - r e^g_t S_p k'_t)
//     S_t = e^g_t S_p + r u_t k'_t'
//     o_t = scale r_q S_t q'_t
// k' and q' are exact in fp16: the 8 bits of a bf16 number, and elements below
// 2^-14 of the row's largest to 2^-25 of it.  The other operand of a product on
// the tensor cores goes in two parts of 11 bits, x = hi + lo + at most 2^-22 |x|,
// so that the state keeps what fp32 gives it; what goes to the output alone is
// taken in one part (2^-11 of a value, bf16's rounding is 2^-8).  What a row of the
// state is multiplied with or grows by goes in fp16 parts, about a power of two that
// brings the row's largest to the top of fp16's range (off by 2^-39 of it then, if that
// is more); what has no such bound in tf32 parts, with fp32's exponents.
#pragma once

#include "sdva_common.cuh"
#include "sdva_internal.cuh"
#include "tc_primitives.cuh"

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

// The power of two that brings a magnitude to [1, 2) (to [2, 4) at fp32's upper
// end, below 1 for subnormals), and its inverse.
struct Scale {
  float down, up;
};
__device__ __forceinline__ Scale scale_of_row(float amax) {
  const uint32_t e = min(max(__float_as_uint(amax) >> 23, 1u), 253u);
  return {__uint_as_float((254u - e) << 23), __uint_as_float(e << 23)};
}
// As scale_of_row, to the top of fp16's range, [2^13, 2^14): what is 2^-16 of the largest
// still has two whole parts.  All of a row of zeros, or of less than 2^-113, stays below.
__device__ __forceinline__ Scale scale_to_top(float amax) {
  const uint32_t e = min(max(__float_as_uint(amax) >> 23, 14u), 253u);
  return {__uint_as_float((254u + 13u - e) << 23), __uint_as_float((e - 13u) << 23)};
}
// r = 2^e / sqrt(|k|^2 + eps) from sum_sq = |k'|^2.  eps 2^-2e overflows for rows
// below 2^-64 or so, whose kn is below 2^-54 then and taken as 0.
__device__ __forceinline__ float row_factor(float sum_sq, float eps, Scale s) {
  return eps < 0.0f ? s.up : rsqrtf(sum_sq + eps * s.down * s.down);
}

// Waits for the bulk copies that `bar` counts.  Where that takes more than `limit` cycles (0: where they are not there
// yet) it returns false, but not before they are, or the default limit has run out too: no copy outlives the CTA.
__device__ __forceinline__ bool copies_here(uint32_t bar, uint32_t parity, int* never, long long limit) {
  if (tc::mbar_test_wait(bar, parity) || (limit > 0 && tc::mbar_wait<false>(bar, parity, never, limit))) return true;
  tc::mbar_wait<false>(bar, parity, never);
  return false;
}

// The transpose of an 8 x 8 matrix of 16-bit elements held as two to a thread.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The same of 32-bit elements, two to a thread.
__device__ __forceinline__ void transpose8(float& x0, float& x1) {
  const uint32_t a = __float_as_uint(x0), b = __float_as_uint(x1);
  const uint32_t lo = transpose8(__byte_perm(a, b, 0x5410)), hi = transpose8(__byte_perm(a, b, 0x7632));
  x0 = __uint_as_float(__byte_perm(lo, hi, 0x5410));
  x1 = __uint_as_float(__byte_perm(lo, hi, 0x7632));
}
// Two values in two fp16 parts.
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_f16x2(x0 - f.x, x1 - f.y);
}

__device__ __forceinline__ void split_f16(float2 x, uint32_t& hi, uint32_t& lo) { split_f16(x.x, x.y, hi, lo); }

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// The upper 11 bits of x.
__device__ __forceinline__ float upper_11(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFFE000u); }
// x in two parts of 11 bits, off by 2^-22 |x| at most in all of fp32's range.
__device__ __forceinline__ void split_tf32(float x, float& hi, float& lo) {
  hi = to_tf32(x);
  lo = upper_11(x - hi);
}
// x rounded to 22 bits, and those in two parts.
__device__ __forceinline__ float round_22(float x) { return __uint_as_float((__float_as_uint(x) + 2u) & ~3u); }
__device__ __forceinline__ void split_22(float x, float& hi, float& lo) {
  hi = upper_11(x);
  lo = x - hi;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

}  // namespace delta
}  // namespace sdva
