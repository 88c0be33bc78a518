// prompt_attn.cu -- causal attention of packed prompts over their own bf16
// keys and values, before the prompts' K/V go into the quantised cache.
//
// For row t of a lane and q head h of kv head g:  s_j = scale q_t . k_j over
// the lane's rows j <= t, out = sum_j exp(s_j - lse) v_j, lse = log sum exp s_j,
// in one pass over the keys with the running maximum and sum.
#include <math.h>

#include "sdva_common.cuh"
#include "sdva_internal.cuh"

namespace sdva {
namespace {

constexpr int kMaxPromptLanes = 1024;
constexpr int kThreads = 256;

struct PromptArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  long long q_stride, k_stride, v_stride;
  const int32_t* cu;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int Hq, G, total, num_lanes;
  float scale_log2;
};

// One warp per (row, q head), 4 dims a lane.
__global__ void __launch_bounds__(kThreads) prompt_attn_kernel(PromptArgs a) {
  int bad = 0;
  for (int i = threadIdx.x; i < a.num_lanes; i += kThreads) {
    const int lo = a.cu[i], hi = a.cu[i + 1];
    bad |= lo < 0 || hi < lo || hi > a.total;
  }
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_status(a.status, SDVA_STATUS_BAD_COUNT);
    return;
  }
  const int lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (id >= (long long)a.total * a.Hq) return;
  const int t = (int)(id / a.Hq), h = (int)(id % a.Hq);
  int lo = 0, hi = a.num_lanes;  // the last lane that starts at or before t
  if (t < a.cu[0] || t >= a.cu[a.num_lanes]) return;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const size_t col = (size_t)(h / a.G) * kHeadDim + lane * 4;
  const uint2 qw = *reinterpret_cast<const uint2*>(a.q + (size_t)t * a.q_stride + (size_t)h * kHeadDim + lane * 4);
  const float q0 = bf16_lo(qw.x), q1 = bf16_hi(qw.x), q2 = bf16_lo(qw.y), q3 = bf16_hi(qw.y);
  float m = __int_as_float(0xff800000), l = 0.0f, o0 = 0.0f, o1 = 0.0f, o2 = 0.0f, o3 = 0.0f;
  for (int j = a.cu[lo]; j <= t; ++j) {
    const uint2 kw = *reinterpret_cast<const uint2*>(a.k + (size_t)j * a.k_stride + col);
    const uint2 vw = *reinterpret_cast<const uint2*>(a.v + (size_t)j * a.v_stride + col);
    float s = q0 * bf16_lo(kw.x) + q1 * bf16_hi(kw.x) + q2 * bf16_lo(kw.y) + q3 * bf16_hi(kw.y);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s);
    const float c = m == mn ? 1.0f : fast_exp2(m - mn), p = fast_exp2(s - mn);
    m = mn;
    l = l * c + p;
    o0 = o0 * c + p * bf16_lo(vw.x);
    o1 = o1 * c + p * bf16_hi(vw.x);
    o2 = o2 * c + p * bf16_lo(vw.y);
    o3 = o3 * c + p * bf16_hi(vw.y);
  }
  const float inv = 1.0f / l;
  *reinterpret_cast<uint2*>(a.out + ((size_t)t * a.Hq + h) * kHeadDim + lane * 4) =
      make_uint2(pack_bf16x2(o0 * inv, o1 * inv), pack_bf16x2(o2 * inv, o3 * inv));
  if (lane == 0 && a.lse != nullptr) a.lse[(size_t)t * a.Hq + h] = m * 0.6931471805599453f + logf(l);
}

}  // namespace
}  // namespace sdva

using namespace sdva;

extern "C" int prompt_attn(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, int num_q_heads, int num_kv_heads, int total_tokens,
                           const int32_t* cu_tokens, int num_lanes, float sm_scale, void* out, float* lse,
                           int32_t* status, sdva_stream_t stream) {
  if (total_tokens == 0) return SDVA_OK;
  if (q == nullptr || k == nullptr || v == nullptr || cu_tokens == nullptr || out == nullptr) return SDVA_ERR_INVALID;
  if (total_tokens < 0 || num_lanes <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_q_heads % num_kv_heads != 0 || !(sm_scale > 0.0f) || !isfinite(sm_scale))
    return SDVA_ERR_INVALID;
  const int64_t qw = (int64_t)num_q_heads * kHeadDim, kw = (int64_t)num_kv_heads * kHeadDim;
  if (q_stride < qw || k_stride < kw || v_stride < kw || ((q_stride | k_stride | v_stride) & 7) ||
      ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
        reinterpret_cast<uintptr_t>(out)) &
       15u))
    return SDVA_ERR_INVALID;
  const int G = num_q_heads / num_kv_heads;
  if (num_lanes > kMaxPromptLanes || G > 128 || num_kv_heads > 65535) return SDVA_ERR_UNSUPPORTED;
  PromptArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cu = cu_tokens;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = status;
  a.Hq = num_q_heads;
  a.G = G;
  a.total = total_tokens;
  a.num_lanes = num_lanes;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  const long long warps = (long long)total_tokens * num_q_heads;
  const long long blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffLL) return SDVA_ERR_UNSUPPORTED;
  prompt_attn_kernel<<<(unsigned)blocks, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}
