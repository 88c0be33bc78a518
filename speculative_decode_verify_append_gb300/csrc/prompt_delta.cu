// prompt_delta.cu -- the gated delta rule over packed prompts of different
// lengths, which leaves each lane's state behind its last token.
#include "delta_common.cuh"

namespace sdva {
namespace {

using namespace delta;

constexpr int kThreads = 128;

struct PromptArgs {
  float* state;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const float* log_decay;
  const float* beta;
  const int32_t* cu;
  const int32_t* slots;
  const int32_t* seq_lens;
  uint16_t* out;
  int32_t* status;
  long long q_stride, k_stride, v_stride;
  int num_slots, hk, hv, num_lanes, total;
  float scale, eps;
};

// One value row of the state per thread, token by token.
__global__ void __launch_bounds__(kThreads) prompt_delta_kernel(PromptArgs a) {
  const int h = blockIdx.x, b = blockIdx.y, th = threadIdx.x, kh = h / (a.hv / a.hk);
  __shared__ float sk[kHeadDim], sq[kHeadDim], part[2][kThreads / 32];
  const bool report = h == 0 && th == 0;
  bool bad = false;
  for (int i = th; i < a.num_lanes; i += kThreads) {
    const int lo = a.cu[i], hi = a.cu[i + 1];
    bad |= lo < 0 || hi < lo || hi > a.total;
  }
  if (__syncthreads_or(bad)) {
    if (report && b == 0) raise_status(a.status, SDVA_STATUS_BAD_COUNT);
    return;
  }
  const int row0 = a.cu[b], n = a.cu[b + 1] - row0;
  if (n == 0) return;
  const int slot = a.slots[b], L = a.seq_lens != nullptr ? a.seq_lens[b] : 1;
  if (L < 0 || slot < 0 || slot >= a.num_slots) {
    if (report) raise_status(a.status, L < 0 ? SDVA_STATUS_OVERFLOW : SDVA_STATUS_BAD_PAGE);
    return;
  }
  float* const row = a.state + ((size_t)slot * a.hv + h) * kStateElems + (size_t)th * kHeadDim;
  float S[kHeadDim];
#pragma unroll
  for (int d = 0; d < kHeadDim; d += 4) {
    const float4 x = L > 0 ? *reinterpret_cast<const float4*>(row + d) : make_float4(0.f, 0.f, 0.f, 0.f);
    S[d] = x.x, S[d + 1] = x.y, S[d + 2] = x.z, S[d + 3] = x.w;
  }
  for (int t = 0; t < n; ++t) {
    const size_t r = (size_t)row0 + t;
    const float k = __uint_as_float((uint32_t)a.k[r * a.k_stride + kh * kHeadDim + th] << 16);
    const float q = __uint_as_float((uint32_t)a.q[r * a.q_stride + kh * kHeadDim + th] << 16);
    float kk = k * k, qq = q * q;
    for (int o = 16; o > 0; o >>= 1) {
      kk += __shfl_xor_sync(0xffffffffu, kk, o);
      qq += __shfl_xor_sync(0xffffffffu, qq, o);
    }
    __syncthreads();
    sk[th] = k;
    sq[th] = q;
    if ((th & 31) == 0) part[0][th >> 5] = kk, part[1][th >> 5] = qq;
    __syncthreads();
    const float rk = norm_factor(part[0][0] + part[0][1] + part[0][2] + part[0][3], a.eps);
    const float rq = norm_factor(part[1][0] + part[1][1] + part[1][2] + part[1][3], a.eps);
    const float eg = expf(a.log_decay[r * a.hv + h]);
    float s = 0.0f, o = 0.0f;
#pragma unroll
    for (int d = 0; d < kHeadDim; ++d) {
      S[d] *= eg;
      s = fmaf(S[d], sk[d], s);
    }
    const float v = __uint_as_float((uint32_t)a.v[r * a.v_stride + h * kHeadDim + th] << 16);
    const float w = rk * a.beta[r * a.hv + h] * (v - rk * s);
#pragma unroll
    for (int d = 0; d < kHeadDim; ++d) {
      S[d] = fmaf(w, sk[d], S[d]);
      o = fmaf(S[d], sq[d], o);
    }
    a.out[(r * a.hv + h) * kHeadDim + th] = (uint16_t)(pack_bf16x2(a.scale * rq * o, 0.0f) & 0xFFFFu);
  }
#pragma unroll
  for (int d = 0; d < kHeadDim; d += 4)
    *reinterpret_cast<float4*>(row + d) = make_float4(S[d], S[d + 1], S[d + 2], S[d + 3]);
}

}  // namespace
}  // namespace sdva

using namespace sdva;

extern "C" size_t prompt_delta_workspace_size(int total_tokens, int num_lanes, int num_k_heads, int num_v_heads) {
  if (total_tokens <= 0 || num_lanes <= 0 || num_k_heads <= 0 || num_v_heads <= 0 || num_v_heads % num_k_heads != 0)
    return 0;
  return 256;
}

extern "C" int prompt_delta(float* state, int num_slots, const void* q, const void* k, const void* v, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, const float* log_decay, const float* beta,
                            int num_k_heads, int num_v_heads, int total_tokens, const int32_t* cu_tokens,
                            int num_lanes, const int32_t* slots, const int32_t* seq_lens, float scale, float qk_eps,
                            void* out, void* workspace, size_t workspace_bytes, int32_t* status,
                            sdva_stream_t stream) {
  if (total_tokens == 0) return SDVA_OK;
  if (state == nullptr || log_decay == nullptr || beta == nullptr || cu_tokens == nullptr || slots == nullptr ||
      out == nullptr || num_slots <= 0 || num_k_heads <= 0 || num_v_heads <= 0 || num_lanes <= 0 || total_tokens < 0 ||
      num_v_heads % num_k_heads != 0)
    return SDVA_ERR_INVALID;
  if (!rows_ok(q, q_stride, num_k_heads) || !rows_ok(k, k_stride, num_k_heads) || !rows_ok(v, v_stride, num_v_heads) ||
      !aligned16(state) || !aligned16(out))
    return SDVA_ERR_INVALID;
  if (!(scale > 0.0f) || scale > 3.0e38f || qk_eps != qk_eps || qk_eps > 3.0e38f) return SDVA_ERR_INVALID;
  if (num_lanes > 65535 || num_v_heads > 65535) return SDVA_ERR_UNSUPPORTED;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < prompt_delta_workspace_size(total_tokens, num_lanes, num_k_heads, num_v_heads))
    return SDVA_ERR_WORKSPACE;
  const PromptArgs a = {state,
                        static_cast<const uint16_t*>(q),
                        static_cast<const uint16_t*>(k),
                        static_cast<const uint16_t*>(v),
                        log_decay,
                        beta,
                        cu_tokens,
                        slots,
                        seq_lens,
                        static_cast<uint16_t*>(out),
                        status,
                        q_stride,
                        k_stride,
                        v_stride,
                        num_slots,
                        num_k_heads,
                        num_v_heads,
                        num_lanes,
                        total_tokens,
                        scale,
                        qk_eps};
  prompt_delta_kernel<<<dim3(num_v_heads, num_lanes), kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}
