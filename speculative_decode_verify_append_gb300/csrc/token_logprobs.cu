// token_logprobs.cu -- log probability of a given token per logits row, the
// row's entropy and its most probable tokens.
//
// With m = max x, S = sum exp(x - m), T = sum exp(x - m) (x - m):
//   logprob = (x_t - m) - log S,  entropy = log S - T / S.
// One CTA per row: maximum, sums, then one pass per listed token that finds
// the largest (value, lowest index) behind the one before it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "sdva_common.cuh"

namespace sdva {
namespace {

constexpr int kThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;

struct LogprobArgs {
  const void* logits;
  long long row_stride;
  const int32_t* tokens;
  float* logprobs;
  float* entropy;
  int32_t* top_tokens;
  float* top_logprobs;
  int32_t* status;
  int vocab, num_top;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// (value, index) as one number that orders by value, then lowest index; NaN
// below -inf, the zeros equal.
__device__ __forceinline__ unsigned long long key_of(float x, int i) {
  const int b = __float_as_int(x + 0.0f);
  const uint32_t u = x != x ? 0u : (uint32_t)(b >= 0 ? b : b ^ 0x7fffffff) ^ 0x80000000u;
  return ((unsigned long long)u << 32) | (uint32_t)~i;
}

template <typename V, typename F>
__device__ V block_reduce(V v, F f) {
  __shared__ V part[kThreads / 32];
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
  for (int w = 1; w < kThreads / 32; ++w) v = f(v, part[w]);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(LogprobArgs a) {
  const int row = blockIdx.x;
  const int token = a.tokens[row];
  if (token < 0 || token >= a.vocab) {
    if (threadIdx.x == 0) {
      if (token != -1) raise_status(a.status, SDVA_STATUS_BAD_DRAFT);
      a.logprobs[row] = 0.0f;
      if (a.entropy != nullptr) a.entropy[row] = 0.0f;
    }
    for (int j = threadIdx.x; j < a.num_top; j += kThreads) {
      a.top_tokens[(size_t)row * a.num_top + j] = -1;
      a.top_logprobs[(size_t)row * a.num_top + j] = 0.0f;
    }
    return;
  }
  const T* x = static_cast<const T*>(a.logits) + (size_t)row * a.row_stride;
  const float ninf = __int_as_float(0xff800000);
  float m = ninf;
  bool nan = false;
  for (int i = threadIdx.x; i < a.vocab; i += kThreads) {
    const float v = to_f32(x[i]);
    nan |= v != v;
    m = fmaxf(m, v);
  }
  m = block_reduce(m, [](float p, float q) { return fmaxf(p, q); });
  float s = 0.0f, t = 0.0f;
  for (int i = threadIdx.x; i < a.vocab; i += kThreads) {
    const float d = to_f32(x[i]) - m, e = fast_exp2(d * kLog2e);
    s += e;
    t += e > 0.0f ? e * d : 0.0f;
  }
  s = block_reduce(s, [](float p, float q) { return p + q; });
  t = block_reduce(t, [](float p, float q) { return p + q; });
  nan = __syncthreads_or(nan) || m == ninf || m == -ninf;
  const float log_s = nan ? __int_as_float(0x7fc00000) : logf(s);
  if (threadIdx.x == 0) {
    a.logprobs[row] = to_f32(x[token]) - m - log_s;
    if (a.entropy != nullptr) a.entropy[row] = log_s - t / s;
  }
  unsigned long long last = ~0ull;
  for (int j = 0; j < a.num_top; ++j) {
    unsigned long long best = 0;
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) {
      const unsigned long long key = key_of(to_f32(x[i]), i);
      if (key < last && key > best) best = key;
    }
    last = best = block_reduce(best, [](unsigned long long p, unsigned long long q) { return p > q ? p : q; });
    if (threadIdx.x == 0) {
      const int i = (int)~(uint32_t)best;
      a.top_tokens[(size_t)row * a.num_top + j] = i;
      a.top_logprobs[(size_t)row * a.num_top + j] = to_f32(x[i]) - m - log_s;
    }
  }
}

}  // namespace
}  // namespace sdva

using namespace sdva;

extern "C" int token_logprobs(const void* logits, int logits_dtype, int64_t row_stride, int num_rows, int vocab,
                              const int32_t* tokens, int num_top, float* logprobs, float* entropy,
                              int32_t* top_tokens, float* top_logprobs, int32_t* status, sdva_stream_t stream) {
  if (num_rows == 0) return SDVA_OK;
  if (logits == nullptr || tokens == nullptr || logprobs == nullptr || num_rows < 0 || vocab <= 0 ||
      row_stride < vocab || num_top < 0 || num_top > vocab ||
      (num_top > 0 && (top_tokens == nullptr || top_logprobs == nullptr)))
    return SDVA_ERR_INVALID;
  if (num_top > SDVA_MAX_TOP || logits_dtype < SDVA_LOGITS_F32 || logits_dtype > SDVA_LOGITS_F16)
    return SDVA_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(logits) & (logits_dtype == SDVA_LOGITS_F32 ? 3u : 1u)) return SDVA_ERR_INVALID;
  const LogprobArgs a = {logits, row_stride, tokens, logprobs, entropy, top_tokens, top_logprobs, status, vocab, num_top};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (logits_dtype == SDVA_LOGITS_F32) {
    token_logprobs_kernel<float><<<num_rows, kThreads, 0, s>>>(a);
  } else if (logits_dtype == SDVA_LOGITS_BF16) {
    token_logprobs_kernel<__nv_bfloat16><<<num_rows, kThreads, 0, s>>>(a);
  } else {
    token_logprobs_kernel<__half><<<num_rows, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}
