// token_logprobs.cu -- log probability of a given token per logits row, the
// row's entropy and its most probable tokens.
//
// With m = max x, S = sum exp(x - m), T = sum exp(x - m) (x - m):
//   logprob = (x_t - m) - log S,  entropy = log S - T / S,
// all three in one pass with a running maximum per thread.  The call is bound
// by reading the logits.
//
// One cluster of up to 8 CTAs per row, joined through distributed shared
// memory: no workspace, no second launch.  A thread reads 16-byte vectors at
// a stride of the block and keeps the running (m, S, T) and the place of its
// maximum.  The listed tokens come out of these maxima: no element of a
// thread whose maximum is not among the k largest of the block's threads can
// be among the k largest elements, so the block sorts its threads' maxima
// (64-bit keys of value and place, bitonic in the warps, then merged pairwise)
// and reads again only what the k threads at the top had read.  Comparing a
// list on every element instead would cost more than the sums.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <utility>

#include "sdva_common.cuh"

namespace cg = cooperative_groups;

namespace sdva {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 4;            // vectors in flight per thread
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNothing = -150.0f;   // exp is 0 in fp32 from here on down: lower values need no forming
typedef unsigned long long Key;

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

// Element types: 16 bytes as floats, and one element.
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static __device__ float one(float x) { return x; }
  static __device__ void unpack(uint4 w, float* f) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ float one(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ void unpack(uint4 w, float* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(u[i]), f[2 * i + 1] = bf16_hi(u[i]);
  }
};
template <>
struct Elem<__half> {
  static constexpr int kVec = 8;
  static __device__ float one(__half x) { return __half2float(x); }
  static __device__ void unpack(uint4 w, float* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = v.x, f[2 * i + 1] = v.y;
    }
  }
};

// (value, index) as one number that orders by value, then lowest index; NaN
// below -inf, the zeros equal; never 0, which stands for "none".
__device__ __forceinline__ Key key_of(float x, int i) {
  const int b = __float_as_int(x + 0.0f);
  const uint32_t u = x != x ? 0u : (uint32_t)(b >= 0 ? b : b ^ 0x7fffffff) ^ 0x80000000u;
  return ((Key)u << 32) | (uint32_t)~i;
}
__device__ __forceinline__ int index_of(Key k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float value_of(Key k) {
  const uint32_t u = (uint32_t)(k >> 32);
  const int b = (int)(u ^ 0x80000000u);
  return u == 0u ? __int_as_float(0x7fc00000) : __int_as_float(b >= 0 ? b : b ^ 0x7fffffff);
}

// Running statistics of a set of logits; s == 0: empty or all -inf.
struct Stat {
  float m, s, t;
};
__device__ __forceinline__ Stat moved(Stat a, float m) {  // the same with reference m >= a.m
  if (a.s == 0.0f || a.m == m) return {m, a.s, a.t};
  const float d = fmaxf(a.m - m, kNothing), c = fast_exp2(d * kLog2e);
  return {m, a.s * c, (a.t + a.s * d) * c};
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sorted lists of 32 keys, one a lane, largest first.
__device__ __forceinline__ Key exchange(Key k, int j, bool larger_low) {
  const Key o = __shfl_xor_sync(0xffffffffu, k, j);
  const bool low = ((threadIdx.x & 31) & j) == 0;
  return (low == larger_low) == (k > o) ? k : o;
}
__device__ __forceinline__ Key warp_sort(Key k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int j = n / 2; j > 0; j /= 2) k = exchange(k, j, (lane & n) == 0);
  return k;
}
// the 32 largest of two sorted lists, sorted
__device__ __forceinline__ Key warp_merge(Key a, Key b) {
  const Key r = __shfl_sync(0xffffffffu, b, 31 - (threadIdx.x & 31));
  Key k = a > r ? a : r;
#pragma unroll
  for (int j = 16; j > 0; j /= 2) k = exchange(k, j, true);
  return k;
}
// the 32 largest of the warps' sorted lists, in warp 0
__device__ Key block_merge(Key k, Key (*buf)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int half = kWarps / 2; half > 0; half /= 2) {
    if (warp >= half && warp < 2 * half) buf[warp][lane] = k;
    __syncthreads();
    if (warp < half) k = warp_merge(k, buf[warp + half][lane]);
  }
  return k;
}

// The part of a row that one CTA reads.  Vectors start at the row's first
// 16-byte boundary; the few elements before it and behind the last whole
// vector go one each to the first threads of CTA 0.
template <typename T>
struct Part {
  static constexpr int kVec = Elem<T>::kVec;
  const T* x;
  int head, vocab, first, vectors;  // elements before the vectors; this CTA's vectors of the row
  int extra;                        // single elements
  int tail0;                        // index of the first element behind the vectors

  __device__ Part(const T* row, int V, int part, int parts) {
    x = row;
    vocab = V;
    const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / (int)sizeof(T);
    head = min(V, off ? kVec - off : 0);
    const int all = (V - head) / kVec;
    tail0 = head + all * kVec;
    const int each = (all + parts - 1) / parts;
    first = min(all, part * each);
    vectors = min(all, first + each) - first;
    extra = part == 0 ? head + V - tail0 : 0;
  }
  __device__ uint4 load(int v) const { return __ldg(reinterpret_cast<const uint4*>(x + head) + first + v); }
  __device__ int index(int v) const { return head + (first + v) * kVec; }
  __device__ int extra_index(int e) const { return e < head ? e : tail0 + e - head; }
  // thread that reads element i
  __device__ int owner(int i) const {
    if (i < head) return i;
    if (i >= tail0) return head + i - tail0;
    return ((i - head) / kVec - first) % kThreads;
  }
  __device__ int owned(int th) const { return max(0, (vectors - th + kThreads - 1) / kThreads) * kVec + (th < extra); }
  __device__ int owned_index(int th, int e) const {  // its e-th element
    const int n = owned(th) - (th < extra);
    return e < n ? index(th + e / kVec * kThreads) + e % kVec : extra_index(th);
  }
};

// 16 logits, element j at index i0 + (j / kVec) * stride + j % kVec: into the
// thread's statistics; m is the thread's maximum, best its first place.
template <int kVec>
__device__ __forceinline__ void add16(Stat& a, int& best, const float (&x)[16], int i0, int stride) {
  float m = fmaxf(x[0], x[1]);
#pragma unroll
  for (int j = 2; j < 16; ++j) m = fmaxf(m, x[j]);
  if (m > a.m || best < 0) {
    int at = 0;
#pragma unroll
    for (int j = 15; j > 0; --j)
      if (x[j] == m) at = j;
    if (x[0] == m) at = 0;
    best = i0 + at / kVec * stride + at % kVec;
    a = moved(a, m);
  }
  const float ref = a.m == __int_as_float(0xff800000) ? 0.0f : a.m;  // all -inf so far
  float s[2] = {0.0f, 0.0f}, t[2] = {0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float d = max_nan(x[j] - ref, kNothing), e = fast_exp2(d * kLog2e);
    s[j & 1] += e;
    t[j & 1] += e * d;
  }
  a.s += s[0] + s[1];
  a.t += t[0] + t[1];
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) token_logprobs_kernel(LogprobArgs a, int parts) {
  constexpr int kVec = Elem<T>::kVec;
  __shared__ Stat s_stat[kWarps];
  __shared__ Key s_keys[kWarps][32];
  __shared__ Key s_hot[32];
  __shared__ int s_odd;
  __shared__ Stat c_stat[kMaxCluster];  // in CTA 0: one entry per CTA of the cluster
  __shared__ Key c_keys[kMaxCluster][32];
  const int row = blockIdx.x / parts, part = blockIdx.x % parts;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, th = threadIdx.x;
  const int token = a.tokens[row];
  if (token < 0 || token >= a.vocab) {  // the same for the whole cluster
    if (part != 0) return;
    if (th == 0) {
      if (token != -1) raise_status(a.status, SDVA_STATUS_BAD_DRAFT);
      a.logprobs[row] = 0.0f;
      if (a.entropy != nullptr) a.entropy[row] = 0.0f;
    }
    if (th < a.num_top) {
      a.top_tokens[(size_t)row * a.num_top + th] = -1;
      a.top_logprobs[(size_t)row * a.num_top + th] = 0.0f;
    }
    return;
  }
  // CTA 0's shared memory is written to once every CTA of the cluster runs
  cg::cluster_group cluster = cg::this_cluster();
  auto started = cluster.barrier_arrive();
  const float ninf = __int_as_float(0xff800000);
  const Part<T> p(static_cast<const T*>(a.logits) + (size_t)row * a.row_stride, a.vocab, part, parts);
  float x_t = 0.0f;
  if (part == 0 && th == 0) x_t = Elem<T>::one(p.x[token]);

  Stat st = {ninf, 0.0f, 0.0f};
  int best = -1;
  for (int v = th; v < p.vectors; v += kUnroll * kThreads) {
    uint4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (v + u * kThreads < p.vectors) w[u] = p.load(v + u * kThreads);
    constexpr int kPer = 16 / kVec;  // vectors per sixteen elements
#pragma unroll
    for (int u = 0; u < kUnroll; u += kPer) {
      float x[16];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (v + (u + k) * kThreads < p.vectors) {
          Elem<T>::unpack(w[u + k], x + k * kVec);
        } else {
#pragma unroll
          for (int j = 0; j < kVec; ++j) x[k * kVec + j] = ninf;  // no part in anything
        }
      }
      if (v + u * kThreads < p.vectors) add16<kVec>(st, best, x, p.index(v + u * kThreads), kThreads * kVec);
    }
  }
  if (th < p.extra) {
    const int i = p.extra_index(th);
    float x[16];
    x[0] = Elem<T>::one(p.x[i]);
#pragma unroll
    for (int j = 1; j < 16; ++j) x[j] = ninf;
    // behind the vectors in index order or before them: an equal value there keeps its place only if it comes first
    const float m = st.m;
    const int was = best;
    add16<kVec>(st, best, x, i, 0);
    if (x[0] == m && was >= 0) best = min(was, i);
  }
  const Key own = best < 0 ? 0 : key_of(st.m, best);

  // the block's statistics
  {
    float m = st.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    Stat w = moved(st, m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      w.s += __shfl_xor_sync(0xffffffffu, w.s, o);
      w.t += __shfl_xor_sync(0xffffffffu, w.t, o);
    }
    if (lane == 0) s_stat[warp] = w;
  }
  if (a.num_top > 0) {
    // the threads with the largest maxima, largest first
    Key k = block_merge(warp_sort(own), s_keys);
    if (warp == 0) s_hot[lane] = k;
  }
  __syncthreads();
  cluster.barrier_wait(std::move(started));
  if (warp == 0) {
    const Stat w = lane < kWarps ? s_stat[lane] : Stat{ninf, 0.0f, 0.0f};
    float m = w.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    Stat b = moved(w, m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      b.s += __shfl_xor_sync(0xffffffffu, b.s, o);
      b.t += __shfl_xor_sync(0xffffffffu, b.t, o);
    }
    if (lane == 0) {
      s_odd = b.s != b.s;
      *cluster.map_shared_rank(&c_stat[part], 0) = b;
    }
  }
  if (a.num_top > 0) {
    __syncthreads();
    // A NaN (or +inf, which makes one) hides its thread's maximum: then every
    // thread's elements are looked at again.
    const bool odd = s_odd != 0;
    const Key least = odd ? 0 : s_hot[a.num_top - 1];
    Key list = 0;
    for (int h = warp; h < (odd ? kThreads : a.num_top); h += kWarps) {
      if (!odd && s_hot[h] == 0) break;
      const int who = odd ? h : p.owner(index_of(s_hot[h])), n = p.owned(who);
      for (int e = lane; e - lane < n; e += 32) {
        Key k = 0;
        if (e < n) {
          const int i = p.owned_index(who, e);
          k = key_of(Elem<T>::one(p.x[i]), i);
        }
        if (k < least) k = 0;
        const Key last = __shfl_sync(0xffffffffu, list, a.num_top - 1);
        if (__any_sync(0xffffffffu, k > last)) list = warp_merge(list, warp_sort(k));
      }
    }
    __syncthreads();
    list = block_merge(list, s_keys);
    if (warp == 0) cluster.map_shared_rank(&c_keys[part][0], 0)[lane] = list;
  }
  cluster.sync();
  if (part != 0 || warp != 0) return;
  const Stat w = lane < parts ? c_stat[lane] : Stat{ninf, 0.0f, 0.0f};
  float m = w.m;
#pragma unroll
  for (int o = kMaxCluster / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  Stat b = moved(w, m);
#pragma unroll
  for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
    b.s += __shfl_xor_sync(0xffffffffu, b.s, o);
    b.t += __shfl_xor_sync(0xffffffffu, b.t, o);
  }
  // no distribution: all -inf, or a NaN or +inf in the row
  const float log_s = b.s > 0.0f ? logf(b.s) : __int_as_float(0x7fc00000);
  if (lane == 0) {
    a.logprobs[row] = x_t - b.m - log_s;
    if (a.entropy != nullptr) a.entropy[row] = log_s - b.t / b.s;
  }
  if (a.num_top > 0) {
    const float ref = __shfl_sync(0xffffffffu, b.m, 0), ls = __shfl_sync(0xffffffffu, log_s, 0);
    Key k = c_keys[0][lane];
    for (int q = 1; q < parts; ++q) k = warp_merge(k, c_keys[q][lane]);
    if (lane < a.num_top) {
      a.top_tokens[(size_t)row * a.num_top + lane] = index_of(k);
      a.top_logprobs[(size_t)row * a.num_top + lane] = value_of(k) - ref - ls;
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
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SDVA_ERR_CUDA;
  const LogprobArgs a = {logits, row_stride, tokens, logprobs, entropy, top_tokens, top_logprobs, status, vocab, num_top};
  // CTAs per row: enough that every SM has its two, and no less than one round of loads for each thread
  int parts = 1;
  const long long round = (long long)kThreads * (logits_dtype == SDVA_LOGITS_F32 ? 4 : 8);
  while (parts < kMaxCluster && (long long)num_rows * parts < 2LL * sms && vocab > 2 * parts * round) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_rows * parts, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = logits_dtype == SDVA_LOGITS_F32    ? token_logprobs_kernel<float>
                      : logits_dtype == SDVA_LOGITS_BF16 ? token_logprobs_kernel<__nv_bfloat16>
                                                         : token_logprobs_kernel<__half>;
  return cudaLaunchKernelEx(&cfg, kernel, a, parts) == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}
