// token_logprobs.cu -- log probability of a given token per logits row, the
// row's entropy and its most probable tokens.
//
// In log2 units, with y = (x - m) log2 e for the maximum m, S = sum 2^y and
// T = sum 2^y y:
//   logprob = ln 2 (y_t - log2 S),  entropy = ln 2 (log2 S - T / S),
// all in one pass with a running maximum per thread.  The call is bound by
// reading the logits (16-bit logits also by the work per element, about four
// instructions).
//
// One cluster of up to 8 CTAs per row, joined through distributed shared
// memory: no workspace, no second launch.  A thread reads 16-byte vectors at
// a stride of the block and keeps its maximum, S and T.  The listed tokens come out of these maxima: the k-th largest of the
// maxima of 128 groups of threads is a bound that k elements reach, so only
// threads whose maximum reaches it read their elements again (a few more
// than k), and what reaches it is put in order by counting.  Comparing a list on every element
// instead would cost more than the sums.  Where that bound says little (fewer
// than k finite values, long ties, NaN), every element is looked at again in
// index order against sorted lists of the warps.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <utility>

#include "tc_primitives.cuh"

namespace cg = cooperative_groups;

namespace sdva {
namespace {

using tc::f2_pack;
using tc::f2_unpack;
using tc::fadd2;
using tc::ffma2;
using tc::fmul2;

constexpr int kMaxCluster = 8;
constexpr int kBig = 512;       // threads per CTA (128 for short rows)
constexpr int kGroups = 128;    // groups of threads whose maxima bound the list
constexpr int kCandidates = 512;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNothing = -200.0f;  // 2^y is 0 in fp32 from here on down: lower values need no forming
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

// Element types: 16 bytes as floats, their largest, and one element.
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4, kUnroll = 4;  // elements per vector; vectors per thread and round
  static constexpr uint32_t kNone = 0xff800000u;  // -inf
  static __device__ float one(float x) { return x; }
  static __device__ void unpack(uint4 w, float* f) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
  static __device__ float largest(uint4 w) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8, kUnroll = 4;
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ float one(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ void unpack(uint4 w, float* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(u[i]), f[2 * i + 1] = bf16_hi(u[i]);
  }
  static __device__ float largest(uint4 w) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
};
template <>
struct Elem<__half> {
  static constexpr int kVec = 8, kUnroll = 4;
  static constexpr uint32_t kNone = 0xfc00fc00u;
  static __device__ float one(__half x) { return __half2float(x); }
  static __device__ void unpack(uint4 w, float* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = v.x, f[2 * i + 1] = v.y;
    }
  }
  static __device__ float largest(uint4 w) {
    const __half2* h = reinterpret_cast<const __half2*>(&w);
    const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
};

// (value, index) as one number that orders by value, then lowest index; NaN
// below -inf, the zeros equal; never 0, which stands for "none".
__device__ __forceinline__ uint32_t order_of(float x) {
  const int b = __float_as_int(x + 0.0f);
  return x != x ? 0u : (uint32_t)(b >= 0 ? b : b ^ 0x7fffffff) ^ 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t u) {
  const int b = (int)(u ^ 0x80000000u);
  return u == 0u ? __int_as_float(0x7fc00000) : __int_as_float(b >= 0 ? b : b ^ 0x7fffffff);
}
__device__ __forceinline__ Key key_of(float x, int i) { return ((Key)order_of(x) << 32) | (uint32_t)~i; }
__device__ __forceinline__ int index_of(Key k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float value_of(Key k) { return of_order((uint32_t)(k >> 32)); }

// Running statistics of a set of logits: m (0 where all are -inf), S, T.
struct Stat {
  float m, s, t;
};
__device__ __forceinline__ Stat moved(Stat a, float m) {  // the same about a larger m
  if (a.s == 0.0f || a.m == m) return {m, a.s, a.t};
  const float d = fmaxf((a.m - m) * kLog2e, kNothing), c = fast_exp2(d);
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
template <int kWarps>
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
template <typename T, int kThreads>
struct Part {
  static constexpr int kVec = Elem<T>::kVec;
  const T* x;
  int head, vectors;        // elements before the row's vectors; this CTA's vectors
  int first;                // index of their first element
  int tail0, extra;         // index of the first element behind the row's vectors; single elements

  __device__ Part(const T* row, int V, int part, int parts) {
    x = row;
    const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / (int)sizeof(T);
    head = min(V, off ? kVec - off : 0);
    const int all = (V - head) / kVec;
    tail0 = head + all * kVec;
    const int each = (all + parts - 1) / parts, lo = min(all, part * each);
    vectors = min(all, lo + each) - lo;
    first = head + lo * kVec;
    extra = part == 0 ? head + V - tail0 : 0;
  }
  __device__ uint4 load(int v) const { return __ldg(reinterpret_cast<const uint4*>(x + first) + v); }
  __device__ int extra_index(int e) const { return e < head ? e : tail0 + e - head; }
};

// 16 logits with maximum m into the thread's statistics; `top` is the
// thread's maximum.
__device__ __forceinline__ void add16(Stat& a, float& top, float m, const float (&x)[16]) {
  if (m > top) {
    top = m;
    a = moved(a, m);
  }
  const unsigned long long c2 = f2_pack(kLog2e, kLog2e), r2 = f2_pack(-a.m, -a.m);
  unsigned long long s[2] = {0ull, 0ull}, t[2] = {0ull, 0ull};
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const unsigned long long y2 = fmul2(fadd2(f2_pack(x[j], x[j + 1]), r2), c2);
    const float2 y = f2_unpack(y2);
    const unsigned long long e = f2_pack(fast_exp2(y.x), fast_exp2(y.y));
    s[(j >> 1) & 1] = fadd2(s[(j >> 1) & 1], e);
    t[(j >> 1) & 1] = ffma2(e, y2, t[(j >> 1) & 1]);
  }
  const float2 sum = f2_unpack(fadd2(s[0], s[1])), dot = f2_unpack(fadd2(t[0], t[1]));
  float d = dot.x + dot.y;
  if (d != d) {  // 0 * -inf: forbidden tokens have no part
    d = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float y = max_nan((x[j] - a.m) * kLog2e, kNothing);
      d += fast_exp2(y) * y;
    }
  }
  a.s += sum.x + sum.y;
  a.t += d;
}

// The statistics of n lanes' sets (a power of two), in every lane of them.
template <int n>
__device__ __forceinline__ Stat warp_join(Stat a) {
  float m = a.s == 0.0f ? __int_as_float(0xff800000) : a.m;  // of an empty set it means nothing
#pragma unroll
  for (int o = n / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  Stat b = moved(a, m == __int_as_float(0xff800000) ? 0.0f : m);
#pragma unroll
  for (int o = n / 2; o > 0; o >>= 1) {
    b.s += __shfl_xor_sync(0xffffffffu, b.s, o);
    b.t += __shfl_xor_sync(0xffffffffu, b.t, o);
  }
  return b;
}

// kThreads: 512, or 128 for short rows.
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) token_logprobs_kernel(LogprobArgs a, int parts) {
  constexpr int kVec = Elem<T>::kVec, kPer = 16 / kVec, kUnroll = Elem<T>::kUnroll, kWarps = kThreads / 32;
  __shared__ Stat s_stat[kWarps];
  __shared__ float4 s_group4[kGroups / 4];  // read four at a time
  __shared__ Key s_keys[kCandidates];  // candidates, or the warps' lists
  __shared__ uint32_t s_bound;
  __shared__ int s_count, s_odd;
  __shared__ Stat c_stat[kMaxCluster];  // in CTA 0: one entry per CTA of the cluster
  __shared__ Key c_keys[kMaxCluster][32];
  float* const s_group = reinterpret_cast<float*>(s_group4);
  static_assert(kCandidates >= kWarps * 32, "the warps' lists share the candidates' place");
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
  const Part<T, kThreads> p(static_cast<const T*>(a.logits) + (size_t)row * a.row_stride, a.vocab, part, parts);
  float x_t = 0.0f;
  if (part == 0 && th == 0) x_t = Elem<T>::one(p.x[token]);

  Stat st = {0.0f, 0.0f, 0.0f};
  float top = ninf;
  // rounds of whole vectors, the next one's loads in flight
  auto add = [&](const uint4 (&w)[kPer]) {
    float x[16], m = ninf;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      Elem<T>::unpack(w[k], x + k * kVec);
      m = fmaxf(m, Elem<T>::largest(w[k]));
    }
    add16(st, top, m, x);
  };
  constexpr int kRound = kUnroll * kThreads;
  int v = th;
  if (v + (kUnroll - 1) * kThreads < p.vectors) {
    uint4 next[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) next[u] = p.load(v + u * kThreads);
    do {
      uint4 w[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) w[u] = next[u];
      v += kRound;
      if (v + (kUnroll - 1) * kThreads < p.vectors) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) next[u] = p.load(v + u * kThreads);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; u += kPer) {
        uint4 g[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) g[k] = w[u + k];
        add(g);
      }
    } while (v + (kUnroll - 1) * kThreads < p.vectors);
  }
  if (v < p.vectors) {
    // fewer than a round: what is missing has no part in anything
    uint4 w[kUnroll];
    constexpr uint32_t none = Elem<T>::kNone;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      w[u] = v + u * kThreads < p.vectors ? p.load(v + u * kThreads) : make_uint4(none, none, none, none);
#pragma unroll
    for (int u = 0; u < kUnroll; u += kPer) {
      uint4 g[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) g[k] = w[u + k];
      if (v + u * kThreads < p.vectors) add(g);
    }
  }
  if (th < p.extra) {
    float x[16];
    x[0] = Elem<T>::one(p.x[p.extra_index(th)]);
#pragma unroll
    for (int j = 1; j < 16; ++j) x[j] = ninf;
    add16(st, top, x[0], x);
  }

  const Stat ws = warp_join<32>(st);
  if (lane == 0) s_stat[warp] = ws;
  if (a.num_top > 0) {
    float g = top;
#pragma unroll
    for (int o = kThreads / kGroups / 2; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (th % (kThreads / kGroups) == 0) s_group[th / (kThreads / kGroups)] = g;
    if (th == 0) {
      s_count = 0;
      s_bound = 0xffffffffu;
    }
  }
  __syncthreads();
  cluster.barrier_wait(std::move(started));
  if (warp == kWarps - 1) {
    const Stat b = warp_join<kWarps>(lane < kWarps ? s_stat[lane] : Stat{0.0f, 0.0f, 0.0f});
    if (lane == 0) {
      s_odd = b.s != b.s;  // a NaN, or +inf, which makes one
      *cluster.map_shared_rank(&c_stat[part], 0) = b;
    }
  }
  if (a.num_top > 0) {
    // The bound, the num_top-th largest group maximum: the smallest with
    // fewer than num_top above it.  A group's threads share the comparisons.
    {
      constexpr int kShare = kThreads / kGroups;
      const float own = s_group[th / kShare];
      int above = 0;
#pragma unroll
      for (int i = 0; i < kGroups / 4 / kShare; ++i) {
        const float4 o = s_group4[i * kShare + th % kShare];
        above += (o.x > own) + (o.y > own) + (o.z > own) + (o.w > own);
      }
#pragma unroll
      for (int o = kShare / 2; o > 0; o >>= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
      if (th % kShare == 0 && above < a.num_top) atomicMin(&s_bound, order_of(own));
    }
    __syncthreads();
    const float bound = of_order(s_bound);
    bool all = s_odd != 0 || bound == ninf;
    if (!all) {
      auto offer = [&](float x, int i) {
        if (x >= bound) {
          const int at = atomicAdd(&s_count, 1);
          if (at < kCandidates) s_keys[at] = key_of(x, i);
        }
      };
      unsigned hot = __ballot_sync(0xffffffffu, top >= bound);
      while (hot != 0 && __all_sync(0xffffffffu, s_count <= kCandidates)) {  // a count beyond the place ends the search
        const int who = warp * 32 + __ffs(hot) - 1;
        hot &= hot - 1;
#pragma unroll 3
        for (int v = who + lane * kThreads; v < p.vectors; v += 32 * kThreads) {
          const uint4 w = p.load(v);
          if (Elem<T>::largest(w) >= bound) {
            float x[kVec];
            Elem<T>::unpack(w, x);
#pragma unroll
            for (int j = 0; j < kVec; ++j) offer(x[j], p.first + v * kVec + j);
          }
        }
        if (lane == 0 && who < p.extra) offer(Elem<T>::one(p.x[p.extra_index(who)]), p.extra_index(who));
        __syncwarp();
      }
      __syncthreads();
      const int count = s_count;
      all = count > kCandidates;
      if (!all) {
        Key* const list = cluster.map_shared_rank(&c_keys[part][0], 0);
        for (int i = th; i < max(count, 32); i += kThreads) {
          const Key k = i < count ? s_keys[i] : 0;
          int rank = i;
          if (i < count) {
            rank = 0;
            for (int j = 0; j < count; ++j) rank += s_keys[j] > k;
          }
          if (rank < 32) list[rank] = k;
        }
      }
    }
    if (all) {  // the same for the whole CTA
      __syncthreads();
      Key list = 0;
      const int n = p.vectors * kVec + p.extra;
      for (int e0 = warp * 32; e0 < n; e0 += kThreads) {
        const int e = e0 + lane;
        Key k = 0;
        if (e < n) {
          const int i = e < p.extra ? p.extra_index(e) : p.first + e - p.extra;
          k = key_of(Elem<T>::one(p.x[i]), i);
        }
        const Key last = __shfl_sync(0xffffffffu, list, a.num_top - 1);
        if (__any_sync(0xffffffffu, k > last)) list = warp_merge(list, warp_sort(k));
      }
      list = block_merge<kWarps>(list, reinterpret_cast<Key(*)[32]>(s_keys));
      if (warp == 0) cluster.map_shared_rank(&c_keys[part][0], 0)[lane] = list;
    }
  }
  cluster.sync();
  if (part != 0 || warp != 0) return;
  const Stat b = warp_join<kMaxCluster>(lane < parts ? c_stat[lane] : Stat{0.0f, 0.0f, 0.0f});
  // no distribution: all -inf, or a NaN or +inf in the row
  const float log_s = (b.s > 0.0f ? log2f(b.s) : __int_as_float(0x7fc00000)) * kLn2;
  if (th == 0) {
    a.logprobs[row] = x_t - b.m - log_s;
    if (a.entropy != nullptr) a.entropy[row] = log_s - b.t / b.s * kLn2;
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

template <typename T, int kThreads>
int launch(const LogprobArgs& a, int num_rows, int sms, cudaStream_t stream) {
  // CTAs per row: two for every SM, and no less than two rounds of loads for a thread
  int parts = 1;
  while (parts < kMaxCluster && (long long)num_rows * parts < 2LL * sms &&
         a.vocab > 2LL * parts * kThreads * Elem<T>::kUnroll * Elem<T>::kVec)
    parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_rows * parts, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, kThreads>, a, parts) == cudaSuccess ? SDVA_OK
                                                                                              : SDVA_ERR_CUDA;
}

template <typename T>
int launch(const LogprobArgs& a, int num_rows, int sms, cudaStream_t stream) {
  return a.vocab < 8 * kBig * Elem<T>::kVec ? launch<T, 128>(a, num_rows, sms, stream)
                                            : launch<T, kBig>(a, num_rows, sms, stream);
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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return logits_dtype == SDVA_LOGITS_F32    ? launch<float>(a, num_rows, sms, s)
         : logits_dtype == SDVA_LOGITS_BF16 ? launch<__nv_bfloat16>(a, num_rows, sms, s)
                                            : launch<__half>(a, num_rows, sms, s);
}
