// token_logprobs.cu -- log probability of a given token per logits row, the
// row's entropy and its most probable tokens.
//
// In log2 units, with y = (x - m) log2 e for the maximum m, S = sum 2^y and
// T = sum 2^y y:
//   logprob = ln 2 (y_t - log2 S),  entropy = ln 2 (log2 S - T / S),
// all in one pass with a running maximum per thread.  The call is bound by
// reading the logits (16-bit logits also by the work per element, about four
// instructions): 4,096 bf16 rows of 151,936 with a list of 5 200 us, 6.2 TB/s;
// few rows by a chain of steps (one fp32 row 4.8 us, with a list of 20 8.2).
//
// Few rows: a cluster of up to 8 CTAs per row, joined through distributed
// shared memory; no workspace, no second launch.  A thread reads 16-byte
// vectors at a stride of the block and keeps its maximum, S and T.  The listed
// tokens come out of these maxima: the k-th largest of the maxima of 128
// groups of threads is a bound that k elements reach, so only threads whose
// maximum reaches it read their elements again (a few more than k), and what
// reaches it is put in order by counting.  Comparing a list on every element
// instead would cost more than the sums.  Where that bound says little (fewer
// than k finite values, long ties, NaN), every element is looked at again
// against sorted lists of the warps.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <utility>

#include "sdva_internal.cuh"
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
  static constexpr int kVec = 4;  // elements per vector
  static constexpr uint32_t kNone = 0xff800000u;  // -inf
  static __device__ float one(float x) { return x; }
  static __device__ uint32_t word(float x) { return __float_as_uint(x); }
  static __device__ void unpack(uint4 w, float* f) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
  static __device__ float largest(uint4 w) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ float one(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ uint32_t word(__nv_bfloat16 x) { return (kNone & 0xffff0000u) | __bfloat16_as_ushort(x); }
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
  static constexpr int kVec = 8;
  static constexpr uint32_t kNone = 0xfc00fc00u;
  static __device__ float one(__half x) { return __half2float(x); }
  static __device__ uint32_t word(__half x) { return (kNone & 0xffff0000u) | __half_as_ushort(x); }
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
template <typename T>
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

// 16 logits (w) into the thread's statistics; `top` is the thread's maximum.
// Returns theirs.  0 * -inf, of a forbidden token, would make T a NaN: either y
// is kept above kNothing, two instructions more for two logits, or the sum is
// done again where it came out a NaN (of 4,096 bf16 rows of 151,936 the first
// takes 207 us whatever they hold, the second 199 and, where nine tokens in ten
// are forbidden, 282).
template <typename T, bool kAbove>
__device__ __forceinline__ float add16(Stat& a, float& top, const uint4 (&w)[16 / Elem<T>::kVec]) {
  constexpr int kVec = Elem<T>::kVec, kPer = 16 / kVec;
  float m = __int_as_float(0xff800000);
#pragma unroll
  for (int k = 0; k < kPer; ++k) m = fmaxf(m, Elem<T>::largest(w[k]));
  if (m > top) {
    top = m;
    a = moved(a, m);
  }
  float x[16];
#pragma unroll
  for (int k = 0; k < kPer; ++k) Elem<T>::unpack(w[k], x + k * kVec);
  const unsigned long long c2 = f2_pack(kLog2e, kLog2e), r2 = f2_pack(-a.m, -a.m);
  unsigned long long s[2] = {0ull, 0ull}, t[2] = {0ull, 0ull};
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    unsigned long long y2 = fmul2(fadd2(f2_pack(x[j], x[j + 1]), r2), c2);
    float2 y = f2_unpack(y2);
    if (kAbove) {
      y.x = max_nan(y.x, kNothing), y.y = max_nan(y.y, kNothing);
      y2 = f2_pack(y.x, y.y);
    }
    const unsigned long long e = f2_pack(fast_exp2(y.x), fast_exp2(y.y));
    s[(j >> 1) & 1] = fadd2(s[(j >> 1) & 1], e);
    t[(j >> 1) & 1] = ffma2(e, y2, t[(j >> 1) & 1]);
  }
  const float2 sum = f2_unpack(fadd2(s[0], s[1])), dot = f2_unpack(fadd2(t[0], t[1]));
  float d = dot.x + dot.y;
  if (!kAbove && d != d) {
    d = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float y = max_nan((x[j] - a.m) * kLog2e, kNothing);
      d += fast_exp2(y) * y;
    }
  }
  a.s += sum.x + sum.y;
  a.t += d;
  return m;
}
// one logit
template <typename T>
__device__ __forceinline__ void add1(Stat& a, float& top, T x) {
  constexpr uint32_t none = Elem<T>::kNone;
  uint4 w[16 / Elem<T>::kVec];
#pragma unroll
  for (int k = 0; k < 16 / Elem<T>::kVec; ++k) w[k] = make_uint4(none, none, none, none);
  w[0].x = Elem<T>::word(x);
  add16<T, true>(a, top, w);
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

// The statistics of a cluster's CTAs, in every lane.
__device__ __forceinline__ Stat cluster_join(const Stat* c, int parts) {
  const int i = threadIdx.x % kMaxCluster;
  return warp_join<kMaxCluster>(i < parts ? c[i] : Stat{0.0f, 0.0f, 0.0f});
}

// A row's outputs, by one warp: b in every lane, x_t in lane 0, the sorted
// lists of `parts` CTAs.
__device__ __forceinline__ void write_row(const LogprobArgs& a, int row, float x_t, const Stat& b,
                                          const Key (*lists)[32], int parts) {
  const int lane = threadIdx.x & 31;
  // no distribution: all -inf, or a NaN or +inf in the row
  const float log_s = (b.s > 0.0f ? log2f(b.s) : __int_as_float(0x7fc00000)) * kLn2;
  if (lane == 0) {
    a.logprobs[row] = x_t - b.m - log_s;
    if (a.entropy != nullptr) a.entropy[row] = log_s - b.t / b.s * kLn2;
  }
  if (a.num_top > 0) {
    Key k = lists[0][lane];
    for (int q = 1; q < parts; ++q) k = warp_merge(k, lists[q][lane]);
    if (lane < a.num_top) {
      a.top_tokens[(size_t)row * a.num_top + lane] = index_of(k);
      a.top_logprobs[(size_t)row * a.num_top + lane] = value_of(k) - b.m - log_s;
    }
  }
}

// Short rows: 128 threads, a thread's rounds of loads in registers.  A row in
// one block has nothing of a cluster: its barriers and launch take a
// microsecond (333 fp16 rows of 32,003 14.0 against 13.0 us, 8,192 fp32 rows of
// 5,000 59.6 against 52.0).
constexpr int kShortThreads = 128;
constexpr int kShortVecs = 32 * kShortThreads;  // fewer vectors to a row: a warp reads a thread's at once
template <typename T, bool kCluster, int kUnroll>
__global__ void __launch_bounds__(128, 32 / kUnroll) short_logprobs_kernel(LogprobArgs a, int parts) {
  constexpr int kThreads = kShortThreads;
  constexpr int kVec = Elem<T>::kVec, kPer = 16 / kVec, kWarps = kThreads / 32;
  __shared__ Stat s_stat[kWarps];
  __shared__ float4 s_group4[kGroups / 4];  // read four at a time
  __shared__ Key s_keys[kCandidates];  // candidates, or the warps' lists
  __shared__ uint32_t s_bound;
  __shared__ int s_count, s_odd;
  constexpr int kLists = kCluster ? kMaxCluster : 1;
  __shared__ Stat c_stat[kLists];  // in CTA 0: one entry per CTA of the cluster
  __shared__ Key c_keys[kLists][32];
  float* const s_group = reinterpret_cast<float*>(s_group4);
  static_assert(kCandidates >= kWarps * 32, "the warps' lists share the candidates' place");
  const int row = kCluster ? blockIdx.x / parts : blockIdx.x, part = kCluster ? blockIdx.x % parts : 0;
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
  cg::cluster_group::arrival_token started;
  if (kCluster) started = cluster.barrier_arrive();
  Stat* stat_out = &c_stat[part];
  Key* list_out = &c_keys[part][0];
  if (kCluster) {
    stat_out = cluster.map_shared_rank(stat_out, 0);
    list_out = cluster.map_shared_rank(list_out, 0);
  }
  const float ninf = __int_as_float(0xff800000);
  const Part<T> p(static_cast<const T*>(a.logits) + (size_t)row * a.row_stride, a.vocab, part, parts);
  float x_t = 0.0f;
  if (part == 0 && th == 0) x_t = Elem<T>::one(p.x[token]);

  Stat st = {0.0f, 0.0f, 0.0f};
  float top = ninf;
  // rounds of whole vectors, the next one's loads in flight
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
        add16<T, true>(st, top, g);
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
      if (v + u * kThreads < p.vectors) add16<T, true>(st, top, g);
    }
  }
  if (th < p.extra) add1(st, top, p.x[p.extra_index(th)]);

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
  if (kCluster) cluster.barrier_wait(std::move(started));
  if (warp == kWarps - 1) {
    const Stat b = warp_join<kWarps>(lane < kWarps ? s_stat[lane] : Stat{0.0f, 0.0f, 0.0f});
    if (lane == 0) {
      s_odd = b.s != b.s;  // a NaN, or +inf, which makes one
      *stat_out = b;
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
      if (th < p.extra && top >= bound) offer(Elem<T>::one(p.x[p.extra_index(th)]), p.extra_index(th));
      // the vectors of the threads that reach it, one a lane, of four threads at a time
      unsigned hot = __ballot_sync(0xffffffffu, top >= bound);
      while (hot != 0 && __all_sync(0xffffffffu, s_count <= kCandidates)) {  // a count beyond the place ends the search
        uint4 w[4];
        int v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[u] = hot != 0 ? warp * 32 + __ffs(hot) - 1 + lane * kThreads : p.vectors;
          hot &= hot - 1;
          w[u] = v[u] < p.vectors ? p.load(v[u]) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (v[u] < p.vectors && Elem<T>::largest(w[u]) >= bound) {
            float x[kVec];
            Elem<T>::unpack(w[u], x);
#pragma unroll
            for (int j = 0; j < kVec; ++j) offer(x[j], p.first + v[u] * kVec + j);
          }
        __syncwarp();
      }
      __syncthreads();
      const int count = s_count;
      all = count > kCandidates;
      if (!all) {
        for (int i = th; i < max(count, 32); i += kThreads) {
          const Key k = i < count ? s_keys[i] : 0;
          int rank = i;
          if (i < count) {
            rank = 0;
            for (int j = 0; j < count; ++j) rank += s_keys[j] > k;
          }
          if (rank < 32) list_out[rank] = k;
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
      if (warp == 0) list_out[lane] = list;
    }
  }
  if (kCluster) cluster.sync();
  else __syncthreads();
  if (part != 0 || warp != 0) return;
  const Stat b = kCluster ? cluster_join(c_stat, parts) : c_stat[0];
  write_row(a, row, x_t, b, c_keys, kCluster ? parts : 1);
}

// Long rows.  Warps 0-7 stream: they add up what a ring of 16 KB stages
// brings and hand their sums and maxima to warps 8-11 (the team), which
// finish the row while the next one streams; warp 12 fills the ring with bulk
// copies.  The reading of one row after the other never stops for the end of
// a row, and the copies leave the load path to the team: with one kind of
// warps that loads through registers, a row's end costs 3,000 cycles of
// shuffles and shared-memory reads queued behind the loads (4,096 bf16 rows
// 251 us against 198).  Many rows: a CTA takes units of consecutive rows
// and, when one is on its way, the next one's CTA's place.  Few rows
// (kCluster): one cluster of `parts` CTAs per row.
constexpr int kStreamThreads = 256, kTeamThreads = 128, kLongThreads = kStreamThreads + kTeamThreads + 32;
constexpr int kStages = 6, kStageVecs = 4 * kStreamThreads;  // 16-byte vectors per stage
constexpr uint32_t kStageBytes = kStageVecs * 16;
constexpr int kRowRing = 4;
constexpr int kTeamWarps = kTeamThreads / 32, kStreamWarps = kStreamThreads / 32;
static_assert(kShortVecs == 4 * kStageVecs, "rows of fewer than four stages are short");
static_assert(kGroups == kTeamThreads && kStreamThreads == 2 * kGroups,
              "a group is a team thread's two stream threads");

struct LongCtl {
  uint64_t full[kStages], empty[kStages], row_full[kRowRing], row_free[kRowRing], sums_full[2], sums_free[2], next_full;
  alignas(16) uint32_t next_cta[4];
  float4 group4[kGroups / 4];
  Key keys[kCandidates];  // candidates, or the warps' lists
  Key c_keys[kMaxCluster][32];
  Stat c_stat[kMaxCluster];
  Stat stat[2][kStreamWarps];
  // of each stream thread: its maximum, the stage of the row that holds the
  // largest vectors' maximum, and the largest of the other stages'
  float top[2][kStreamThreads], second[2][kStreamThreads];
  int stage[2][kStreamThreads];
  int hot[kStreamThreads], wide[kStreamThreads];
  int row[kRowRing];  // -1: no more
  float x_t;       // of the given token, across the cluster's barrier
  uint32_t bound;
  int count, hots, wides, abort;
};
constexpr size_t kLongSmem = kStages * kStageBytes + sizeof(LongCtl);
static_assert(2 * (kLongSmem + 1024) <= 233472, "two CTAs per SM");

__device__ __forceinline__ void team_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kTeamThreads) : "memory"); }
// whether every thread of the team says so, the same for all
__device__ __forceinline__ bool team_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "n"(kTeamThreads)
      : "memory");
  return r != 0;
}

template <typename T, bool kCluster>
__global__ void __launch_bounds__(kLongThreads, 2)
    long_logprobs_kernel(LogprobArgs a, int num_rows, int unit, int parts, long long limit) {
  constexpr int kVec = Elem<T>::kVec, kPer = 16 / kVec;
  // many rows of 16-bit logits (a prompt's, where nothing is forbidden) are bound by the work per element
  constexpr bool kAbove = kCluster || sizeof(T) == 4;
  extern __shared__ __align__(16) uint8_t smem[];
  LongCtl* const ctl = reinterpret_cast<LongCtl*>(smem + kStages * kStageBytes);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31, th = threadIdx.x;
  const int part = kCluster ? blockIdx.x % parts : 0;
  const float ninf = __int_as_float(0xff800000);
  auto scored = [&](int row) {
    const int token = a.tokens[row];
    return token >= 0 && token < a.vocab;
  };
  auto leave_row = [&](int row) {  // by one warp: a row that is not scored
    if (lane == 0) {
      if (a.tokens[row] != -1) raise_status(a.status, SDVA_STATUS_BAD_DRAFT);
      a.logprobs[row] = 0.0f;
      if (a.entropy != nullptr) a.entropy[row] = 0.0f;
    }
    if (lane < a.num_top) {
      a.top_tokens[(size_t)row * a.num_top + lane] = -1;
      a.top_logprobs[(size_t)row * a.num_top + lane] = 0.0f;
    }
  };
  if (kCluster && !scored(blockIdx.x / parts)) {  // the same for the whole cluster
    if (part == 0 && warp == 0) leave_row(blockIdx.x / parts);
    return;
  }
  if (th == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(smem_u32(&ctl->full[i]), 1);
      tc::mbar_init(smem_u32(&ctl->empty[i]), kStreamWarps);
    }
    for (int i = 0; i < kRowRing; ++i) {
      tc::mbar_init(smem_u32(&ctl->row_full[i]), 1);
      tc::mbar_init(smem_u32(&ctl->row_free[i]), kStreamWarps + kTeamWarps);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(smem_u32(&ctl->sums_full[i]), kStreamWarps);
      tc::mbar_init(smem_u32(&ctl->sums_free[i]), kTeamWarps);
    }
    tc::mbar_init(smem_u32(&ctl->next_full), 1);
    ctl->abort = 0;
    tc::mbar_fence_init();
  }
  __syncthreads();
  cg::cluster_group cluster = cg::this_cluster();
  // CTA 0's shared memory is written to once every CTA of the cluster runs
  if (kCluster) cluster.sync();
  volatile int* const abort_flag = &ctl->abort;
  auto wait = [&](uint64_t& bar, uint32_t parity) {
    return tc::mbar_wait<false>(smem_u32(&bar), parity & 1u, abort_flag, limit);
  };
  auto arrive = [&](uint64_t& bar) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(smem_u32(&bar));
  };
  auto give_up = [&]() {
    if (lane == 0) {
      ctl->abort = 1;
      raise_status(a.status, SDVA_STATUS_TIMEOUT);
    }
  };
  auto part_of = [&](int row) {
    return Part<T>(static_cast<const T*>(a.logits) + (size_t)row * a.row_stride, a.vocab, part, parts);
  };
  bool ok = true;

  if (warp == kStreamWarps + kTeamWarps) {
    // ---- the copies ----
    uint32_t fills = 0, rows = 0, asks = 0;
    auto publish = [&](int row) {
      const uint32_t slot = rows % kRowRing;
      if (rows >= kRowRing && !wait(ctl->row_free[slot], rows / kRowRing - 1)) return false;
      if (lane == 0) {
        ctl->row[slot] = row;
        tc::mbar_arrive(smem_u32(&ctl->row_full[slot]));
      }
      __syncwarp();
      ++rows;
      return true;
    };
    uint32_t next = kCluster ? blockIdx.x / parts : blockIdx.x;
    for (bool more = true; more && ok;) {
      const int first = (int)next * unit, end = (int)min((long long)num_rows, (long long)first + unit);
      for (int row = first; row < end && ok; ++row) {
        if (!kCluster && !scored(row)) {
          leave_row(row);
          continue;
        }
        if (!(ok = publish(row))) break;
        const Part<T> p = part_of(row);
        for (int v = 0; v < p.vectors && ok; v += kStageVecs, ++fills) {
          const uint32_t st = fills % kStages;
          if (fills >= kStages && !(ok = wait(ctl->empty[st], fills / kStages - 1))) break;
          if (lane == 0) {
            const uint32_t bytes = 16u * (uint32_t)min(kStageVecs, p.vectors - v), bar = smem_u32(&ctl->full[st]);
            tc::mbar_arrive_expect_tx(bar, bytes);
            tc::bulk_load(smem_u32(smem) + st * kStageBytes, reinterpret_cast<const uint4*>(p.x + p.first) + v, bytes,
                          bar);
          }
          __syncwarp();
        }
      }
      more = false;
      if (!kCluster && ok) {
        if (lane == 0) tc::take_over_next(smem_u32(ctl->next_cta), smem_u32(&ctl->next_full));
        __syncwarp();
        if ((ok = wait(ctl->next_full, asks++))) {
          more = tc::taken_over(smem_u32(ctl->next_cta), &next);
          tc::fence_proxy_async_smem();  // the answer is read before the next one is written
          __syncwarp();
        }
      }
    }
    if (ok) ok = publish(-1);
    if (!ok) give_up();
    // No copy outlives the CTA, whichever warp gave up (bounded; where none
    // did, the sums wait for the same copies).
    int none = 0;
    for (uint32_t f = fills > kStages ? fills - kStages : 0; f < fills; ++f)
      tc::mbar_wait<false>(smem_u32(&ctl->full[f % kStages]), (f / kStages) & 1u, &none, 400000000LL);
    if (asks > 0) tc::mbar_wait<false>(smem_u32(&ctl->next_full), (asks - 1) & 1u, &none, 400000000LL);
  } else if (warp < kStreamWarps) {
    // ---- the sums ----
    uint32_t st = 0, phase = 0;
    for (uint32_t r = 0;; ++r) {
      const uint32_t slot = r % kRowRing;
      if (!(ok = wait(ctl->row_full[slot], r / kRowRing))) break;
      const int row = ctl->row[slot];
      if (row < 0) break;
      const Part<T> p = part_of(row);
      T x0;
      if (th < p.extra) x0 = p.x[p.extra_index(th)];
      Stat sum = {0.0f, 0.0f, 0.0f};
      float top = ninf, best = ninf, second = ninf;
      int at_best = 0;
      for (int v0 = 0; v0 < p.vectors && ok; v0 += kStageVecs) {
        if (!(ok = wait(ctl->full[st], phase))) break;
        float here = ninf;
        const uint4* const stage = reinterpret_cast<const uint4*>(smem + st * kStageBytes);
        uint4 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int at = u * kStreamThreads + th;
          // what a last, shorter stage lacks has no part in anything
          w[u] = v0 + at < p.vectors ? stage[at]
                                     : make_uint4(Elem<T>::kNone, Elem<T>::kNone, Elem<T>::kNone, Elem<T>::kNone);
        }
        // The next copy may overwrite the stage: the arrival orders these loads
        // before ordinary accesses that follow it, not before those of the
        // copies, which are another proxy's; the fence does.
        tc::fence_proxy_async_smem();
        arrive(ctl->empty[st]);
        if (++st == kStages) {
          st = 0;
          phase ^= 1u;
        }
#pragma unroll
        for (int u = 0; u < 4; u += kPer) {
          uint4 g[kPer];
#pragma unroll
          for (int k = 0; k < kPer; ++k) g[k] = w[u + k];
          here = fmaxf(here, add16<T, kAbove>(sum, top, g));
        }
        second = fmaxf(second, fminf(best, here));
        if (here > best) {
          best = here;
          at_best = v0 / kStageVecs;
        }
      }
      if (!ok) break;
      if (th < p.extra) add1(sum, top, x0);
      const uint32_t d = r & 1u;
      if (r >= 2 && !(ok = wait(ctl->sums_free[d], r / 2 - 1))) break;
      const Stat joined = warp_join<32>(sum);
      if (lane == 0) ctl->stat[d][warp] = joined;
      ctl->top[d][th] = top;
      ctl->second[d][th] = second;
      ctl->stage[d][th] = at_best;
      arrive(ctl->sums_full[d]);
      if (lane == 0) tc::mbar_arrive(smem_u32(&ctl->row_free[slot]));
    }
    if (!ok) give_up();
  } else {
    // ---- the end of a row ----
    const int tt = th - kStreamThreads, tw = warp - kStreamWarps;
    float* const group = reinterpret_cast<float*>(ctl->group4);
    for (uint32_t r = 0;; ++r) {
      const uint32_t slot = r % kRowRing, d = r & 1u;
      if (!team_all(ok = wait(ctl->row_full[slot], r / kRowRing))) break;
      const int row = ctl->row[slot];
      if (row < 0) break;
      const Part<T> p = part_of(row);
      float x_t = 0.0f;
      if (part == 0 && tt == 0) x_t = Elem<T>::one(p.x[a.tokens[row]]);
      if (!team_all(ok = wait(ctl->sums_full[d], r / 2))) break;
      // this thread's two stream threads
      float top[2], second[2];
      int at_best[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int who = tt + k * kTeamThreads;
        top[k] = ctl->top[d][who];
        second[k] = ctl->second[d][who];
        at_best[k] = ctl->stage[d][who];
      }
      const Stat b = warp_join<kStreamWarps>(ctl->stat[d][lane % kStreamWarps]);
      arrive(ctl->sums_free[d]);
      group[tt] = fmaxf(top[0], top[1]);
      if (tt == 0) {
        ctl->count = ctl->hots = ctl->wides = 0;
        ctl->bound = 0xffffffffu;
      }
      team_sync();
      if (a.num_top > 0) {
        // the bound: the smallest group maximum with fewer than num_top above it
        {
          const float mine = group[tt];
          int above = 0;
#pragma unroll 8
          for (int i = 0; i < kGroups / 4; ++i) {
            const float4 o = ctl->group4[i];
            above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
          }
          if (above < a.num_top) atomicMin(&ctl->bound, order_of(mine));
        }
        team_sync();
        const float bound = of_order(ctl->bound);
        Key* list = &ctl->c_keys[part][0];
        if (kCluster) list = cluster.map_shared_rank(list, 0);
        // a NaN (or +inf, which makes one) hides its thread's maximum
        bool all = b.s != b.s || bound == ninf;
        if (!all) {
          auto offer = [&](float x, int i) {
            if (x >= bound) {
              const int at = atomicAdd(&ctl->count, 1);
              if (at < kCandidates) ctl->keys[at] = key_of(x, i);
            }
          };
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (top[k] >= bound) {
              const int who = tt + k * kTeamThreads;
              if (second[k] >= bound) ctl->wide[atomicAdd(&ctl->wides, 1)] = who;
              else ctl->hot[atomicAdd(&ctl->hots, 1)] = at_best[k] * kStageVecs + who;
              if (who < p.extra) offer(Elem<T>::one(p.x[p.extra_index(who)]), p.extra_index(who));
            }
          team_sync();
          auto look = [&](uint4 w, int v) {
            if (Elem<T>::largest(w) >= bound) {
              float x[kVec];
              Elem<T>::unpack(w, x);
#pragma unroll
              for (int j = 0; j < kVec; ++j) offer(x[j], p.first + v * kVec + j);
            }
          };
          // Their vectors, dealt to the team: of the one stage that reaches the
          // bound, or of all; in a cluster's short parts mostly one to a thread,
          // where less code to fetch is worth more (one row 8.4 against 9.1 us).
          constexpr int kBatch = kCluster ? 1 : 4;
          const int single = 4 * ctl->hots, each = (p.vectors + kStreamThreads - 1) / kStreamThreads;
          const int items = single + ctl->wides * each;
#pragma unroll 1
          for (int i0 = tt; i0 < items; i0 += kBatch * kTeamThreads) {
            uint4 w[kBatch];
            int v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
              const int i = i0 + u * kTeamThreads, k = i - single;
              v[u] = i < single  ? ctl->hot[i >> 2] + (i & 3) * kStreamThreads
                     : i < items ? ctl->wide[k / each] + k % each * kStreamThreads
                                 : p.vectors;
              w[u] = v[u] < p.vectors ? p.load(v[u]) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
              if (v[u] < p.vectors) look(w[u], v[u]);
          }
          team_sync();
          const int count = ctl->count;
          all = count > kCandidates;
          if (!all)
            for (int i = tt; i < max(count, 32); i += kTeamThreads) {
              const Key k = i < count ? ctl->keys[i] : 0;
              int rank = i;
              if (i < count) {
                rank = 0;
                for (int j = 0; j < count; ++j) rank += ctl->keys[j] > k;
              }
              if (rank < 32) list[rank] = k;
            }
        }
        if (all) {  // the same for the whole team
          team_sync();
          Key mine = 0;
          auto take = [&](Key k) {
            const Key last = __shfl_sync(0xffffffffu, mine, a.num_top - 1);
            if (__any_sync(0xffffffffu, k > last)) mine = warp_merge(mine, warp_sort(k));
          };
          if (tw == 0) take(lane < p.extra ? key_of(Elem<T>::one(p.x[p.extra_index(lane)]), p.extra_index(lane)) : 0);
          for (int v0 = tw * 32; v0 < p.vectors; v0 += 4 * kTeamThreads) {
            uint4 w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int v = v0 + u * kTeamThreads + lane;
              w[u] = v < p.vectors ? p.load(v) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int v = v0 + u * kTeamThreads + lane;
              float x[kVec];
              Elem<T>::unpack(w[u], x);
#pragma unroll
              for (int j = 0; j < kVec; ++j) take(v < p.vectors ? key_of(x[j], p.first + v * kVec + j) : 0);
            }
          }
          // the warps' lists into one
          ctl->keys[tw * 32 + lane] = mine;
          team_sync();
          if (tw == 0) {
#pragma unroll
            for (int o = 1; o < kTeamWarps; ++o) mine = warp_merge(mine, ctl->keys[o * 32 + lane]);
            list[lane] = mine;
          }
        }
      }
      if (kCluster) {
        if (tt == 0) {
          *cluster.map_shared_rank(&ctl->c_stat[part], 0) = b;
          ctl->x_t = x_t;
        }
      } else {
        team_sync();
        if (tw == 0) write_row(a, row, x_t, b, ctl->c_keys, 1);
      }
      arrive(ctl->row_free[slot]);
    }
    if (!ok) give_up();
  }
  if (kCluster) {
    cluster.sync();
    if (part == 0 && warp == 0) {
      const Stat b = cluster_join(ctl->c_stat, parts);
      write_row(a, blockIdx.x / parts, ctl->x_t, b, ctl->c_keys, parts);
    }
  }
}

template <typename T>
int launch(const LogprobArgs& a, int num_rows, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SDVA_ERR_CUDA;
  constexpr int kVec = Elem<T>::kVec;
  // Rows of fewer than four stages go to the small blocks: the team's time on
  // a row is that of about as many (4,000 rows of 10,000 fp32 47 us in small
  // blocks, 56 streamed; 2,000 of 30,000 bf16 38 and 40).
  const bool is_short = a.vocab < kShortVecs * kVec;
  // CTAs per row: while every SM would not have one, and each has two rounds of loads
  const long long round = is_short ? kShortThreads * 4LL * kVec : (long long)kStageVecs * kVec;
  const long long wanted = is_short ? 2LL * sms : sms;
  int parts = 1;
  while (parts < kMaxCluster && (long long)num_rows * parts < wanted && a.vocab > 2 * parts * round) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cudaError_t e;
  if (is_short) {
    cfg.gridDim = dim3((unsigned)num_rows * parts, 1, 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.numAttrs = parts > 1 ? 1 : 0;
    // Up to four blocks per SM have eight vectors of a thread in flight, and as
    // many again, where a thread has as many; more blocks four, which leaves
    // registers for eight of them (333 fp16 rows of 32,003 11.9 against 12.7 us,
    // 333 fp32 rows of 15,000 9.4 / 10.9; one row of 32,000 bf16 8.9 / 8.5, 1,000
    // of 32,003 23.7 / 22.1, 8,192 of 5,000 62.6 / 50.6).
    const bool deep = (long long)num_rows * parts <= 4 * sms && a.vocab >= 8LL * kShortThreads * kVec * parts;
    const auto kernel = parts > 1 ? (deep ? short_logprobs_kernel<T, true, 8> : short_logprobs_kernel<T, true, 4>)
                                  : (deep ? short_logprobs_kernel<T, false, 8> : short_logprobs_kernel<T, false, 4>);
    e = cudaLaunchKernelEx(&cfg, kernel, a, parts);
  } else {
    const auto kernel = parts > 1 ? long_logprobs_kernel<T, true> : long_logprobs_kernel<T, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLongSmem) != cudaSuccess)
      return SDVA_ERR_CUDA;
    // consecutive rows per unit of work: more than one only where units stay many for each SM
    const int unit = parts > 1 ? 1 : (int)std::min(8LL, std::max(1LL, num_rows / (32LL * sms)));
    cfg.gridDim = dim3(parts > 1 ? (unsigned)num_rows * parts : ((unsigned)num_rows + unit - 1) / unit, 1, 1);
    cfg.blockDim = dim3(kLongThreads, 1, 1);
    cfg.dynamicSmemBytes = kLongSmem;
    cfg.numAttrs = parts > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kernel, a, num_rows, unit, parts, wait_limit());
  }
  return e == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
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
  const LogprobArgs a = {logits,     row_stride,   tokens, logprobs, entropy,
                         top_tokens, top_logprobs, status, vocab,    num_top};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return logits_dtype == SDVA_LOGITS_F32    ? launch<float>(a, num_rows, s)
         : logits_dtype == SDVA_LOGITS_BF16 ? launch<__nv_bfloat16>(a, num_rows, s)
                                            : launch<__half>(a, num_rows, s);
}
