// verify_delta.cu -- verify_delta and commit_delta: the gated delta rule over a
// verify window and the move of a state by the updates that were accepted.
//
// A window's updates and outputs follow from the state in front of it:
// with D_ij the product of e^g on the way from slot j (left out) to slot i (0
// where j is no ancestor of i) and a_i the product of e^g down to i,
//     u_i = b_i (v_i - r_i a_i S k_i - r_i sum_j<i D_ij r_j (k_i . k_j) u_j)
//     o_i = scale r_q (a_i S q_i + sum_j<=i D_ij r_j (q_i . k_j) u_j)
// so that the state is read once for all of them, and a tree costs what a
// chain does.
#include "delta_common.cuh"

namespace sdva {
namespace {

using namespace delta;

constexpr int kThreads = 128;

struct VerifyArgs {
  float* state;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const float* log_decay;
  const float* beta;
  const int32_t* n_lane;
  const int32_t* parent;
  const int32_t* slots;
  uint16_t* out;
  float* deltas;
  int32_t* status;
  long long q_stride, k_stride, v_stride;
  int num_slots, hk, hv, window;
  float scale, eps;
};

__global__ void __launch_bounds__(kThreads) verify_delta_kernel(VerifyArgs a) {
  const int h = blockIdx.x, b = blockIdx.y, th = threadIdx.x, W = a.window;
  const int kh = h / (a.hv / a.hk);
  __shared__ float sk[kMaxWindow][kHeadDim], sq[kMaxWindow][kHeadDim];
  __shared__ float rk[kMaxWindow], rq[kMaxWindow], eg[kMaxWindow], beta[kMaxWindow], fall[kMaxWindow];
  __shared__ float dm[kMaxWindow][kMaxWindow], A[kMaxWindow][kMaxWindow], P[kMaxWindow][kMaxWindow];
  __shared__ int par[kMaxWindow];
  const bool report = h == 0 && th == 0;
  int n = a.n_lane != nullptr ? a.n_lane[b] : W;
  if (n < 0 || n > W) {
    if (report) raise_status(a.status, SDVA_STATUS_BAD_COUNT);
    n = 0;
  }
  const int slot = a.slots[b];
  if (n > 0 && (slot < 0 || slot >= a.num_slots)) {
    if (report) raise_status(a.status, SDVA_STATUS_BAD_PAGE);
    n = 0;
  }
  if (n > 0) {
    int wrong = 0;
    if (th < n) {
      const int p = a.parent != nullptr && th > 0 ? a.parent[b * W + th] : th - 1;
      par[th] = p;
      wrong = th > 0 && (p < 0 || p >= th);
    }
    if (__syncthreads_or(wrong)) {
      if (report) raise_status(a.status, SDVA_STATUS_BAD_TREE);
      n = 0;
    }
  }
  const size_t row0 = (size_t)b * W;
  for (int i = n; i < W; ++i) {
    const size_t at = ((row0 + i) * a.hv + h) * kHeadDim + th;
    a.out[at] = 0;
    if (a.deltas != nullptr) a.deltas[at] = 0.0f;
  }
  if (n == 0) return;
  for (int i = 0; i < n; ++i) {
    sk[i][th] = __uint_as_float((uint32_t)a.k[(row0 + i) * a.k_stride + kh * kHeadDim + th] << 16);
    sq[i][th] = __uint_as_float((uint32_t)a.q[(row0 + i) * a.q_stride + kh * kHeadDim + th] << 16);
  }
  if (th < n) {
    eg[th] = expf(a.log_decay[(row0 + th) * a.hv + h]);
    beta[th] = a.beta[(row0 + th) * a.hv + h];
  }
  __syncthreads();
  if (th < n) {
    float s = 0.0f, t = 0.0f;
    for (int d = 0; d < kHeadDim; ++d) {
      s = fmaf(sk[th][d], sk[th][d], s);
      t = fmaf(sq[th][d], sq[th][d], t);
    }
    rk[th] = norm_factor(s, a.eps);
    rq[th] = norm_factor(t, a.eps);
    for (int i = 0; i < n; ++i) dm[i][th] = i < th ? 0.0f : i == th ? 1.0f : dm[par[i]][th] * eg[i];
    if (th == 0)
      for (int i = 0; i < n; ++i) fall[i] = i == 0 ? eg[0] : fall[par[i]] * eg[i];
  }
  __syncthreads();
  for (int x = th; x < n * n; x += kThreads) {
    const int i = x / n, j = x % n;
    float s = 0.0f, t = 0.0f;
    for (int d = 0; d < kHeadDim; ++d) {
      s = fmaf(sk[i][d], sk[j][d], s);
      t = fmaf(sq[i][d], sk[j][d], t);
    }
    A[i][j] = j < i && dm[i][j] != 0.0f ? dm[i][j] * rk[j] * s : 0.0f;
    P[i][j] = dm[i][j] != 0.0f ? dm[i][j] * rk[j] * t : 0.0f;
  }
  __syncthreads();
  float* const row = a.state + ((size_t)slot * a.hv + h) * kStateElems + (size_t)th * kHeadDim;
  float S[kHeadDim];
#pragma unroll
  for (int d = 0; d < kHeadDim; d += 4) {
    const float4 x = *reinterpret_cast<const float4*>(row + d);
    S[d] = x.x, S[d + 1] = x.y, S[d + 2] = x.z, S[d + 3] = x.w;
  }
  float u[kMaxWindow];
#pragma unroll
  for (int i = 0; i < kMaxWindow; ++i) {
    if (i >= n) break;
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int d = 0; d < kHeadDim; ++d) {
      s = fmaf(S[d], sk[i][d], s);
      t = fmaf(S[d], sq[i][d], t);
    }
    s *= fall[i];
    t *= fall[i];
#pragma unroll
    for (int j = 0; j < i; ++j) s = fmaf(A[i][j], u[j], s);
    const float v = __uint_as_float((uint32_t)a.v[(row0 + i) * a.v_stride + h * kHeadDim + th] << 16);
    u[i] = beta[i] * (v - rk[i] * s);
#pragma unroll
    for (int j = 0; j <= i; ++j) t = fmaf(P[i][j], u[j], t);
    const size_t at = ((row0 + i) * a.hv + h) * kHeadDim + th;
    a.out[at] = (uint16_t)(pack_bf16x2(a.scale * rq[i] * t, 0.0f) & 0xFFFFu);
    if (a.deltas != nullptr) a.deltas[at] = rk[i] * u[i];
  }
  if (a.deltas != nullptr) return;
  // the whole window is committed
#pragma unroll
  for (int d = 0; d < kHeadDim; ++d) S[d] *= fall[n - 1];
#pragma unroll
  for (int i = 0; i < kMaxWindow; ++i) {
    if (i >= n) break;
    const float w = rk[i] * u[i] * dm[n - 1][i];
#pragma unroll
    for (int d = 0; d < kHeadDim; ++d) S[d] = fmaf(w, sk[i][d], S[d]);
  }
#pragma unroll
  for (int d = 0; d < kHeadDim; d += 4)
    *reinterpret_cast<float4*>(row + d) = make_float4(S[d], S[d + 1], S[d + 2], S[d + 3]);
}

struct CommitArgs {
  float* state;
  const uint16_t* k;
  const float* log_decay;
  const float* deltas;
  const int32_t* accept_len;
  const int32_t* path;
  const int32_t* slots;
  int32_t* status;
  long long k_stride;
  int num_slots, hk, hv, window;
};

__global__ void __launch_bounds__(kThreads) commit_delta_kernel(CommitArgs a) {
  const int h = blockIdx.x, b = blockIdx.y, th = threadIdx.x, W = a.window;
  const int kh = h / (a.hv / a.hk);
  __shared__ int at[kMaxWindow];
  __shared__ float coef[kMaxWindow];
  __shared__ float all;
  const bool report = h == 0 && th == 0;
  const int m = a.accept_len[b] + 1, slot = a.slots[b];
  if (m < 0 || m > W) {
    if (report) raise_status(a.status, SDVA_STATUS_BAD_COUNT);
    return;
  }
  if (m == 0) return;
  if (slot < 0 || slot >= a.num_slots) {
    if (report) raise_status(a.status, SDVA_STATUS_BAD_PAGE);
    return;
  }
  int wrong = 0;
  if (th < m) {
    const int p = a.path != nullptr ? a.path[b * W + th] : th;
    at[th] = p;
    wrong = p < 0 || p >= W;
  }
  if (__syncthreads_or(wrong)) {
    if (report) raise_status(a.status, SDVA_STATUS_BAD_TREE);
    return;
  }
  const size_t row0 = (size_t)b * W;
  if (th == 0) {
    float c = 1.0f;
    for (int j = m - 1; j >= 0; --j) {
      coef[j] = c;
      c *= expf(a.log_decay[(row0 + at[j]) * a.hv + h]);
    }
    all = c;
  }
  __syncthreads();
  float* const s = a.state + ((size_t)slot * a.hv + h) * kStateElems;
  for (int r = 0; r < kHeadDim; ++r) {
    float x = s[r * kHeadDim + th] * all;
    for (int j = 0; j < m; ++j) {
      const float w = coef[j] * a.deltas[((row0 + at[j]) * a.hv + h) * kHeadDim + r];
      x = fmaf(w, __uint_as_float((uint32_t)a.k[(row0 + at[j]) * a.k_stride + kh * kHeadDim + th] << 16), x);
    }
    s[r * kHeadDim + th] = x;
  }
}

}  // namespace
}  // namespace sdva

using namespace sdva;

extern "C" int verify_delta(float* state, int num_slots, const void* q, const void* k, const void* v, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, const float* log_decay, const float* beta,
                            int num_k_heads, int num_v_heads, int num_lanes, int window, const int32_t* n_lane,
                            const int32_t* parent, const int32_t* slots, float scale, float qk_eps, void* out,
                            float* deltas, int32_t* status, sdva_stream_t stream) {
  if (state == nullptr || log_decay == nullptr || beta == nullptr || slots == nullptr || out == nullptr ||
      num_slots <= 0 || num_k_heads <= 0 || num_v_heads <= 0 || num_lanes <= 0 || window <= 0 ||
      num_v_heads % num_k_heads != 0)
    return SDVA_ERR_INVALID;
  if (!rows_ok(q, q_stride, num_k_heads) || !rows_ok(k, k_stride, num_k_heads) || !rows_ok(v, v_stride, num_v_heads) ||
      !aligned16(state) || !aligned16(out) || !aligned16(deltas))
    return SDVA_ERR_INVALID;
  if (!(scale > 0.0f) || scale > 3.0e38f || qk_eps != qk_eps || qk_eps > 3.0e38f) return SDVA_ERR_INVALID;
  if (parent != nullptr && deltas == nullptr && window > 1) return SDVA_ERR_INVALID;  // a tree has no last token
  if (window > kMaxWindow || num_lanes > 65535 || num_v_heads > 65535) return SDVA_ERR_UNSUPPORTED;
  const VerifyArgs a = {state,
                        static_cast<const uint16_t*>(q),
                        static_cast<const uint16_t*>(k),
                        static_cast<const uint16_t*>(v),
                        log_decay,
                        beta,
                        n_lane,
                        parent,
                        slots,
                        static_cast<uint16_t*>(out),
                        deltas,
                        status,
                        q_stride,
                        k_stride,
                        v_stride,
                        num_slots,
                        num_k_heads,
                        num_v_heads,
                        window,
                        scale,
                        qk_eps};
  verify_delta_kernel<<<dim3(num_v_heads, num_lanes), kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}

extern "C" int commit_delta(float* state, int num_slots, const void* k, int64_t k_stride, const float* log_decay,
                            const float* deltas, int num_k_heads, int num_v_heads, int num_lanes, int window,
                            const int32_t* accept_len, const int32_t* path, const int32_t* slots, int32_t* status,
                            sdva_stream_t stream) {
  if (state == nullptr || log_decay == nullptr || deltas == nullptr || accept_len == nullptr || slots == nullptr ||
      num_slots <= 0 || num_k_heads <= 0 || num_v_heads <= 0 || num_lanes <= 0 || window <= 0 ||
      num_v_heads % num_k_heads != 0)
    return SDVA_ERR_INVALID;
  if (!rows_ok(k, k_stride, num_k_heads) || !aligned16(state) || !aligned16(deltas)) return SDVA_ERR_INVALID;
  if (window > kMaxWindow || num_lanes > 65535 || num_v_heads > 65535) return SDVA_ERR_UNSUPPORTED;
  const CommitArgs a = {state, static_cast<const uint16_t*>(k), log_decay, deltas, accept_len, path, slots, status,
                        k_stride, num_slots, num_k_heads, num_v_heads, window};
  commit_delta_kernel<<<dim3(num_v_heads, num_lanes), kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}
