// verify_delta.cu -- verify_delta and commit_delta: the gated delta rule over a
// verify window and the move of a state by the updates that were accepted.
//
// A window's updates and outputs follow from the state S in front of it (the
// notation is delta_common.cuh's): with D_ij the product of e^g on the way from
// slot j (left out) to slot i, 0 where j is no ancestor of i, and a_i that from
// the root on,
//     x_i = b_i (v_i - r_i a_i S k'_i)
//     u   = T x,  T the inverse of 1 + A,  A_ij = b_i r_i r_j D_ij k'_i . k'_j
//     o_i = scale r_q (a_i S q'_i + sum_j P_ij u_j),  P_ij = r_j D_ij q'_i . k'_j
// so that the state is read once for all of a window's rows, and a tree costs
// what a chain does.  Both calls are bound by the state: 64 KB a head, read by
// verify_delta and also written by commit_delta and by a committed window.
//
// verify_delta: a warp has 16 value rows of a head's state in registers, as the
// tensor cores' B operand (and, committed, as their accumulators); its loads are
// the first thing a CTA issues, under which the window's rows are normalised,
// multiplied with each other and T is solved for, 16 columns in 16 lanes.
// commit_delta: fp32 multiply-adds of one row of the state per warp.
#include "delta_common.cuh"

namespace sdva {
namespace {

using namespace delta;

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

constexpr int kRows = kMaxWindow;  // of the tensor cores' tile; rows behind the lane's count are zeros

__device__ __forceinline__ int key_at(int row, int piece) { return row * 256 + ((piece ^ (row & 7)) << 4); }
// 16 x 16 fp16, 32-byte rows: their two pieces change places every four rows
__device__ __forceinline__ int tri_at(int row, int col) {
  return row * 32 + (((col >> 3) ^ ((row >> 2) & 1)) << 4) + (col & 7) * 2;
}

struct VerifySmem {
  alignas(16) uint8_t key[2][kRows * kHeadDim * 2];  // k', q' in fp16
  alignas(16) uint8_t tri[3][kRows * kRows * 2];     // T in two parts, P
  float gram[2][kRows][kRows + 1];                   // k' . k', q' . k'
  alignas(16) float a[kRows][kRows];
  float d[kRows][33];  // D, and a in column 16
  float r[2][kRows];   // factors of k', q'
  float k_own[kRows];  // 1 / sqrt(|k|^2 + eps)
  float fa[kRows], beta[kRows], eg[kRows], fc[kRows], o1[kRows], o2[kRows];
  float t_up, c_up, f;
  int par[kRows];
};

// kWarps warps of 16 value rows each; kCommit: the window's updates go to the state.
template <int kWarps, bool kCommit>
__global__ void __launch_bounds__(kWarps * 32, 16 / kWarps) verify_delta_kernel(VerifyArgs a) {
  constexpr int kThreads = kWarps * 32;
  __shared__ VerifySmem s;
  const int h = blockIdx.y, b = blockIdx.z, th = threadIdx.x, lane = th & 31, warp = th >> 5, W = a.window;
  const int g = lane >> 2, c = lane & 3, kh = h / (a.hv / a.hk);
  const int row16 = (blockIdx.x * kWarps + warp) * 16;  // the warp's first value row
  const bool report = blockIdx.x == 0 && h == 0 && th == 0;
  const size_t row0 = (size_t)b * W;
  int n = a.n_lane != nullptr ? a.n_lane[b] : W;
  const int slot = a.slots[b];
  int wrong = 0;
  if (n < 0 || n > W) {
    wrong = SDVA_STATUS_BAD_COUNT;
  } else if (n > 0 && (slot < 0 || slot >= a.num_slots)) {
    wrong = SDVA_STATUS_BAD_PAGE;
  }
  if (wrong) {
    if (report) raise_status(a.status, wrong);
    n = 0;
  }
  // S[t][m]: value rows 8 t + g, key dims 16 m + 2 c, + 1 and 16 m + 8 + 2 c, + 1
  float2 S[2][8][2];
  float* const st = a.state + ((size_t)(n > 0 ? slot : 0) * a.hv + h) * kStateElems + (size_t)(row16 + g) * kHeadDim + 2 * c;
  if (n > 0) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          S[t][m][i] = *reinterpret_cast<const float2*>(st + (size_t)8 * t * kHeadDim + 16 * m + 8 * i);
  }
  uint32_t v[2][2];  // rows g, g + 8 of the window, value rows 8 t + 2 c, + 1
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t)
      v[i][t] = g + 8 * i < n ? *reinterpret_cast<const uint32_t*>(a.v + (row0 + g + 8 * i) * (size_t)a.v_stride +
                                                                  (size_t)h * kHeadDim + row16 + 8 * t + 2 * c)
                              : 0u;
  int bad = 0;
  if (th < kRows) {
    const bool on = th < n;
    s.eg[th] = on ? expf(a.log_decay[(row0 + th) * a.hv + h]) : 1.0f;
    s.beta[th] = on ? a.beta[(row0 + th) * a.hv + h] : 0.0f;
    const int p = on && a.parent != nullptr && th > 0 ? a.parent[row0 + th] : th - 1;
    bad = on && th > 0 && (p < 0 || p >= th);
    s.par[th] = p;
  }
  // k' and q': 16 threads to a row
#pragma unroll
  for (int x = th; x < 2 * kRows * 16; x += kThreads) {
    const int m = x >> 8, r = (x >> 4) & 15, p = x & 15;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (r < n)
      w = __ldg(reinterpret_cast<const uint4*>((m ? a.q : a.k) + (row0 + r) * (size_t)(m ? a.q_stride : a.k_stride) +
                                               (size_t)kh * kHeadDim) + p);
    uint32_t y[4] = {w.x, w.y, w.z, w.w}, top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(y[i] << 16 & 0x7FFF0000u, y[i] & 0x7FFF0000u));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const Scale sc = scale_of_row(__uint_as_float(top));
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f0 = bf16_lo(y[i]) * sc.down, f1 = bf16_hi(y[i]) * sc.down;
      sq = fmaf(f0, f0, fmaf(f1, f1, sq));
      y[i] = pack_f16x2(f0, f1);
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (p == 0) {
      s.r[m][r] = r < n ? row_factor(sq, a.eps, sc) : 0.0f;
      // small rows by their own sum, where 2^-e would overflow
      if (m == 0) s.k_own[r] = a.eps < 0.0f ? 1.0f : sc.up < 1.0f ? rsqrtf(fmaf(sq * sc.up, sc.up, a.eps)) : s.r[0][r] * sc.down;
    }
    *reinterpret_cast<uint4*>(s.key[m] + key_at(r, p)) = make_uint4(y[0], y[1], y[2], y[3]);
  }
  if (__syncthreads_or(bad)) {
    if (report) raise_status(a.status, SDVA_STATUS_BAD_TREE);
    n = 0;
  }
  const size_t at0 = (row0 * a.hv + h) * kHeadDim + row16 + 2 * c;  // this thread's first output
  const size_t row_out = (size_t)a.hv * kHeadDim;
  if (n == 0) {
    for (int r = g; r < W; r += 8)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        *reinterpret_cast<uint32_t*>(a.out + at0 + r * row_out + 8 * t) = 0u;
        if (!kCommit) *reinterpret_cast<float2*>(a.deltas + at0 + r * row_out + 8 * t) = make_float2(0.0f, 0.0f);
      }
    return;
  }
  const uint32_t kbase = smem_u32(s.key[0]), qbase = smem_u32(s.key[1]);
  const int a_row = lane & 15, a_piece = lane >> 4;
  // the products of rows, one warp for k' and one for q'; D meanwhile by a third where there is one
  if (warp < 2) {
    float acc[2][4] = {};
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t f[4], b0[2], b1[2];
      ldmatrix_x4((warp ? qbase : kbase) + key_at(a_row, 2 * ks + a_piece), f[0], f[1], f[2], f[3]);
      ldmatrix_x4(kbase + key_at((lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)), b0[0], b1[0], b0[1], b1[1]);
      mma_f16_16816(acc[0], f, b0[0], b1[0]);
      mma_f16_16816(acc[1], f, b0[1], b1[1]);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) s.gram[warp][g + (i >> 1) * 8][8 * t + 2 * c + (i & 1)] = acc[t][i];
  }
  if (warp == 2 && lane <= kRows) {
    // lane 16 stands for the state in front of the window, the root's parent
    float d = lane == kRows ? 1.0f : 0.0f;
    for (int i = 0; i < n; ++i) {
      if (a.parent != nullptr && i > 0) d = s.d[s.par[i]][lane];
      d = i == lane ? 1.0f : i < lane && lane < kRows ? 0.0f : d * s.eg[i];
      s.d[i][lane] = d;
    }
  }
  // S q' and S k' need no T
  float sig[2], isig[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float x = 0.0f;
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) x = fmaxf(x, fmaxf(fabsf(S[t][m][i].x), fabsf(S[t][m][i].y)));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
    const Scale sc = scale_of_row(x);
    sig[t] = sc.down, isig[t] = sc.up;
  }
  float sk[2][2][4] = {}, sq[2][4] = {};
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    uint32_t fk[4], fq[4];
    ldmatrix_x4(kbase + key_at(a_row, 2 * m + a_piece), fk[0], fk[1], fk[2], fk[3]);
    ldmatrix_x4(qbase + key_at(a_row, 2 * m + a_piece), fq[0], fq[1], fq[2], fq[3]);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) split_f16(S[t][m][i].x * sig[t], S[t][m][i].y * sig[t], hi[i], lo[i]);
      mma_f16_16816(sk[0][t], fk, hi[0], hi[1]);
      mma_f16_16816(sk[1][t], fk, lo[0], lo[1]);
      mma_f16_16816(sq[t], fq, hi[0], hi[1]);
    }
  }
  __syncthreads();
  if (warp == 0) {
    // T and P: a column to a lane (lanes 16 .. 31 do the same again)
    const int j = lane & 15;
    const float rk = s.r[0][j];
    float p[kRows], top = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float d = i < n ? s.d[i][j] : 0.0f, w = d * rk;
      const float x = s.beta[i] * s.r[0][i] * w * s.gram[0][i][j];
      p[i] = w * s.gram[1][i][j];
      if (d == 0.0f) p[i] = 0.0f;
      top = fmaxf(top, fabsf(p[i]));
      if (lane < kRows) s.a[i][j] = i > j && d != 0.0f ? x : 0.0f;
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const Scale ps = scale_of_row(top);
    if (lane < kRows) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) *reinterpret_cast<__half*>(s.tri[2] + tri_at(i, j)) = __float2half_rn(p[i] * ps.down);
      const float rq = s.r[1][j], fall = j < n ? s.d[j][kRows] : 0.0f;
      s.fa[j] = fall * rk;
      s.o1[j] = a.scale * rq * fall;
      s.o2[j] = a.scale * rq * ps.up;
    }
    __syncwarp();
    float t[kRows];
    top = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (i >= n) {  // rows of the unit matrix, which no update needs
        t[i] = 0.0f;
        continue;
      }
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int l = 0; l < i; l += 4) {
        const float4 r = *reinterpret_cast<const float4*>(&s.a[i][l]);
        x[0] = fmaf(r.x, t[l], x[0]);
        if (l + 1 < i) x[1] = fmaf(r.y, t[l + 1], x[1]);
        if (l + 2 < i) x[2] = fmaf(r.z, t[l + 2], x[2]);
        if (l + 3 < i) x[3] = fmaf(r.w, t[l + 3], x[3]);
      }
      t[i] = i == j ? 1.0f : -((x[0] + x[1]) + (x[2] + x[3]));
      top = fmaxf(top, fabsf(t[i]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const Scale ts = scale_of_row(top);
    if (lane < kRows) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float x = t[i] * ts.down;
        const __half hi = __float2half_rn(x);
        *reinterpret_cast<__half*>(s.tri[0] + tri_at(i, j)) = hi;
        *reinterpret_cast<__half*>(s.tri[1] + tri_at(i, j)) = __float2half_rn(x - __half2float(hi));
      }
    }
    if (lane == 0) s.t_up = ts.up;
    if (kCommit) {  // factors of the updates in the state behind the window, the largest brought to [1, 2)
      const float fc = j < n ? s.d[n - 1][j] * rk : 0.0f;
      float x = fabsf(fc);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
      const Scale cs = scale_of_row(fmaxf(x, 0x1p-60f));  // S times the scales stays in fp32's range
      if (lane < kRows) s.fc[j] = fc * cs.down;
      if (lane == 0) {
        s.c_up = cs.up;
        s.f = s.d[n - 1][kRows];
      }
    }
  }
  __syncthreads();
  // x; its columns' scales leave u, at most 32 x, inside fp16's range, and are no finer than the state needs
  float xs[2][2], xi[2][2];
  uint32_t xh[2][2], xl[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float x[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float up = __shfl_sync(0xffffffffu, isig[t], 4 * (2 * c + i));
      float top = up * 0x1p-40f;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float y = (sk[0][t][2 * r + i] + sk[1][t][2 * r + i]) * up;
        x[r][i] = s.beta[8 * r + g] * ((i ? bf16_hi(v[r][t]) : bf16_lo(v[r][t])) - s.fa[8 * r + g] * y);
        top = fmaxf(top, fabsf(x[r][i]));
      }
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const Scale sc = scale_of_row(top);
      xs[t][i] = sc.down, xi[t][i] = sc.up;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      split_f16(x[r][0] * xs[t][0], x[r][1] * xs[t][1], xh[t][r], xl[t][r]);
      xh[t][r] = transpose8(xh[t][r]);
      xl[t][r] = transpose8(xl[t][r]);
    }
  }
  uint32_t fh[4], fl[4], fp[4];
  {
    const uint32_t tri = smem_u32(s.tri[0]) + tri_at(a_row, 8 * a_piece);
    ldmatrix_x4(tri, fh[0], fh[1], fh[2], fh[3]);
    ldmatrix_x4(tri + kRows * kRows * 2, fl[0], fl[1], fl[2], fl[3]);
    ldmatrix_x4(tri + 2 * kRows * kRows * 2, fp[0], fp[1], fp[2], fp[3]);
  }
  uint32_t ch[4], cl[4];  // the updates with their factors, value rows by tokens
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float u[4] = {}, o[4] = {};
    mma_f16_16816(u, fl, xh[t][0], xh[t][1]);
    mma_f16_16816(u, fh, xl[t][0], xl[t][1]);
    mma_f16_16816(u, fh, xh[t][0], xh[t][1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] *= s.t_up;
    mma_f16_16816(o, fp, transpose8(pack_f16x2(u[0], u[1])), transpose8(pack_f16x2(u[2], u[3])));
    const float up0 = __shfl_sync(0xffffffffu, isig[t], 8 * c), up1 = __shfl_sync(0xffffffffu, isig[t], 8 * c + 4);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = 8 * r + g;
      if (i < W) {
        const float o1 = s.o1[i], o2 = s.o2[i];
        const size_t at = at0 + i * row_out + 8 * t;
        *reinterpret_cast<uint32_t*>(a.out + at) =
            i < n ? pack_bf16x2(fmaf(o1, sq[t][2 * r] * up0, o2 * (o[2 * r] * xi[t][0])),
                                fmaf(o1, sq[t][2 * r + 1] * up1, o2 * (o[2 * r + 1] * xi[t][1])))
                  : 0u;
        if (!kCommit) {
          const float rk = s.k_own[i];
          *reinterpret_cast<float2*>(a.deltas + at) =
              i < n ? make_float2(rk * (u[2 * r] * xi[t][0]), rk * (u[2 * r + 1] * xi[t][1]))
                    : make_float2(0.0f, 0.0f);
        }
      }
    }
    if (kCommit) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float fc = s.fc[8 * r + g];
        split_f16(u[2 * r] * fc, u[2 * r + 1] * fc, ch[2 * r + t], cl[2 * r + t]);
        ch[2 * r + t] = transpose8(ch[2 * r + t]);
        cl[2 * r + t] = transpose8(cl[2 * r + t]);
      }
    }
  }
  if (kCommit) {
    // S as accumulators: value rows g (t = 0) and g + 8 (t = 1), key dims 8 x + 2 c, + 1
    float in[2], back[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float s0 = __shfl_sync(0xffffffffu, xs[t][0], g >> 1), s1 = __shfl_sync(0xffffffffu, xs[t][1], g >> 1);
      const float i0 = __shfl_sync(0xffffffffu, xi[t][0], g >> 1), i1 = __shfl_sync(0xffffffffu, xi[t][1], g >> 1);
      in[t] = g & 1 ? s1 : s0;
      back[t] = g & 1 ? i1 : i0;
    }
    const float f = s.f, c_up = s.c_up;
    const float c_down = 1.0f / c_up;  // a power of two
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      uint32_t k0[2], k1[2];
      ldmatrix_x4_trans(kbase + key_at((lane & 7) + ((lane >> 3) & 1) * 8, 2 * m + (lane >> 4)), k0[0], k1[0], k0[1], k1[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float acc[4] = {S[0][m][i].x * f * in[0] * c_down, S[0][m][i].y * f * in[0] * c_down,
                        S[1][m][i].x * f * in[1] * c_down, S[1][m][i].y * f * in[1] * c_down};
        mma_f16_16816(acc, ch, k0[i], k1[i]);
        mma_f16_16816(acc, cl, k0[i], k1[i]);
        *reinterpret_cast<float2*>(st + 16 * m + 8 * i) = make_float2(acc[0] * c_up * back[0], acc[1] * c_up * back[0]);
        *reinterpret_cast<float2*>(st + (size_t)8 * kHeadDim + 16 * m + 8 * i) =
            make_float2(acc[2] * c_up * back[1], acc[3] * c_up * back[1]);
      }
    }
  }
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

constexpr int kCommitThreads = 256;
constexpr int kCommitRows = 32;  // value rows of a CTA, four to a warp

__global__ void __launch_bounds__(kCommitThreads) commit_delta_kernel(CommitArgs a) {
  constexpr int kPer = kCommitRows / (kCommitThreads / 32);
  const int h = blockIdx.y, b = blockIdx.z, th = threadIdx.x, lane = th & 31, W = a.window;
  const int kh = h / (a.hv / a.hk), r0 = blockIdx.x * kCommitRows;
  __shared__ int at[kMaxWindow];
  __shared__ float eg[kMaxWindow];
  __shared__ float w[kCommitRows][kMaxWindow];
  const bool report = blockIdx.x == 0 && h == 0 && th == 0;
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
  // a warp's rows, four key dims of each to a thread
  float* const st = a.state + ((size_t)slot * a.hv + h) * kStateElems + (size_t)(r0 + (th >> 5) * kPer) * kHeadDim + 4 * lane;
  float4 S[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) S[i] = *reinterpret_cast<const float4*>(st + i * kHeadDim);
  const size_t row0 = (size_t)b * W;
  int wrong = 0;
  if (th < m) {
    const int p = a.path != nullptr ? a.path[row0 + th] : th;
    wrong = p < 0 || p >= W;
    at[th] = p;
    if (!wrong) eg[th] = expf(a.log_decay[(row0 + p) * a.hv + h]);
  }
  if (__syncthreads_or(wrong)) {
    if (report) raise_status(a.status, SDVA_STATUS_BAD_TREE);
    return;
  }
  // products of e^g behind each update, and all of them
  float f = 1.0f;
  for (int x = th; x < m * kCommitRows; x += kCommitThreads) {
    const int j = x / kCommitRows, r = x % kCommitRows;
    float rest = 1.0f;
    for (int i = j + 1; i < m; ++i) rest *= eg[i];
    w[r][j] = rest * a.deltas[((row0 + at[j]) * a.hv + h) * kHeadDim + r0 + r];
  }
  for (int i = 0; i < m; ++i) f *= eg[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) S[i].x *= f, S[i].y *= f, S[i].z *= f, S[i].w *= f;
  for (int j = 0; j < m; ++j) {
    const uint2 kk = __ldg(reinterpret_cast<const uint2*>(a.k + (row0 + at[j]) * (size_t)a.k_stride + (size_t)kh * kHeadDim) + lane);
    const float k0 = bf16_lo(kk.x), k1 = bf16_hi(kk.x), k2 = bf16_lo(kk.y), k3 = bf16_hi(kk.y);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float x = w[(th >> 5) * kPer + i][j];
      S[i].x = fmaf(x, k0, S[i].x), S[i].y = fmaf(x, k1, S[i].y), S[i].z = fmaf(x, k2, S[i].z), S[i].w = fmaf(x, k3, S[i].w);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) *reinterpret_cast<float4*>(st + i * kHeadDim) = S[i];
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
  constexpr int kWarps = 4;
  const dim3 grid(kHeadDim / (16 * kWarps), num_v_heads, num_lanes);
  (deltas == nullptr ? verify_delta_kernel<kWarps, true>
                     : verify_delta_kernel<kWarps, false>)<<<grid, kWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
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
  commit_delta_kernel<<<dim3(kHeadDim / kCommitRows, num_v_heads, num_lanes), kCommitThreads, 0,
                        reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}
