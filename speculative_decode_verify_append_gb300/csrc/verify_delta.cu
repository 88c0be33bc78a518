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
// verify_delta has two kernels.  rows_kernel takes a chain of two or three
// tokens at most, one after the other in fp32: a warp has 16 value rows of a head's state
// in registers, eight lanes to a row, and needs no other warp.
// window_kernel takes up to 16 in the form above: a CTA has a head, a warp 16
// value rows of its state as the tensor cores' B operand (and, committed, as
// their accumulators), copied to shared memory while the window's rows are
// normalised.  Two more warps multiply the rows with each other and solve for T
// and P, a column to a lane, under the products with S.
// T goes to x, and P to u, in tf32 (T and x in two parts, P and u in one, 11 bits
// each): where a token's map expands (beta |k|^2 above 2, which keys that are taken
// as they are may have; decays above 1), T's entries and u range over more than
// fp16 has, and a token owes nothing to the sizes of later ones.  With fp16 parts
// about one power of two for T and one for x, which overflowed there, the same
// calls were 1.5 to 2.5 us shorter.
// commit_delta: fp32 multiply-adds, eight value rows of a state to a warp.
//
// 64 lanes, 16 / 32 heads (134 MB of states), and what a copy's rate would take:
// a plain step 43.6 us (40.4), 16 rows recorded 44.7 (26.4), committed 66.3
// (44.0), the commit of up to 16 updates, 4.7 on average, 52.3 (41.1).  8 lanes of
// 16 rows 7.3 us, one lane's commit 3.5.  A window's CTA lives some 10,500 cycles
// (clock readings in the kernel): the loads take 5,400, S k' and S q' 2,900 (T is
// there by then) and the rest 2,100; with two on an SM, 128 KB are under way.
#include "delta_common.cuh"

namespace sdva {
namespace {

using namespace delta;
using tc::f2_pack;
using tc::f2_unpack;
using tc::ffma2;
using tc::fmul2;

__device__ __forceinline__ float f2_sum(unsigned long long x) {
  const float2 f = f2_unpack(x);
  return f.x + f.y;
}

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


__device__ __forceinline__ int key_at(int row, int piece) { return row * 256 + ((piece ^ (row & 7)) << 4); }
// 16 x 16 fp32: a row's halves change places every two rows, so that four rows' eight bytes of four threads each are in
// different banks
__device__ __forceinline__ int tri_at(int row, int col) { return row * kMaxWindow + (col ^ ((row << 2) & 8)); }

// The lane's rows, and what is wrong with it (then none).  The window's own
// arrays are read without waiting for it; what lies behind the count is dropped.
struct LaneRows {
  int n, slot, wrong;
};
__device__ __forceinline__ LaneRows lane_rows(const VerifyArgs& a, int b) {
  LaneRows r = {a.n_lane != nullptr ? a.n_lane[b] : a.window, a.slots[b], 0};
  if (r.n < 0 || r.n > a.window) {
    r.wrong = SDVA_STATUS_BAD_COUNT;
  } else if (r.n > 0 && (r.slot < 0 || r.slot >= a.num_slots)) {
    r.wrong = SDVA_STATUS_BAD_PAGE;
  }
  if (r.wrong) r.n = r.slot = 0;
  return r;
}

// Tokens that rows_kernel takes.  64 lanes, 16 / 32 heads, us of rows_kernel and of window_kernel: recorded, 1 token 27.3
// and 41.3, 2 35.0 and 41.4, 3 42.4 and 41.5; committed, 1 43.6 and 63.8, 3 57.6 and 64.1, 4 64.0 and 64.3.  Of one
// lane: recorded, 2 3.5 and 5.4, 4 4.8 and 5.4; committed, 3 4.3 and 7.4.
constexpr int kSeqRecorded = 2, kSeqCommitted = 3;
constexpr int kSeqThreads = 128;

// Value rows 4 i + lane / 8 of a warp's 16; key dims 4 (lane & 7) + 32 p.
template <bool kCommit>
__global__ void __launch_bounds__(kSeqThreads) rows_kernel(VerifyArgs a) {
  const int h = blockIdx.y, b = blockIdx.z, th = threadIdx.x, lane = th & 31, W = a.window;
  const int kh = h / (a.hv / a.hk), j = lane & 7, gr = lane >> 3;
  const int row16 = (blockIdx.x * (kSeqThreads / 32) + (th >> 5)) * 16;
  const LaneRows lr = lane_rows(a, b);
  if (lr.wrong && blockIdx.x == 0 && h == 0 && th == 0) raise_status(a.status, lr.wrong);
  const int n = lr.n;
  float* const st = a.state + ((size_t)lr.slot * a.hv + h) * kStateElems + (size_t)(row16 + gr) * kHeadDim + 4 * j;
  unsigned long long S[4][4][2];
  if (n > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float4 x = *reinterpret_cast<const float4*>(st + (size_t)4 * i * kHeadDim + 32 * p);
        S[i][p][0] = f2_pack(x.x, x.y);
        S[i][p][1] = f2_pack(x.z, x.w);
      }
  }
  const int row = row16 + 4 * (j & 3) + gr;  // the value row whose results this thread writes (j < 4)
  for (int t = 0; t < W; ++t) {
    const size_t r = (size_t)b * W + t, at = (r * a.hv + h) * kHeadDim + row;
    if (t >= n) {
      if (j < 4) {
        a.out[at] = 0;
        if (!kCommit) a.deltas[at] = 0.0f;
      }
      continue;
    }
    const uint16_t* const kr = a.k + r * (size_t)a.k_stride + (size_t)kh * kHeadDim + 4 * j;
    const uint16_t* const qr = a.q + r * (size_t)a.q_stride + (size_t)kh * kHeadDim + 4 * j;
    const uint16_t* const vr = a.v + r * (size_t)a.v_stride + (size_t)h * kHeadDim + row16 + gr;
    uint2 kw[4], qw[4];
    float v[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      kw[p] = __ldg(reinterpret_cast<const uint2*>(kr + 32 * p));
      qw[p] = __ldg(reinterpret_cast<const uint2*>(qr + 32 * p));
      v[p] = __uint_as_float((uint32_t)__ldg(vr + 4 * p) << 16);
    }
    const float eg = expf(a.log_decay[r * a.hv + h]), beta = a.beta[r * a.hv + h];
    unsigned long long k2[4][2], q2[4][2], kk2 = 0, qq2 = 0, kq2 = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      k2[p][0] = f2_pack(bf16_lo(kw[p].x), bf16_hi(kw[p].x));
      k2[p][1] = f2_pack(bf16_lo(kw[p].y), bf16_hi(kw[p].y));
      q2[p][0] = f2_pack(bf16_lo(qw[p].x), bf16_hi(qw[p].x));
      q2[p][1] = f2_pack(bf16_lo(qw[p].y), bf16_hi(qw[p].y));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        kk2 = ffma2(k2[p][e], k2[p][e], kk2);
        qq2 = ffma2(q2[p][e], q2[p][e], qq2);
        kq2 = ffma2(k2[p][e], q2[p][e], kq2);
      }
    }
    float sum[11];  // k.k, q.q, k.q, then S k and S q of the four rows
    sum[0] = f2_sum(kk2), sum[1] = f2_sum(qq2), sum[2] = f2_sum(kq2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unsigned long long x = 0, y = 0;
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x = ffma2(S[i][p][e], k2[p][e], x);
          y = ffma2(S[i][p][e], q2[p][e], y);
        }
      sum[3 + i] = f2_sum(x);
      sum[7 + i] = f2_sum(y);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
#pragma unroll
      for (int x = 0; x < 11; ++x) sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], o);
    const float rk = norm_factor(sum[0], a.eps), rq = norm_factor(sum[1], a.eps);
    float w[4], o = 0.0f, mine = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = rk * (beta * (v[i] - rk * eg * sum[3 + i]));
      if ((j & 3) == i) {
        mine = w[i];
        o = a.scale * rq * fmaf(eg, sum[7 + i], w[i] * sum[2]);
      }
    }
    if (j < 4) {
      a.out[at] = (uint16_t)(pack_bf16x2(o, 0.0f) & 0xFFFFu);
      if (!kCommit) a.deltas[at] = mine;
    }
    if (kCommit || t + 1 < n) {
      const unsigned long long eg2 = f2_pack(eg, eg);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned long long w2 = f2_pack(w[i], w[i]);
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int e = 0; e < 2; ++e) S[i][p][e] = ffma2(w2, k2[p][e], fmul2(eg2, S[i][p][e]));
      }
    }
  }
  if (kCommit && n > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 x = f2_unpack(S[i][p][0]), y = f2_unpack(S[i][p][1]);
        *reinterpret_cast<float4*>(st + (size_t)4 * i * kHeadDim + 32 * p) = make_float4(x.x, x.y, y.x, y.y);
      }
  }
}

constexpr int kRows = kMaxWindow;  // of the tensor cores' tile; rows behind the lane's count are zeros
constexpr int kWarps = 8;          // with a part of the state
constexpr int kThreads = (kWarps + 2) * 32;
constexpr int kStateBytes = (int)(kStateElems * sizeof(float));
// From a value row of the state to the next in shared memory: four threads read 64 bytes of a row, eight in one pass
// those of two rows, out of different banks.
constexpr int kStatePitch = kHeadDim * 4 + 64;

struct VerifySmem {
  uint64_t bar[kWarps];  // the copies of each warp's part of the state
  // k', q' in fp16.  Of 16 key dims a B operand's thread c has 4 c .. 4 c + 3 of the
  // state, so that the rows hold dims 0 1 4 5 8 9 12 13, then 2 3 6 7 10 11 14 15.
  alignas(16) uint8_t key[2][kRows * kHeadDim * 2];
  alignas(16) uint8_t v[kRows * kHeadDim * 2];
  alignas(16) float tri[3][kRows * kRows];        // T in two parts of 11 bits, P in one
  float gram[2][kRows][kRows + 1];                // k' . k', q' . k'
  alignas(16) float a[kRows][kRows + 4];          // columns of A
  float d[2][kRows][kRows + 1];                   // D, and a in column 16 (trees); a copy for T and one for P
  alignas(16) float r[2][kRows];                  // factors of k', q'
  alignas(16) float eg[2][kRows];
  alignas(16) float beta[kRows];
  alignas(16) int par[2][kRows];
  float k_own[kRows];  // 1 / sqrt(|k|^2 + eps)
  float fa[kRows], fc[kRows], o1[kRows], o2[kRows];
  float f;
  int never;    // 0: no role's wait ends another's
  int gave_up;  // whether one ran out
};

// Sixteen floats of shared memory, the same for every thread.
__device__ __forceinline__ void load16(const float* p, float (&x)[kRows]) {
#pragma unroll
  for (int i = 0; i < kRows; i += 4) {
    const float4 y = *reinterpret_cast<const float4*>(p + i);
    x[i] = y.x, x[i + 1] = y.y, x[i + 2] = y.z, x[i + 3] = y.w;
  }
}
// D by columns, for each of the two further warps (m): lane j < 16 has column j;
// lane 16 stands for the state in front of the window, the root's parent, so
// that its column is a.  Returns whether a parent is wrong.
__device__ __forceinline__ bool ways(VerifySmem& s, const VerifyArgs& a, int m, int n, size_t row0, int h, int lane,
                                     float (&d)[kRows]) {
  const int j = min(lane, kRows);
  bool bad = false;
  if (lane < kRows) {
    const bool in = lane < a.window, on = lane < n;
    const float ld = in ? a.log_decay[(row0 + lane) * a.hv + h] : 0.0f;
    const float beta = in ? a.beta[(row0 + lane) * a.hv + h] : 0.0f;
    int p = in && a.parent != nullptr ? a.parent[row0 + lane] : lane - 1;
    bad = on && lane > 0 && (p < 0 || p >= lane);
    if (bad || !on) p = max(lane - 1, 0);
    s.eg[m][lane] = on ? expf(ld) : 1.0f;
    if (m == 0) s.beta[lane] = on ? beta : 0.0f;
    s.par[m][lane] = p;
    if (m == 0 && lane == 0) s.never = s.gave_up = 0;
  }
  __syncwarp();
  float x[kRows];
  load16(s.eg[m], x);
  if (a.parent == nullptr) {
    float y = j == kRows ? 1.0f : 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) d[i] = y = i == j ? 1.0f : y * x[i];
  } else {
    int par[kRows];
#pragma unroll
    for (int i = 0; i < kRows; i += 4) {
      const int4 y = *reinterpret_cast<const int4*>(s.par[m] + i);
      par[i] = y.x, par[i + 1] = y.y, par[i + 2] = y.z, par[i + 3] = y.w;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float y = i == 0 ? (j == kRows ? 1.0f : 0.0f) : s.d[m][par[i]][j];
      d[i] = i == j ? 1.0f : i < j && j < kRows ? 0.0f : y * x[i];
      if (lane <= kRows) s.d[m][i][j] = d[i];
    }
  }
  return bad;
}

// What they do behind the barrier: the products of rows (m = 0: k' with k', then
// T; m = 1: q' with k', then P).
template <bool kCommit>
__device__ __forceinline__ void solve(VerifySmem& s, const VerifyArgs& a, int m, int n, int lane, const float (&d)[kRows]) {
  const int g = lane >> 2, c = lane & 3, j = min(lane, kRows);
  const uint32_t kbase = smem_u32(s.key[0]), base = smem_u32(s.key[m]);
  float acc[2][4] = {};
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    uint32_t f[4], b0[2], b1[2];
    ldmatrix_x4(base + key_at(lane & 15, 2 * ks + (lane >> 4)), f[0], f[1], f[2], f[3]);
    ldmatrix_x4(kbase + key_at((lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)), b0[0], b1[0], b0[1], b1[1]);
    mma_f16_16816(acc[0], f, b0[0], b1[0]);
    mma_f16_16816(acc[1], f, b0[1], b1[1]);
  }
  float x[kRows];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) s.gram[m][g + (i >> 1) * 8][8 * t + 2 * c + (i & 1)] = acc[t][i];
  // the factors that go with a: lane 16 has a, lane i gets a_i
  if (lane == kRows) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) (m ? s.o1 : s.fa)[i] = d[i];
  }
  __syncwarp();
  const bool on = lane < kRows;
  const float rk = on ? s.r[0][j] : 0.0f;
  if (m == 1) {
    if (on) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) s.tri[2][tri_at(i, j)] = d[i] != 0.0f ? to_tf32(d[i] * rk * s.gram[1][i][j]) : 0.0f;
      const float rq = a.scale * s.r[1][j];
      s.o1[j] = j < n ? rq * s.o1[j] : 0.0f;
      s.o2[j] = rq;
    }
    return;
  }
  float br[kRows];
  load16(s.beta, x);
  load16(s.r[0], br);
#pragma unroll
  for (int i = 0; i < kRows; ++i) br[i] = on && i > j && d[i] != 0.0f ? br[i] * x[i] * (d[i] * rk) * s.gram[0][i][j & 15] : 0.0f;
  if (on) {
#pragma unroll
    for (int i = 0; i < kRows; i += 4)
      *reinterpret_cast<float4*>(&s.a[j][i]) = make_float4(br[i], br[i + 1], br[i + 2], br[i + 3]);
  }
  __syncwarp();
  // the columns of the inverse of 1 + A: as soon as a row is known it leaves the rows below
#pragma unroll
  for (int i = 0; i < kRows; ++i) x[i] = i == j ? 1.0f : 0.0f;
#pragma unroll
  for (int l = 0; l < kRows - 1; ++l) {
#pragma unroll
    for (int i = (l + 1) & ~3; i < kRows; i += 4) {
      const float4 y = *reinterpret_cast<const float4*>(&s.a[l][i]);
      if (i > l) x[i] = fmaf(-y.x, x[l], x[i]);
      if (i + 1 > l) x[i + 1] = fmaf(-y.y, x[l], x[i + 1]);
      if (i + 2 > l) x[i + 2] = fmaf(-y.z, x[l], x[i + 2]);
      x[i + 3] = fmaf(-y.w, x[l], x[i + 3]);
    }
  }
  if (on) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) split_tf32(x[i], s.tri[0][tri_at(i, j)], s.tri[1][tri_at(i, j)]);
    s.fa[j] = j < n ? s.fa[j] * rk : 0.0f;
  }
  if (kCommit) {  // factors of the updates in the state behind the window
    float fc = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (i == n - 1) fc = d[i];
    if (lane == kRows) s.f = fc;
    if (on) s.fc[j] = j < n ? fc * rk : 0.0f;
  }
}

// kCommit: the window's updates go to the state.
template <bool kCommit>
__global__ void __launch_bounds__(kThreads, 2) window_kernel(VerifyArgs a, long long limit) {
  __shared__ VerifySmem s;
  const int h = blockIdx.x, b = blockIdx.y, th = threadIdx.x, lane = th & 31, warp = th >> 5, W = a.window;
  const int g = lane >> 2, c = lane & 3, kh = h / (a.hv / a.hk);
  const int row16 = warp * 16;  // the warp's first value row
  const bool report = h == 0 && th == 0;
  const size_t row0 = (size_t)b * W;
  const LaneRows lr = lane_rows(a, b);
  int n = lr.n;
  if (lr.wrong && report) raise_status(a.status, lr.wrong);
  // The window's rows (16 threads to a row), the state by bulk copies: loads
  // through L1 come back in order, and the little ones of both CTAs of an SM would
  // wait for 64 KB each time.
  const int r_row = th >> 4, r_piece = th & 15;
  uint4 rows[2] = {};
  if (r_row < W) {  // 16 rows of the first eight warps
#pragma unroll
    for (int m = 0; m < 2; ++m)
      rows[m] = __ldg(reinterpret_cast<const uint4*>((m ? a.q : a.k) + (row0 + r_row) * (size_t)(m ? a.q_stride : a.k_stride) +
                                                     (size_t)kh * kHeadDim) + r_piece);
    cp_async_16(smem_u32(s.v) + key_at(r_row, r_piece),
                a.v + (row0 + r_row) * (size_t)a.v_stride + (size_t)h * kHeadDim + 8 * r_piece);
  }
  cp_async_commit();
  extern __shared__ __align__(128) uint8_t state_smem[];
  const uint8_t* const mine = state_smem + warp * 16 * kStatePitch;
  float* const st = a.state + ((size_t)lr.slot * a.hv + h) * kStateElems + (size_t)row16 * kHeadDim;
  const uint32_t bar = smem_u32(&s.bar[warp & (kWarps - 1)]);
  float d[kRows];         // of the two further warps
  bool bad = false;
  if (warp < kWarps) {
    if (n > 0) {
      if (lane == 0) {
        tc::mbar_init(bar, 1);
        tc::mbar_fence_init();
        tc::mbar_arrive_expect_tx(bar, kStateBytes / kWarps);
      }
      __syncwarp();
      if (lane < 16) tc::bulk_load(smem_u32(mine) + lane * kStatePitch, st + (size_t)lane * kHeadDim, kHeadDim * 4, bar);
    }
  } else {
    bad = ways(s, a, warp - kWarps, n, row0, h, lane, d);
  }
  if (warp < kWarps) {
    const int r = r_row, p = r_piece;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint4 w = r < n ? rows[m] : make_uint4(0u, 0u, 0u, 0u);
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
        const float f = r < n ? row_factor(sq, a.eps, sc) : 0.0f;
        s.r[m][r] = f;
        // small rows by their own sum, where 2^-e would overflow
        if (m == 0) s.k_own[r] = a.eps < 0.0f ? 1.0f : sc.up < 1.0f ? rsqrtf(fmaf(sq * sc.up, sc.up, a.eps)) : f * sc.down;
      }
      uint8_t* const to = s.key[m] + 8 * (p & 1);
      *reinterpret_cast<uint2*>(to + key_at(r, p & ~1)) = make_uint2(y[0], y[2]);
      *reinterpret_cast<uint2*>(to + key_at(r, p | 1)) = make_uint2(y[1], y[3]);
    }
  }
  if (__syncthreads_or(bad)) {
    if (report) raise_status(a.status, SDVA_STATUS_BAD_TREE);
    n = 0;
  }
  const size_t at0 = (row0 * a.hv + h) * kHeadDim + row16 + 2 * c;  // this thread's first output
  const size_t row_out = (size_t)a.hv * kHeadDim;
  if (n == 0) {
    if (warp < kWarps && lr.n > 0) copies_here(bar, 0, &s.never, limit);
    cp_async_wait<0>();  // v: no copy outlives the CTA
    if (warp < kWarps)
      for (int r = g; r < W; r += 8)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          *reinterpret_cast<uint32_t*>(a.out + at0 + r * row_out + 8 * t) = 0u;
          if (!kCommit) *reinterpret_cast<float2*>(a.deltas + at0 + r * row_out + 8 * t) = make_float2(0.0f, 0.0f);
        }
    return;
  }
  if (warp >= kWarps) {
    solve<kCommit>(s, a, warp - kWarps, n, lane, d);
    __syncthreads();
    return;
  }
  const uint32_t kbase = smem_u32(s.key[0]), qbase = smem_u32(s.key[1]);
  const int a_row = lane & 15, a_piece = lane >> 4;
  if (!copies_here(bar, 0, &s.never, limit)) {
    raise_status(a.status, SDVA_STATUS_TIMEOUT);
    s.gave_up = 1;
  }
  // S k' in two parts, S q' in one; of the state value rows 8 t + g, key dims 16 m + 4 c ..
  const auto state_of = [&](int t, int m) {
    return *reinterpret_cast<const float4*>(mine + (8 * t + g) * kStatePitch + 64 * m + 16 * c);
  };
  float4 S[2][8];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int m = 0; m < 8; ++m) S[t][m] = state_of(t, m);
  float sig[2], isig[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float x = 0.0f;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const float4 y = S[t][m];
      x = max3(x, fabsf(y.x), fabsf(y.y));
      x = max3(x, fabsf(y.z), fabsf(y.w));
    }
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
    const Scale sc = scale_to_top(x);
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
      const float4 y = S[t][m];
      split_f16(f2_unpack(fmul2(f2_pack(y.x, y.y), f2_pack(sig[t], sig[t]))), hi[0], lo[0]);
      split_f16(f2_unpack(fmul2(f2_pack(y.z, y.w), f2_pack(sig[t], sig[t]))), hi[1], lo[1]);
      mma_f16_16816(sk[0][t], fk, hi[0], hi[1]);
      mma_f16_16816(sk[1][t], fk, lo[0], lo[1]);
      mma_f16_16816(sq[t], fq, hi[0], hi[1]);
    }
  }
  cp_async_wait<0>();  // v
  __syncthreads();
  // T and P, of columns 8 kt + 2 c and + 1 of rows g and g + 8: the k indices c and c + 4 of a product are the tokens
  // 2 c and 2 c + 1 in both operands
  float th_[2][4], tl[2][4], p[2][4];
#pragma unroll
  for (int kt = 0; kt < 2; ++kt)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int at = tri_at(8 * r + g, 8 * kt + 2 * c);
      const float2 x = *reinterpret_cast<const float2*>(&s.tri[0][at]), y = *reinterpret_cast<const float2*>(&s.tri[1][at]);
      const float2 z = *reinterpret_cast<const float2*>(&s.tri[2][at]);
      th_[kt][r] = x.x, th_[kt][2 + r] = x.y;
      tl[kt][r] = y.x, tl[kt][2 + r] = y.y;
      p[kt][r] = z.x, p[kt][2 + r] = z.y;
    }
  // x and u as they are: T's entries and the tokens' values have sizes of their own, which fp16 would need a scale for
  uint32_t ch[4], cl[4];  // the updates with their factors, value rows by tokens
  float in[2], back[2];   // their scale
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float x[2][2];
    uint32_t v[2];  // rows g, g + 8 of the window, value rows 8 t + 2 c, + 1
    float up[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) up[i] = __shfl_sync(0xffffffffu, isig[t], 4 * (2 * c + i));
    float u[4] = {}, u1[4] = {}, u2[4] = {}, o[4] = {};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 8 * r + g;
      v[r] = row < n ? *reinterpret_cast<const uint32_t*>(s.v + key_at(row, 2 * warp + t) + 4 * c) : 0u;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float y = (sk[0][t][2 * r + i] + sk[1][t][2 * r + i]) * up[i];
        x[r][i] = s.beta[row] * ((i ? bf16_hi(v[r]) : bf16_lo(v[r])) - s.fa[row] * y);
      }
      transpose8(x[r][0], x[r][1]);
      float hi[2], lo[2];
      split_tf32(x[r][0], hi[0], lo[0]);
      split_tf32(x[r][1], hi[1], lo[1]);
      mma_tf32_1688(u, th_[r], hi[0], hi[1]);
      mma_tf32_1688(u1, tl[r], hi[0], hi[1]);
      mma_tf32_1688(u2, th_[r], lo[0], lo[1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] += u1[i] + u2[i];
    if (!kCommit) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = 8 * r + g;
        const float rk = s.k_own[i];
        if (i < W)
          *reinterpret_cast<float2*>(a.deltas + at0 + i * row_out + 8 * t) =
              i < n ? make_float2(rk * u[2 * r], rk * u[2 * r + 1]) : make_float2(0.0f, 0.0f);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      transpose8(u[2 * r], u[2 * r + 1]);  // value row 8 t + g, tokens 8 r + 2 c, + 1
      mma_tf32_1688(o, p[r], to_tf32(u[2 * r]), to_tf32(u[2 * r + 1]));
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = 8 * r + g;
      if (i < W) {
        const float o1 = s.o1[i], o2 = s.o2[i];
        *reinterpret_cast<uint32_t*>(a.out + at0 + i * row_out + 8 * t) =
            i < n ? pack_bf16x2(fmaf(o1, sq[t][2 * r] * up[0], o2 * o[2 * r]),
                                fmaf(o1, sq[t][2 * r + 1] * up[1], o2 * o[2 * r + 1]))
                  : 0u;
      }
    }
    if (kCommit) {
      // fp16's range from the largest of a value row; S in that scale stays in fp32's
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] *= s.fc[8 * (i >> 1) + 2 * c + (i & 1)];
        top = fmaxf(top, fabsf(u[i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const Scale sc = scale_to_top(fmaxf(top, s.f * isig[t] * 0x1p-40f));
      in[t] = sc.down, back[t] = sc.up;
#pragma unroll
      for (int r = 0; r < 2; ++r) split_f16(u[2 * r] * in[t], u[2 * r + 1] * in[t], ch[2 * r + t], cl[2 * r + t]);
    }
  }
  if (kCommit && s.gave_up == 0) {  // else the head keeps its state
    // S as accumulators: value rows g (t = 0) and g + 8 (t = 1), columns as the rows of k' have their dims
    const float f = s.f;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      uint32_t k0[2], k1[2];
      ldmatrix_x4_trans(kbase + key_at((lane & 7) + ((lane >> 3) & 1) * 8, 2 * m + (lane >> 4)), k0[0], k1[0], k0[1], k1[1]);
      const float4 s0 = state_of(0, m), s1 = state_of(1, m);
      // f first: of a row of zeros in front and behind, in is at its end, and its product with f may be infinite
      float lo[4] = {s0.x * f * in[0], s0.y * f * in[0], s1.x * f * in[1], s1.y * f * in[1]};
      float hi[4] = {s0.z * f * in[0], s0.w * f * in[0], s1.z * f * in[1], s1.w * f * in[1]};
      mma_f16_16816(lo, ch, k0[0], k1[0]);
      mma_f16_16816(hi, ch, k0[1], k1[1]);
      mma_f16_16816(lo, cl, k0[0], k1[0]);
      mma_f16_16816(hi, cl, k0[1], k1[1]);
#pragma unroll
      for (int t = 0; t < 2; ++t)
        *reinterpret_cast<float4*>(st + (size_t)(8 * t + g) * kHeadDim + 16 * m + 4 * c) =
            make_float4(lo[2 * t] * back[t], lo[2 * t + 1] * back[t], hi[2 * t] * back[t], hi[2 * t + 1] * back[t]);
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

constexpr int kCommitThreads = 128;
constexpr int kCommitRows = 32;  // value rows of a CTA, eight to a warp

__global__ void __launch_bounds__(kCommitThreads) commit_delta_kernel(CommitArgs a) {
  constexpr int kPer = kCommitRows / (kCommitThreads / 32);
  const int h = blockIdx.y, b = blockIdx.z, th = threadIdx.x, lane = th & 31, W = a.window;
  const int kh = h / (a.hv / a.hk), r0 = blockIdx.x * kCommitRows;
  __shared__ alignas(16) float w[kMaxWindow][kCommitRows];
  __shared__ alignas(16) uint16_t key[kMaxWindow][kHeadDim];
  const bool report = blockIdx.x == 0 && h == 0 && th == 0;
  const int m = a.accept_len[b] + 1, slot = a.slots[b];
  const size_t row0 = (size_t)b * W;
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
  unsigned long long S[kPer][2];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float4 x = *reinterpret_cast<const float4*>(st + i * kHeadDim);
    S[i][0] = f2_pack(x.x, x.y);
    S[i][1] = f2_pack(x.z, x.w);
  }
  // committed slot j's update (eight threads) and key (sixteen), and in every warp's lane j its e^g
  const auto slot_of = [&](int j) { return a.path != nullptr ? a.path[row0 + j] : j; };
  bool wrong = false;
  float eg = 1.0f;
  if (lane < m) {
    const int p = slot_of(lane);
    wrong = p < 0 || p >= W;
    if (!wrong) eg = expf(a.log_decay[(row0 + p) * a.hv + h]);
  }
  {
    const int j = th >> 3, p = j < m ? slot_of(j) : -1;
    if (p >= 0 && p < W)
      *reinterpret_cast<float4*>(&w[j][4 * (th & 7)]) =
          __ldg(reinterpret_cast<const float4*>(a.deltas + ((row0 + p) * a.hv + h) * kHeadDim + r0) + (th & 7));
  }
#pragma unroll
  for (int x = th; x < kMaxWindow * 16; x += kCommitThreads) {
    const int j = x >> 4, p = j < m ? slot_of(j) : -1;
    if (p >= 0 && p < W)
      *reinterpret_cast<uint4*>(&key[j][8 * (x & 15)]) =
          __ldg(reinterpret_cast<const uint4*>(a.k + (row0 + p) * (size_t)a.k_stride + (size_t)kh * kHeadDim) + (x & 15));
  }
  if (__syncthreads_or(wrong)) {
    if (report) raise_status(a.status, SDVA_STATUS_BAD_TREE);
    return;
  }
  // products of e^g behind each update, and all of them
  float rest = __shfl_down_sync(0xffffffffu, eg, 1);
  if (lane == 31) rest = 1.0f;
#pragma unroll
  for (int o = 1; o < kMaxWindow; o <<= 1) {
    const float x = __shfl_down_sync(0xffffffffu, rest, o);
    if (lane + o < 32) rest *= x;
  }
  const float f = __shfl_sync(0xffffffffu, rest * eg, 0);
  const unsigned long long f2 = f2_pack(f, f);
#pragma unroll
  for (int i = 0; i < kPer; ++i) S[i][0] = fmul2(S[i][0], f2), S[i][1] = fmul2(S[i][1], f2);
  for (int j = 0; j < m; ++j) {
    const float cj = __shfl_sync(0xffffffffu, rest, j);
    const uint2 kk = *reinterpret_cast<const uint2*>(&key[j][4 * lane]);
    const unsigned long long k0 = f2_pack(cj * bf16_lo(kk.x), cj * bf16_hi(kk.x));
    const unsigned long long k1 = f2_pack(cj * bf16_lo(kk.y), cj * bf16_hi(kk.y));
    const float4* const wj = reinterpret_cast<const float4*>(&w[j][(th >> 5) * kPer]);
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const float4 x = wj[i];
      const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned long long w2 = f2_pack(y[e], y[e]);
        S[4 * i + e][0] = ffma2(w2, k0, S[4 * i + e][0]);
        S[4 * i + e][1] = ffma2(w2, k1, S[4 * i + e][1]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float2 x = f2_unpack(S[i][0]), y = f2_unpack(S[i][1]);
    *reinterpret_cast<float4*>(st + i * kHeadDim) = make_float4(x.x, x.y, y.x, y.y);
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
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (window <= (deltas != nullptr ? kSeqRecorded : kSeqCommitted) && parent == nullptr) {
    const dim3 grid(kHeadDim / (16 * (kSeqThreads / 32)), num_v_heads, num_lanes);
    (deltas == nullptr ? rows_kernel<true> : rows_kernel<false>)<<<grid, kSeqThreads, 0, cs>>>(a);
  } else {
    const dim3 grid(num_v_heads, num_lanes);
    const auto kernel = deltas == nullptr ? window_kernel<true> : window_kernel<false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWarps * 16 * kStatePitch) != cudaSuccess)
      return SDVA_ERR_CUDA;
    kernel<<<grid, kThreads, kWarps * 16 * kStatePitch, cs>>>(a, wait_limit());
  }
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
