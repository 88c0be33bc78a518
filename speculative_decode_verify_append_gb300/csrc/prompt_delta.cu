// prompt_delta.cu -- the gated delta rule over packed prompts of different
// lengths, which leaves each lane's state behind its last token.
//
// Chunks of 32 tokens.  With S the state in front of a chunk, D_ij the product
// of e^g over the tokens j + 1 .. i, a_i that over all tokens up to i and f the
// one over the whole chunk (notation of delta_common.cuh):
//     x_i = b_i (v_i - r_i a_i S k'_i)
//     u   = T x,  T the inverse of 1 + A,  A_ij = b_i r_i r_j D_ij k'_i . k'_j  (j < i)
//     o_i = scale r_q (a_i S q'_i + sum_j<=i P_ij u_j),  P_ij = r_j D_ij q'_i . k'_j
//     S  <- f S + sum_j (f / a_j) r_j u_j k'_j'
// D comes from products of e^g, never from differences of sums, so that a decay
// of 0 (a log decay of -inf) is as good as any.
//
// Two kernels.  chunk_kernel, a CTA per chunk and key head, writes what does
// not depend on the state: k' and q' in fp16, T in two parts, P, and each
// token's factors, laid out as the other kernel's shared memory holds them.
// state_kernel goes through a lane's chunks with a head's state in registers.
// A warp has eight value columns of it and works alone: S as 16 x 8 accumulators
// (key dims by values) becomes the B operand of S k' by transposing 8 x 8 tiles
// between registers, and so do x and u.  This chain, state to state, is what a
// long prompt's time is made of (a prompt alone has 16 such warps per head), so
// that nothing else is on it: each of its warps has another one, a chunk behind,
// that takes S and u out of shared memory, makes the outputs, and copies the
// chunks that come.  One barrier of the CTA per chunk.
#include "delta_common.cuh"

namespace sdva {
namespace {

using namespace delta;

constexpr int kChunk = 32;
// A chunk's records in the workspace and in shared memory (bytes).  16-byte
// pieces of a row are stored at piece ^ (row & 7) (k', q': 256-byte rows) and
// piece ^ (row / 2 & 3) (T, P by columns: 64 bytes each), so that eight rows of a matrix load
// fall into different banks.
constexpr int kKeyBytes = kChunk * kHeadDim * 2;
constexpr int kTriBytes = kChunk * kChunk * 2;
constexpr int kKeyRecord = 2 * kKeyBytes;  // k', q' of a key head
constexpr int kFactors = 5;                // per token: a r, b, (f / a) r, scale r_q a, scale r_q / (P's scale)
constexpr int kScalars = 8;
constexpr int kFactorBytes = (kFactors * kChunk + kScalars) * 4;
constexpr int kHeadRecord = 3 * kTriBytes + kFactorBytes;  // T hi, T lo, P, factors of a value head
static_assert(kHeadRecord % 16 == 0, "records are copied 16 bytes at a time");
// A chunk's scalars: f, and bounds of what the chunk can grow to
enum { kF = 0, kSumA = 1, kMaxB = 2, kSumT = 3, kMaxC = 4, kSumC = 5, kTUp = 6 };

__device__ __forceinline__ int key_at(int row, int piece) { return row * 256 + ((piece ^ (row & 7)) << 4); }
__device__ __forceinline__ int tri_at(int row, int piece) { return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4); }

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
  uint8_t* keys;   // [chunk slots][hk][kKeyRecord]
  uint8_t* heads;  // [chunk slots][hv][kHeadRecord]
  long long q_stride, k_stride, v_stride;
  int num_slots, hk, hv, num_lanes, total;
  float scale, eps;
};

// First chunk slot of a lane whose rows start at row `at`: a lane of n tokens
// has at most n / 32 + 1 chunks, and the next lane's base is at least as far.
__host__ __device__ __forceinline__ int chunk_base(int at, int lane) { return at / kChunk + lane; }

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A column of T or P; what fp16 leaves over into the next matrix.
template <bool kParts>
__device__ __forceinline__ void store_column(uint8_t* to, int j, const float (&x)[kChunk], float scale) {
#pragma unroll
  for (int p = 0; p < kChunk / 8; ++p) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_f16(x[8 * p + 2 * i] * scale, x[8 * p + 2 * i + 1] * scale, hi[i], lo[i]);
    *reinterpret_cast<uint4*>(to + tri_at(j, p)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (kParts) *reinterpret_cast<uint4*>(to + kTriBytes + tri_at(j, p)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

constexpr int kChunkThreads = 128;

struct ChunkSmem {
  alignas(16) uint8_t key[2][kKeyBytes];      // k', q'
  float gram[2][kChunk][kChunk + 4];          // k' . k', q' . k' (row, column)
  alignas(16) float a[4][kChunk][kChunk + 4];  // A of each warp's value head
  float sum_sq[2][kChunk], up[2][kChunk], down[2][kChunk], l1[kChunk], top[kChunk];
  uint32_t found[kChunkThreads / 32];
};

__global__ void __launch_bounds__(kChunkThreads) chunk_kernel(PromptArgs a) {
  __shared__ ChunkSmem s;
  const int slot = blockIdx.x, kh = blockIdx.y, th = threadIdx.x, lane = th & 31, warp = th >> 5;
  constexpr uint32_t kBad = 1u << 20;  // above every count: the host refuses more lanes than 65,535
  uint32_t found = 0;
  bool bad = false;
  for (int b = th; b < a.num_lanes; b += kChunkThreads) {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    bad |= lo < 0 || hi < lo || hi > a.total;
    found += chunk_base(lo, b) <= slot;
  }
  found = __reduce_add_sync(0xffffffffu, found + (bad ? kBad : 0u));
  if (lane == 0) s.found[warp] = found;
  __syncthreads();
  found = 0;
#pragma unroll
  for (int w = 0; w < kChunkThreads / 32; ++w) found += s.found[w];
  if (found >= kBad || found == 0) return;  // the other kernel reports it
  const int b = (int)found - 1;
  const int t0 = a.cu[b] + (slot - chunk_base(a.cu[b], b)) * kChunk;
  const int valid = min(a.cu[b + 1] - t0, kChunk);
  if (valid <= 0) return;

  // k' and q': four threads to a row, 16-byte pieces p, p + 4, p + 8, p + 12
  {
    const int r = th >> 2, p = th & 3;
    uint8_t* const rec = a.keys + ((size_t)slot * a.hk + kh) * kKeyRecord;
    uint4 w[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint16_t* const src = (m ? a.q : a.k) + ((size_t)t0 + r) * (size_t)(m ? a.q_stride : a.k_stride) +
                                  (size_t)kh * kHeadDim;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[m][i] = r < valid ? __ldcs(reinterpret_cast<const uint4*>(src) + p + 4 * i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint32_t x[16];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[4 * i] = w[m][i].x, x[4 * i + 1] = w[m][i].y, x[4 * i + 2] = w[m][i].z, x[4 * i + 3] = w[m][i].w;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, max(x[i] << 16 & 0x7FFF0000u, x[i] & 0x7FFF0000u));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const Scale sc = scale_of_row(__uint_as_float(top));
      float sq = 0.0f, l1 = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float f0 = bf16_lo(x[i]) * sc.down, f1 = bf16_hi(x[i]) * sc.down;
        sq = fmaf(f0, f0, fmaf(f1, f1, sq));
        l1 += fabsf(f0) + fabsf(f1);
        x[i] = pack_f16x2(f0, f1);
      }
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        sq += __shfl_xor_sync(0xffffffffu, sq, o);
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
      }
      if (p == 0) {
        s.sum_sq[m][r] = sq;
        s.up[m][r] = sc.up;
        s.down[m][r] = sc.down;
        if (m == 0) {
          s.l1[r] = l1;
          s.top[r] = __uint_as_float(top) * sc.down;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 y = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        const int at = key_at(r, p + 4 * i);
        *reinterpret_cast<uint4*>(s.key[m] + at) = y;
        *reinterpret_cast<uint4*>(rec + m * kKeyBytes + at) = y;
      }
    }
  }
  __syncthreads();
  // the products of rows: warp w has rows 16 (w & 1) .. of k' (w < 2) or q'
  {
    const int mt = warp & 1, m = warp >> 1, g = lane >> 2, c = lane & 3;
    float acc[4][4] = {};
    const uint32_t base = smem_u32(s.key[m]), kbase = smem_u32(s.key[0]);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t f[4], b0[4], b1[4];
      ldmatrix_x4(base + key_at(16 * mt + (lane & 15), 2 * ks + (lane >> 4)), f[0], f[1], f[2], f[3]);
#pragma unroll
      for (int n = 0; n < 2; ++n)  // B: rows 16 n .. of k', both halves of the key dims
        ldmatrix_x4(kbase + key_at(16 * n + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)), b0[2 * n],
                    b1[2 * n], b0[2 * n + 1], b1[2 * n + 1]);
#pragma unroll
      for (int n = 0; n < 4; ++n)
        if (n < 2 * mt + 2) mma_f16_16816(acc[n], f, b0[n], b1[n]);
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s.gram[m][16 * mt + g + (i >> 1) * 8][8 * n + 2 * c + (i & 1)] = acc[n][i];
  }
  __syncthreads();
  // T, and P with the factors, of the key head's value heads: a task per warp, a column to a lane, and token `lane`
  const int group = a.hv / a.hk;
  const bool on = lane < valid;
  const Scale sk = {s.down[0][lane], s.up[0][lane]}, sq = {s.down[1][lane], s.up[1][lane]};
  const float rk = on ? row_factor(s.sum_sq[0][lane], a.eps, sk) : 0.0f;
  const float rq = on ? row_factor(s.sum_sq[1][lane], a.eps, sq) : 0.0f;
  for (int task = warp; task < 2 * group; task += kChunkThreads / 32) {
    const int h = kh * group + (task >> 1);
    uint8_t* const rec = a.heads + ((size_t)slot * a.hv + h) * kHeadRecord;
    float* const fac = reinterpret_cast<float*>(rec + 3 * kTriBytes);
    const size_t at = ((size_t)t0 + lane) * a.hv + h;
    const float eg = on ? expf(a.log_decay[at]) : 1.0f, beta = on ? a.beta[at] : 0.0f;
    float x[kChunk], d = 0.0f, top = 0.0f;
    if (task & 1) {
      // products of e^g up to this token, and from the next one on
      float fall = eg, rest = __shfl_down_sync(0xffffffffu, eg, 1);
      if (lane == 31) rest = 1.0f;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, fall, o), z = __shfl_down_sync(0xffffffffu, rest, o);
        if (lane >= o) fall *= y;
        if (lane + o < 32) rest *= z;
      }
      const float all = __shfl_sync(0xffffffffu, fall, 31);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        const float egi = __shfl_sync(0xffffffffu, eg, i);
        d = i == lane ? 1.0f : d * egi;
        x[i] = i >= lane ? d * rk * s.gram[1][i][lane] : 0.0f;
        top = fmaxf(top, fabsf(x[i]));
      }
      const Scale ps = scale_of_row(warp_max(top));
      store_column<false>(rec + 2 * kTriBytes, lane, x, ps.down);
      const float fa = fall * rk, fc = rest * rk;
      fac[lane] = fa;
      fac[kChunk + lane] = beta;
      fac[2 * kChunk + lane] = fc;
      fac[3 * kChunk + lane] = a.scale * rq * fall;
      fac[4 * kChunk + lane] = a.scale * rq * ps.up;
      const float sum_a = warp_max(fabsf(fa) * s.l1[lane]), max_b = warp_max(fabsf(beta)), max_c = warp_max(fabsf(fc));
      const float sum_c = warp_sum(fabsf(fc) * s.top[lane]);
      if (lane == 0) {
        float* const g = fac + kFactors * kChunk;
        g[kF] = all;
        g[kSumA] = sum_a;
        g[kMaxB] = max_b;
        g[kMaxC] = max_c;
        g[kSumC] = sum_c;
      }
      continue;
    }
    // A by columns, then those of the inverse of 1 + A: as soon as a row is known it leaves the rows below
    float (*const A)[kChunk + 4] = s.a[warp];
    const float br = beta * rk;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const float egi = __shfl_sync(0xffffffffu, eg, i), bri = __shfl_sync(0xffffffffu, br, i);
      d = i == lane ? 1.0f : d * egi;
      x[i] = i > lane ? bri * (d * rk) * s.gram[0][i][lane] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kChunk; i += 4) *reinterpret_cast<float4*>(&A[lane][i]) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kChunk; ++i) x[i] = i == lane ? 1.0f : 0.0f;
#pragma unroll
    for (int l = 0; l < kChunk - 1; ++l) {
#pragma unroll
      for (int i = (l + 1) & ~3; i < kChunk; i += 4) {
        const float4 y = *reinterpret_cast<const float4*>(&A[l][i]);
        if (i > l) x[i] = fmaf(-y.x, x[l], x[i]);
        if (i + 1 > l) x[i + 1] = fmaf(-y.y, x[l], x[i + 1]);
        if (i + 2 > l) x[i + 2] = fmaf(-y.z, x[l], x[i + 2]);
        x[i + 3] = fmaf(-y.w, x[l], x[i + 3]);
      }
    }
#pragma unroll
    for (int i = 0; i < kChunk; ++i) top = fmaxf(top, fabsf(x[i]));
    top = warp_max(top);
    const Scale ts = scale_of_row(top);
    store_column<true>(rec, lane, x, ts.down);
    if (lane == 0) {
      float* const g = fac + kFactors * kChunk;
      g[kSumT] = top * kChunk;
      g[kTUp] = ts.up;
    }
  }
}

constexpr int kWarps = 4;     // of the chain, eight value columns each
constexpr int kStages = 3;    // the outputs' chunk, the chain's, and the one that comes
constexpr int kThreads = 2 * kWarps * 32;
constexpr int kValueBytes = kChunk * kWarps * 16;  // the chunk's values of the CTA's columns
constexpr int kStageBytes = kKeyRecord + kHeadRecord + kValueBytes;
// What a warp of the chain hands over: S (16 words a thread), u (4), the scales of both (4)
constexpr int kHandBytes = 6 * 32 * 16;
constexpr int kStateSmem = kStages * kStageBytes + 2 * kWarps * kHandBytes;

// A column of T or P in A's place: rows are stored by columns, so the matrices come transposed.
__device__ __forceinline__ uint32_t tri_a(uint32_t tri, int m, int jt, int lane) {
  return tri + tri_at(16 * jt + (lane & 7) + ((lane >> 4) << 3), 2 * m + ((lane >> 3) & 1));
}
__device__ __forceinline__ int value_at(int row, int piece) {
  return (row * kWarps + (piece ^ ((row >> 1) & (kWarps - 1)))) << 4;
}

__global__ void __launch_bounds__(kThreads, 2) state_kernel(PromptArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int th = threadIdx.x, lane = th & 31, g = lane >> 2, c = lane & 3;
  const bool chain = th < kWarps * 32;
  const int warp = (th >> 5) & (kWarps - 1);
  const int h = blockIdx.y, kh = h / (a.hv / a.hk);
  bool bad = false;
  for (int i = th; i < a.num_lanes; i += kThreads) {
    const int lo = a.cu[i], hi = a.cu[i + 1];
    bad |= lo < 0 || hi < lo || hi > a.total;
  }
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && h == 0 && blockIdx.z == 0 && th == 0) raise_status(a.status, SDVA_STATUS_BAD_COUNT);
    return;
  }
  const int b = blockIdx.z;
  const bool report = blockIdx.x == 0 && h == 0 && th == 0;
  const int row0 = a.cu[b], n = a.cu[b + 1] - row0;
  if (n == 0) return;
  const int slot = a.slots[b], L = a.seq_lens != nullptr ? a.seq_lens[b] : 1;
  if (L < 0 || slot < 0 || slot >= a.num_slots) {
    if (report) raise_status(a.status, L < 0 ? SDVA_STATUS_OVERFLOW : SDVA_STATUS_BAD_PAGE);
    return;
  }
  const int chunks = (n + kChunk - 1) / kChunk, base = chunk_base(row0, b);
  const uint32_t sbase = smem_u32(smem);
  uint8_t* const hand = smem + kStages * kStageBytes + warp * 2 * kHandBytes + lane * 16;
  const int col0 = (blockIdx.x * kWarps + warp) * 8;  // the warp's first value column

  if (!chain) {
    const int ot = th - kWarps * 32;
    const uint16_t* const vcol = a.v + (size_t)row0 * (size_t)a.v_stride + (size_t)h * kHeadDim + blockIdx.x * kWarps * 8;
    const auto fetch = [&](int i) {  // chunk i into its stage
      if (i >= chunks) return;
      const uint8_t* const keys = a.keys + ((size_t)(base + i) * a.hk + kh) * kKeyRecord + ot * 16;
      const uint8_t* const heads = a.heads + ((size_t)(base + i) * a.hv + h) * kHeadRecord + ot * 16;
      const uint32_t to = sbase + (i % kStages) * kStageBytes + ot * 16;
      constexpr int kStep = kWarps * 32 * 16;
#pragma unroll
      for (int x = 0; x < kKeyRecord; x += kStep) cp_async_16(to + x, keys + x);
#pragma unroll
      for (int x = 0; x < kHeadRecord; x += kStep)
        if (x + kStep <= kHeadRecord || x + ot * 16 < kHeadRecord) cp_async_16(to + kKeyRecord + x, heads + x);
      // values: kWarps 16-byte pieces of a row; those behind the lane's rows are dropped where they are read
      const int r = ot / kWarps, p = ot % kWarps;
      static_assert(kChunk * kWarps == kWarps * 32, "one piece to a thread");
      if (i * kChunk + r < n)
        cp_async_16(sbase + (i % kStages) * kStageBytes + kKeyRecord + kHeadRecord + value_at(r, p),
                    vcol + ((size_t)i * kChunk + r) * (size_t)a.v_stride + 8 * p);
    };
    uint16_t* const orow = a.out + ((size_t)row0 * a.hv + h) * kHeadDim + col0 + 2 * c;
    fetch(0);
    cp_async_commit();
    for (int i = 0; i <= chunks; ++i) {
      cp_async_wait<0>();
      __syncthreads();  // chunk i is there; chunk i - 1 has been handed over, chunk i - 2 is done with
      fetch(i + 1);
      cp_async_commit();
      if (i == 0) continue;
      const int ch = i - 1;
      const uint32_t key = sbase + (ch % kStages) * kStageBytes, tri = key + kKeyRecord;
      const float* const fac = reinterpret_cast<const float*>(smem + (ch % kStages) * kStageBytes + kKeyRecord + 3 * kTriBytes);
      const uint8_t* const from = hand + (ch & 1) * kHandBytes;
      uint32_t S[16], u[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint4 y = *reinterpret_cast<const uint4*>(from + x * 512);
        S[4 * x] = y.x, S[4 * x + 1] = y.y, S[4 * x + 2] = y.z, S[4 * x + 3] = y.w;
      }
      {
        const uint4 y = *reinterpret_cast<const uint4*>(from + 4 * 512);
        u[0] = y.x, u[1] = y.y, u[2] = y.z, u[3] = y.w;
      }
      const float4 up = *reinterpret_cast<const float4*>(from + 5 * 512);
      float qs[2][4] = {}, p[2][4] = {};
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t f[4];
          ldmatrix_x4(key + kKeyBytes + key_at(16 * r + (lane & 15), 2 * m + (lane >> 4)), f[0], f[1], f[2], f[3]);
          mma_f16_16816(qs[r], f, S[2 * m], S[2 * m + 1]);
        }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int jt = 0; jt <= m; ++jt) {
          uint32_t f[4];
          ldmatrix_x4_trans(tri_a(tri + 2 * kTriBytes, m, jt, lane), f[0], f[1], f[2], f[3]);
          mma_f16_16816(p[m], f, u[2 * jt], u[2 * jt + 1]);
        }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int t = 16 * m + 8 * r + g;
          const float o1 = fac[3 * kChunk + t], o2 = fac[4 * kChunk + t];
          if (ch * kChunk + t < n)
            *reinterpret_cast<uint32_t*>(orow + ((size_t)ch * kChunk + t) * a.hv * kHeadDim) =
                pack_bf16x2(fmaf(o1, qs[m][2 * r] * up.x, o2 * (p[m][2 * r] * up.z)),
                            fmaf(o1, qs[m][2 * r + 1] * up.y, o2 * (p[m][2 * r + 1] * up.w)));
        }
    }
    return;
  }

  // S[m]: key dims 16 m + g and + 8, value columns 2 c and + 1, times sig
  float S[8][4];
  float* const st = a.state + ((size_t)slot * a.hv + h) * kStateElems + (size_t)(col0 + 2 * c) * kHeadDim + g;
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) S[m][i] = L > 0 ? st[(size_t)(i & 1) * kHeadDim + 16 * m + (i >> 1) * 8] : 0.0f;
  // powers of two that keep the operands in fp16's range, per value column
  float sig[2], isig[2], top[2];
  const auto tops = [&] {  // the largest of S per column
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = 0.0f;
#pragma unroll
      for (int m = 0; m < 8; ++m) top[i] = max3(top[i], fabsf(S[m][i]), fabsf(S[m][i + 2]));
    }
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1)
#pragma unroll
      for (int i = 0; i < 2; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
  };
  tops();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const Scale sc = scale_of_row(top[i]);
    sig[i] = sc.down, isig[i] = sc.up;
    top[i] *= sc.down;
#pragma unroll
    for (int m = 0; m < 8; ++m) S[m][i] *= sc.down, S[m][i + 2] *= sc.down;
  }

  for (int ch = 0; ch < chunks; ++ch) {
    __syncthreads();
    const uint8_t* const stage = smem + (ch % kStages) * kStageBytes;
    const uint32_t key = sbase + (ch % kStages) * kStageBytes, tri = key + kKeyRecord;
    const float* const fac = reinterpret_cast<const float*>(stage + kKeyRecord + 3 * kTriBytes);
    const float* const sca = fac + kFactors * kChunk;
    uint8_t* const to = hand + (ch & 1) * kHandBytes;

    // values, rows 16 m + 8 r + g, and the scale for x, u and the state behind the chunk, by bounds of all of them
    float v[2][2][2], vtop[2] = {0.0f, 0.0f};
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int t = 16 * m + 8 * r + g;
        uint32_t w = *reinterpret_cast<const uint32_t*>(stage + kKeyRecord + kHeadRecord + value_at(t, warp) + 4 * c);
        if (ch * kChunk + t >= n) w = 0u;
        v[m][r][0] = bf16_lo(w), v[m][r][1] = bf16_hi(w);
#pragma unroll
        for (int i = 0; i < 2; ++i) vtop[i] = fmaxf(vtop[i], fabsf(v[m][r][i]));
      }
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1)
#pragma unroll
      for (int i = 0; i < 2; ++i) vtop[i] = fmaxf(vtop[i], __shfl_xor_sync(0xffffffffu, vtop[i], o));
    float nsig[2], nisig[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float x = top[i] * isig[i];
      const float bx = sca[kMaxB] * (vtop[i] + x * sca[kSumA]), bu = sca[kSumT] * bx;
      const float all = fmaxf(max3(bx, bu, sca[kMaxC] * bu), fmaf(sca[kSumC], bu, x * fabsf(sca[kF])));
      // all * nsig in [2^13, 2^14): sums of products are rounded up past it by less than a factor of two
      const uint32_t e = min(max(__float_as_uint(all) >> 23, 14u), 253u);
      nsig[i] = all == 0.0f ? sig[i] : __uint_as_float((254u + 13u - e) << 23);
      nisig[i] = all == 0.0f ? isig[i] : __uint_as_float((e - 13u) << 23);
    }
    // S k' in two parts: rows are tokens
    float sh[2][4] = {}, sl[2][4] = {};
    uint32_t out[16];
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      uint32_t lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        split_f16(S[m][2 * i], S[m][2 * i + 1], out[2 * m + i], lo[i]);
        out[2 * m + i] = transpose8(out[2 * m + i]);
        lo[i] = transpose8(lo[i]);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t f[4];
        ldmatrix_x4(key + key_at(16 * r + (lane & 15), 2 * m + (lane >> 4)), f[0], f[1], f[2], f[3]);
        mma_f16_16816(sh[r], f, out[2 * m], out[2 * m + 1]);
        mma_f16_16816(sl[r], f, lo[0], lo[1]);
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      *reinterpret_cast<uint4*>(to + x * 512) = make_uint4(out[4 * x], out[4 * x + 1], out[4 * x + 2], out[4 * x + 3]);
    *reinterpret_cast<float4*>(to + 5 * 512) = make_float4(isig[0], isig[1], nisig[0], nisig[1]);
    // x, in two parts as B operands
    uint32_t xh[2][2], xl[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int t = 16 * m + 8 * r + g;
        const float fa = fac[t], beta = fac[kChunk + t];
        float x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          x[i] = (beta * nsig[i]) * (v[m][r][i] - (fa * isig[i]) * (sh[m][2 * r + i] + sl[m][2 * r + i]));
        split_f16(x[0], x[1], xh[m][r], xl[m][r]);
        xh[m][r] = transpose8(xh[m][r]);
        xl[m][r] = transpose8(xl[m][r]);
      }
    // u = T x
    float u[2][4] = {}, ul_[2][4] = {};
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int jt = 0; jt <= m; ++jt) {
        uint32_t f[4], e[4];
        ldmatrix_x4_trans(tri_a(tri, m, jt, lane), f[0], f[1], f[2], f[3]);
        ldmatrix_x4_trans(tri_a(tri + kTriBytes, m, jt, lane), e[0], e[1], e[2], e[3]);
        mma_f16_16816(u[m], f, xh[jt][0], xh[jt][1]);
        mma_f16_16816(ul_[m], f, xl[jt][0], xl[jt][1]);
        mma_f16_16816(ul_[m], e, xh[jt][0], xh[jt][1]);
      }
    // u for the outputs (one part), and with its factors for the state (two)
    uint32_t uo[2][2], uh[2][2], ul[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float fc = fac[2 * kChunk + 16 * m + 8 * r + g];
        const float u0 = (u[m][2 * r] + ul_[m][2 * r]) * sca[kTUp], u1 = (u[m][2 * r + 1] + ul_[m][2 * r + 1]) * sca[kTUp];
        split_f16(u0 * fc, u1 * fc, uh[m][r], ul[m][r]);
        uh[m][r] = transpose8(uh[m][r]);
        ul[m][r] = transpose8(ul[m][r]);
        uo[m][r] = transpose8(pack_f16x2(u0, u1));
      }
    *reinterpret_cast<uint4*>(to + 4 * 512) = make_uint4(uo[0][0], uo[0][1], uo[1][0], uo[1][1]);
    // the state behind the chunk; a factor past fp32's range belongs to a state of zeros
    const float f0 = fminf(sca[kF] * isig[0] * nsig[0], 3.0e38f), f1 = fminf(sca[kF] * isig[1] * nsig[1], 3.0e38f);
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      S[m][0] *= f0, S[m][1] *= f1, S[m][2] *= f0, S[m][3] *= f1;
#pragma unroll
      for (int jt = 0; jt < 2; ++jt) {
        uint32_t f[4];
        ldmatrix_x4_trans(key + key_at(16 * jt + (lane & 7) + ((lane >> 4) << 3), 2 * m + ((lane >> 3) & 1)), f[0], f[1],
                          f[2], f[3]);
        mma_f16_16816(S[m], f, uh[jt][0], uh[jt][1]);
        mma_f16_16816(S[m], f, ul[jt][0], ul[jt][1]);
      }
    }
    tops();
#pragma unroll
    for (int i = 0; i < 2; ++i) sig[i] = nsig[i], isig[i] = nisig[i];
  }
  __syncthreads();  // the last chunk is handed over
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) st[(size_t)(i & 1) * kHeadDim + 16 * m + (i >> 1) * 8] = S[m][i] * isig[i & 1];
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace
}  // namespace sdva

using namespace sdva;

extern "C" size_t prompt_delta_workspace_size(int total_tokens, int num_lanes, int num_k_heads, int num_v_heads) {
  if (total_tokens <= 0 || num_lanes <= 0 || num_k_heads <= 0 || num_v_heads <= 0 || num_v_heads % num_k_heads != 0)
    return 0;
  const size_t slots = (size_t)total_tokens / kChunk + (size_t)num_lanes;
  return align256(slots * num_k_heads * kKeyRecord) + align256(slots * num_v_heads * kHeadRecord);
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
  const size_t chunk_slots = (size_t)total_tokens / kChunk + (size_t)num_lanes;
  if (chunk_slots > 0x7fffffffu) return SDVA_ERR_UNSUPPORTED;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
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
                        ws,
                        ws + align256(chunk_slots * num_k_heads * kKeyRecord),
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
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  chunk_kernel<<<dim3((unsigned)chunk_slots, num_k_heads), kChunkThreads, 0, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SDVA_ERR_CUDA;
  if (cudaFuncSetAttribute(state_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStateSmem) != cudaSuccess)
    return SDVA_ERR_CUDA;
  state_kernel<<<dim3(kHeadDim / (8 * kWarps), num_v_heads, num_lanes), kThreads, kStateSmem, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}
