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
// A warp has 8 or 16 value columns of it and works alone: S as 16 x 8
// accumulators (key dims by values) becomes the B operand of S k' by transposing
// 8 x 8 tiles between registers, so do x and u, and no warp waits for another
// but for the next chunk's copies.
#include "delta_common.cuh"

namespace sdva {
namespace {

using namespace delta;

constexpr int kChunk = 32;
// A chunk's records in the workspace and in shared memory (bytes).  16-byte
// pieces of a row are stored at piece ^ (row & 7) (k', q': 256-byte rows) and
// piece ^ (row / 2 & 3) (T, P: 64-byte rows), so that eight rows of a matrix load
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
__device__ __forceinline__ int tri_at(int row, int col) {
  return row * 64 + (((col >> 3) ^ ((row >> 1) & 3)) << 4) + (col & 7) * 2;
}

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
  // T and P of a value head per warp; a thread has column `lane`, and token `lane`
  const int group = a.hv / a.hk;
  const bool on = lane < valid;
  const Scale sk = {s.down[0][lane], s.up[0][lane]}, sq = {s.down[1][lane], s.up[1][lane]};
  const float rk = on ? row_factor(s.sum_sq[0][lane], a.eps, sk) : 0.0f;
  const float rq = on ? row_factor(s.sum_sq[1][lane], a.eps, sq) : 0.0f;
  for (int j = warp; j < group; j += kChunkThreads / 32) {
    const int h = kh * group + j;
    uint8_t* const rec = a.heads + ((size_t)slot * a.hv + h) * kHeadRecord;
    const size_t at = ((size_t)t0 + lane) * a.hv + h;
    const float eg = on ? expf(a.log_decay[at]) : 1.0f, beta = on ? a.beta[at] : 0.0f;
    // products of e^g up to this token, and from the next one on
    float fall = eg, rest = __shfl_down_sync(0xffffffffu, eg, 1);
    if (lane == 31) rest = 1.0f;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_up_sync(0xffffffffu, fall, o), y = __shfl_down_sync(0xffffffffu, rest, o);
      if (lane >= o) fall *= x;
      if (lane + o < 32) rest *= y;
    }
    const float all = __shfl_sync(0xffffffffu, fall, 31);
    float (*const A)[kChunk + 4] = s.a[warp];
    const float br = beta * rk;
    float p[kChunk], d = 0.0f, top = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const float egi = __shfl_sync(0xffffffffu, eg, i), bri = __shfl_sync(0xffffffffu, br, i);
      d = i == lane ? 1.0f : d * egi;
      const float w = d * rk, x = bri * w * s.gram[0][i][lane];
      A[i][lane] = i > lane ? x : 0.0f;
      p[i] = i >= lane ? w * s.gram[1][i][lane] : 0.0f;
      top = fmaxf(top, fabsf(p[i]));
    }
    const Scale ps = scale_of_row(warp_max(top));
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      *reinterpret_cast<__half*>(rec + 2 * kTriBytes + tri_at(i, lane)) = __float2half_rn(p[i] * ps.down);
    __syncwarp();
    // columns of the inverse of 1 + A, row by row
    float t[kChunk];
    top = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int l = 0; l < i; l += 4) {
        const float4 r = *reinterpret_cast<const float4*>(&A[i][l]);
        x[0] = fmaf(r.x, t[l], x[0]);
        if (l + 1 < i) x[1] = fmaf(r.y, t[l + 1], x[1]);
        if (l + 2 < i) x[2] = fmaf(r.z, t[l + 2], x[2]);
        if (l + 3 < i) x[3] = fmaf(r.w, t[l + 3], x[3]);
      }
      t[i] = i == lane ? 1.0f : -((x[0] + x[1]) + (x[2] + x[3]));
      top = fmaxf(top, fabsf(t[i]));
    }
    top = warp_max(top);
    const Scale ts = scale_of_row(top);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const float x = t[i] * ts.down;
      const __half hi = __float2half_rn(x);
      *reinterpret_cast<__half*>(rec + tri_at(i, lane)) = hi;
      *reinterpret_cast<__half*>(rec + kTriBytes + tri_at(i, lane)) = __float2half_rn(x - __half2float(hi));
    }
    float* const f = reinterpret_cast<float*>(rec + 3 * kTriBytes);
    const float fa = fall * rk, fc = rest * rk;
    f[lane] = fa;
    f[kChunk + lane] = beta;
    f[2 * kChunk + lane] = fc;
    f[3 * kChunk + lane] = a.scale * rq * fall;
    f[4 * kChunk + lane] = a.scale * rq * ps.up;
    const float sum_a = warp_max(fabsf(fa) * s.l1[lane]), max_b = warp_max(fabsf(beta)), max_c = warp_max(fabsf(fc));
    const float sum_c = warp_sum(fabsf(fc) * s.top[lane]);
    if (lane == 0) {
      float* const g = f + kFactors * kChunk;
      g[kF] = all;
      g[kSumA] = sum_a;
      g[kMaxB] = max_b;
      g[kSumT] = top * kChunk;
      g[kMaxC] = max_c;
      g[kSumC] = sum_c;
      g[kTUp] = ts.up;
    }
    __syncwarp();
  }
}

constexpr int kStages = 3;
constexpr int kStageBytes = kKeyRecord + kHeadRecord;

// kTiles: 8-wide tiles of value columns of a warp; kWarps warps per CTA.
template <int kTiles, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) state_kernel(PromptArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kThreads = kWarps * 32;
  const int th = threadIdx.x, lane = th & 31, warp = th >> 5, g = lane >> 2, c = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z, kh = h / (a.hv / a.hk);
  const bool report = blockIdx.x == 0 && h == 0 && th == 0;
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
  const int chunks = (n + kChunk - 1) / kChunk, base = chunk_base(row0, b);
  const uint32_t sbase = smem_u32(smem);
  const auto fetch = [&](int i) {  // chunk i into its stage
    if (i < chunks) {
      const uint8_t* const keys = a.keys + ((size_t)(base + i) * a.hk + kh) * kKeyRecord;
      const uint8_t* const heads = a.heads + ((size_t)(base + i) * a.hv + h) * kHeadRecord;
      const uint32_t to = sbase + (i % kStages) * kStageBytes;
      for (int x = th * 16; x < kKeyRecord; x += kThreads * 16) cp_async_16(to + x, keys + x);
      for (int x = th * 16; x < kHeadRecord; x += kThreads * 16) cp_async_16(to + kKeyRecord + x, heads + x);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);

  const int col0 = (blockIdx.x * kWarps + warp) * kTiles * 8;  // the warp's first value column
  // S[m][n]: key dims 16 m + g and + 8, value columns 8 n + 2 c and + 1, times sig
  float S[8][kTiles][4];
  float* const st = a.state + ((size_t)slot * a.hv + h) * kStateElems + (size_t)(col0 + 2 * c) * kHeadDim + g;
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        S[m][t][i] = L > 0 ? st[(size_t)(8 * t + (i & 1)) * kHeadDim + 16 * m + (i >> 1) * 8] : 0.0f;
  // powers of two that keep the operands in fp16's range, per value column
  float sig[kTiles][2], isig[kTiles][2];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x = 0.0f;
#pragma unroll
      for (int m = 0; m < 8; ++m) x = fmaxf(x, fmaxf(fabsf(S[m][t][i]), fabsf(S[m][t][i + 2])));
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
      const Scale sc = scale_of_row(x);
      sig[t][i] = sc.down, isig[t][i] = sc.up;
#pragma unroll
      for (int m = 0; m < 8; ++m) S[m][t][i] *= sc.down, S[m][t][i + 2] *= sc.down;
    }

  const uint16_t* const vrow = a.v + (size_t)row0 * (size_t)a.v_stride + (size_t)h * kHeadDim + col0 + 2 * c;
  uint16_t* const orow = a.out + ((size_t)row0 * a.hv + h) * kHeadDim + col0 + 2 * c;
  uint32_t v[2][2][kTiles];  // rows 16 m + g (+ 8) of the chunk, two columns
  const auto load_v = [&](int i) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int t = i * kChunk + 16 * m + 8 * x + g;
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
          v[m][x][j] = t < n ? *reinterpret_cast<const uint32_t*>(vrow + (size_t)t * (size_t)a.v_stride + 8 * j) : 0u;
      }
  };
  load_v(0);

  for (int ch = 0; ch < chunks; ++ch) {
    cp_async_wait<kStages - 2>();
    __syncthreads();  // the chunk is there, and every warp is done with the stage that is filled next
    fetch(ch + kStages - 1);
    const uint32_t key = sbase + (ch % kStages) * kStageBytes, tri = key + kKeyRecord;
    const float* const fac = reinterpret_cast<const float*>(smem + (ch % kStages) * kStageBytes + kKeyRecord + 3 * kTriBytes);
    const float* const sca = fac + kFactors * kChunk;

    // S k' (two parts) and S q' (one): rows are tokens
    float kh_[2][kTiles][4] = {}, kl_[2][kTiles][4] = {}, qs[2][kTiles][4] = {};
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      uint32_t fk[2][4], fq[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int at = key_at(16 * r + (lane & 15), 2 * m + (lane >> 4));
        ldmatrix_x4(key + at, fk[r][0], fk[r][1], fk[r][2], fk[r][3]);
        ldmatrix_x4(key + kKeyBytes + at, fq[r][0], fq[r][1], fq[r][2], fq[r][3]);
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          split_f16(S[m][t][2 * i], S[m][t][2 * i + 1], hi[i], lo[i]);
          hi[i] = transpose8(hi[i]);
          lo[i] = transpose8(lo[i]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mma_f16_16816(kh_[r][t], fk[r], hi[0], hi[1]);
          mma_f16_16816(kl_[r][t], fk[r], lo[0], lo[1]);
          mma_f16_16816(qs[r][t], fq[r], hi[0], hi[1]);
        }
      }
    }
    // bounds of x, u and the state behind the chunk, and the scale that they leave room for
    float nsig[kTiles][2], nisig[kTiles][2];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int m = 0; m < 8; ++m) x = fmaxf(x, fmaxf(fabsf(S[m][t][i]), fabsf(S[m][t][i + 2])));
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int r = 0; r < 2; ++r) y = fmaxf(y, fabsf(i ? bf16_hi(v[m][r][t]) : bf16_lo(v[m][r][t])));
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) {
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
        }
        x *= isig[t][i];
        const float bx = sca[kMaxB] * (y + x * sca[kSumA]), bu = sca[kSumT] * bx;
        const float all = fmaxf(fmaxf(bx, bu), fmaxf(sca[kMaxC] * bu, fmaf(sca[kSumC], bu, x * fabsf(sca[kF]))));
        // all * nsig in [2^13, 2^14): sums of products are rounded up past it by less than a factor of two
        const uint32_t e = min(max(__float_as_uint(all) >> 23, 15u), 253u);
        nsig[t][i] = all == 0.0f ? sig[t][i] : __uint_as_float((254u + 13u - max(e, 14u)) << 23);
        nisig[t][i] = all == 0.0f ? isig[t][i] : __uint_as_float((max(e, 14u) - 13u) << 23);
      }
    // x, in two parts as B operands
    uint32_t xh[2][kTiles][2], xl[2][kTiles][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int t = 16 * m + 8 * r + g;
        const float fa = fac[t], beta = fac[kChunk + t];
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          float x[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float sk = (kh_[m][j][2 * r + i] + kl_[m][j][2 * r + i]) * isig[j][i];
            x[i] = beta * ((i ? bf16_hi(v[m][r][j]) : bf16_lo(v[m][r][j])) - fa * sk) * nsig[j][i];
          }
          split_f16(x[0], x[1], xh[m][j][r], xl[m][j][r]);
          xh[m][j][r] = transpose8(xh[m][j][r]);
          xl[m][j][r] = transpose8(xl[m][j][r]);
        }
      }
    if (ch + 1 < chunks) load_v(ch + 1);
    // u = T x
    float u[2][kTiles][4] = {};
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int jt = 0; jt <= m; ++jt) {
        uint32_t th_[4], tl[4];
        const int at = (16 * m + (lane & 15)) * 64 + (((2 * jt + (lane >> 4)) ^ (((lane & 15) >> 1) & 3)) << 4);
        ldmatrix_x4(tri + at, th_[0], th_[1], th_[2], th_[3]);
        ldmatrix_x4(tri + kTriBytes + at, tl[0], tl[1], tl[2], tl[3]);
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          mma_f16_16816(u[m][j], th_, xh[jt][j][0], xh[jt][j][1]);
          mma_f16_16816(u[m][j], th_, xl[jt][j][0], xl[jt][j][1]);
          mma_f16_16816(u[m][j], tl, xh[jt][j][0], xh[jt][j][1]);
        }
      }
    // u for the outputs (one part), and with its factors for the state (two)
    uint32_t uo[2][kTiles][2], uh[2][kTiles][2], ul[2][kTiles][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float fc = fac[2 * kChunk + 16 * m + 8 * r + g];
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          const float u0 = u[m][j][2 * r] * sca[kTUp], u1 = u[m][j][2 * r + 1] * sca[kTUp];
          uo[m][j][r] = transpose8(pack_f16x2(u0, u1));
          split_f16(u0 * fc, u1 * fc, uh[m][j][r], ul[m][j][r]);
          uh[m][j][r] = transpose8(uh[m][j][r]);
          ul[m][j][r] = transpose8(ul[m][j][r]);
        }
      }
    // the state behind the chunk
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // a factor past fp32's range belongs to a state of zeros
        const float f = fminf(sca[kF] * isig[t][i] * nsig[t][i], 3.0e38f);
#pragma unroll
        for (int m = 0; m < 8; ++m) S[m][t][i] *= f, S[m][t][i + 2] *= f;
      }
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int jt = 0; jt < 2; ++jt) {
        uint32_t f[4];
        ldmatrix_x4_trans(key + key_at(16 * jt + (lane & 7) + ((lane >> 4) << 3), 2 * m + ((lane >> 3) & 1)), f[0], f[1],
                          f[2], f[3]);
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          mma_f16_16816(S[m][j], f, uh[jt][j][0], uh[jt][j][1]);
          mma_f16_16816(S[m][j], f, ul[jt][j][0], ul[jt][j][1]);
        }
      }
    // outputs
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float p[kTiles][4] = {};
#pragma unroll
      for (int jt = 0; jt <= m; ++jt) {
        uint32_t f[4];
        const int at = (16 * m + (lane & 15)) * 64 + (((2 * jt + (lane >> 4)) ^ (((lane & 15) >> 1) & 3)) << 4);
        ldmatrix_x4(tri + 2 * kTriBytes + at, f[0], f[1], f[2], f[3]);
#pragma unroll
        for (int j = 0; j < kTiles; ++j) mma_f16_16816(p[j], f, uo[jt][j][0], uo[jt][j][1]);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int t = 16 * m + 8 * r + g;
        const float o1 = fac[3 * kChunk + t], o2 = fac[4 * kChunk + t];
        if (ch * kChunk + t < n)
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
            float o[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
              o[i] = fmaf(o1, qs[m][j][2 * r + i] * isig[j][i], o2 * (p[j][2 * r + i] * nisig[j][i]));
            *reinterpret_cast<uint32_t*>(orow + ((size_t)ch * kChunk + t) * a.hv * kHeadDim + 8 * j) =
                pack_bf16x2(o[0], o[1]);
          }
      }
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) sig[t][i] = nsig[t][i], isig[t][i] = nisig[t][i];
  }
  cp_async_wait<0>();
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st[(size_t)(8 * t + (i & 1)) * kHeadDim + 16 * m + (i >> 1) * 8] = S[m][t][i] * isig[t][i & 1];
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int kTiles, int kWarps>
int launch_state(const PromptArgs& a, cudaStream_t s) {
  const auto kernel = state_kernel<kTiles, kWarps>;
  constexpr int bytes = kStages * kStageBytes;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return SDVA_ERR_CUDA;
  kernel<<<dim3(kHeadDim / (8 * kTiles * kWarps), a.hv, a.num_lanes), kWarps * 32, bytes, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}

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
  return launch_state<1, 4>(a, s);
}
