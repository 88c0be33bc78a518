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
// not depend on the state: k' and q' in fp16, T, P, and each token's factors,
// laid out as the other kernel's shared memory holds them.
// state_kernel goes through a lane's chunks with a head's state in registers.
// A warp has 16 value rows of it, as accumulators of values by key dims, which
// are the A operand of S k' as they stand; x and u come out values by tokens and
// are A of the product behind them in turn.  No warp needs another one's values.
// This chain, state to state, is what a long prompt's time is made of (a prompt
// alone has eight such warps per head), so that nothing else is on it: each of its
// warps has another one, a chunk behind, that takes S and u out of shared memory,
// makes the outputs, and copies the chunks that come.  One barrier of the CTA per
// chunk.
//
// Ranges.  The state and the updates that are added to it go in two fp16 parts
// about a power of two of each value row, chosen behind u from the largest of both;
// T x and P u are tf32 products (T and x in two parts of 11 bits, u in one), P is
// in fp16 about a power of two of each of its rows.  So a token's output depends
// on the sizes of no later token and of no other value row, and T's entries and u
// may grow as far as fp32 goes where a token's map expands (beta |k|^2 above 2, decays
// above 1).  With one power of two for a chunk's T, x, u and 16 rows of S, which
// failed there, the calls below took 668, 445, 119 and 11.5 us.
//
// 16 / 32 heads: one prompt of 16,384 tokens 722 us, of which 104 are
// chunk_kernel's (shared memory comes first: L1 is at 79% of its peak, DRAM at 16%)
// and the rest 512 chunks at 1.21 us; eight of 2,048 486 us.  8 / 24 heads, eight
// prompts of 1 to 2,011 tokens 126 us; 4 / 8 heads, 40 tokens 10.5.  A chunk is
// 158 products of 16 x 8 x 16 (or 8, tf32) a warp, 8 cycles each, in some 2,300
// cycles; the others are the ways from one product's accumulators to the next one's
// operands, which depend on each other, and the barrier.  The legacy tensor path
// (mma.sync) is taken with intent: its operands are the chain's own registers,
// 16 value rows are its tile, and a head's chain is spread over eight quarters of
// SMs.  A tcgen05 product has 128 rows: one SM would hold a head's whole chain.
// By arithmetic (not built) the chain's products would take some 600 cycles a
// chunk there (8 warps' 158 of 2,048 multiply-adds at 3,900 a cycle), and each of
// its three dependent steps would add a way through tensor memory.
#include "delta_common.cuh"

namespace sdva {
namespace {

using namespace delta;

constexpr int kChunk = 32;
// A chunk's records in the workspace and in shared memory (bytes).  16-byte
// pieces of a row of k' and q' (256 bytes) are stored at piece ^ (row & 7), so that
// eight rows of a matrix load fall into different banks.
constexpr int kKeyBytes = kChunk * kHeadDim * 2;
constexpr int kKeyRecord = 2 * kKeyBytes;  // k', q' of a key head
constexpr int kTBytes = kChunk * kChunk * 3;            // three 16 x 16 tiles, fp32
constexpr int kPBytes = kChunk * kChunk * 3 / 2;        // the same, fp16
constexpr int kFactors = 5;  // per token: a r, b, (f / a) r, scale r_q a, scale r_q / (P's scale of the row)
constexpr int kScalars = 4;  // f
constexpr int kFactorBytes = (kFactors * kChunk + kScalars) * 4;
constexpr int kHeadRecord = kTBytes + kPBytes + kFactorBytes;  // of a value head
static_assert(kHeadRecord % 16 == 0 && kTBytes % 16 == 0, "records are copied 16 bytes at a time");

__device__ __forceinline__ int key_at(int row, int piece) { return row * 256 + ((piece ^ (row & 7)) << 4); }
// T's element: 16 columns in rows 0 .. 15, 32 in the others; groups of eight change places so that four rows' eight bytes
// of four threads each are in different banks.
__device__ __forceinline__ int t_at(int row, int col) {
  return row < 16 ? row * 16 + (col ^ ((row << 2) & 8)) : 256 + (row - 16) * 32 + (col ^ ((row & 3) << 3));
}
// P's 16-byte pieces, eight rows of a column: 32 bytes a column and 16 rows, columns 16 and on behind those of rows 16
// and on.  Columns four apart change their pieces' places.
__device__ __forceinline__ int p_at(int col, int piece) {
  return (col + (piece & 2 ? 16 : 0)) * 32 + (((piece & 1) ^ ((col >> 2) & 1)) << 4);
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

// The largest of a warp's x >= 0.
__device__ __forceinline__ float positive_max(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

// A warp's bytes from shared memory to a record, 512 at a time: a column of its own is 16 bytes of 32 lines a store,
// which kept L1 busy for 80% of the kernel's time.
template <int kBytes>
__device__ __forceinline__ void copy_out(uint8_t* to, const uint8_t* from, int lane) {
  __syncwarp();
#pragma unroll
  for (int x = 16 * lane; x < kBytes; x += 512)
    *reinterpret_cast<uint4*>(to + x) = *reinterpret_cast<const uint4*>(from + x);
}

constexpr int kChunkThreads = 128;

struct ChunkSmem {
  union {
    alignas(16) uint8_t key[2][kKeyBytes];       // k', q', until their products are there
    alignas(16) float a[4][kChunk][kChunk + 4];  // A of each warp's value head
  };
  float gram[2][kChunk][kChunk + 4];  // k' . k', q' . k' (row, column)
  alignas(16) float eg[4][kChunk];    // of each warp's value head
  alignas(16) float br[4][kChunk];
  float sum_sq[2][kChunk], up[2][kChunk], down[2][kChunk];
  uint32_t found[kChunkThreads / 32];
};

__global__ void __launch_bounds__(kChunkThreads, 6) chunk_kernel(PromptArgs a) {
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

  // decays and strengths of the warp's first value head, ahead of their use
  const int group = a.hv / a.hk;
  const bool on = lane < valid;
  const auto decay_at = [&](int task) { return ((size_t)t0 + lane) * a.hv + kh * group + (task >> 1); };
  float log_decay = on && warp < 2 * group ? a.log_decay[decay_at(warp)] : 0.0f;
  float beta_ = on && warp < 2 * group ? a.beta[decay_at(warp)] : 0.0f;
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
      unsigned long long sq2 = 0;
      const unsigned long long down = tc::f2_pack(sc.down, sc.down);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const unsigned long long f = tc::fmul2(tc::f2_pack(bf16_lo(x[i]), bf16_hi(x[i])), down);
        sq2 = tc::ffma2(f, f, sq2);
        const float2 y = tc::f2_unpack(f);
        x[i] = pack_f16x2(y.x, y.y);
      }
      float sq = tc::f2_unpack(sq2).x + tc::f2_unpack(sq2).y;
      sq += __shfl_xor_sync(0xffffffffu, sq, 1);
      sq += __shfl_xor_sync(0xffffffffu, sq, 2);
      if (p == 0) {
        s.sum_sq[m][r] = sq;
        s.up[m][r] = sc.up;
        s.down[m][r] = sc.down;
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
  const Scale sk = {s.down[0][lane], s.up[0][lane]}, sq = {s.down[1][lane], s.up[1][lane]};
  const float rk = on ? row_factor(s.sum_sq[0][lane], a.eps, sk) : 0.0f;
  const float rq = on ? row_factor(s.sum_sq[1][lane], a.eps, sq) : 0.0f;
  for (int task = warp; task < 2 * group; task += kChunkThreads / 32) {
    const int h = kh * group + (task >> 1);
    uint8_t* const rec = a.heads + ((size_t)slot * a.hv + h) * kHeadRecord;
    float* const fac = reinterpret_cast<float*>(rec + kTBytes + kPBytes);
    if (task != warp) {
      log_decay = on ? a.log_decay[decay_at(task)] : 0.0f;
      beta_ = on ? a.beta[decay_at(task)] : 0.0f;
    }
    const float eg = on ? expf(log_decay) : 1.0f, beta = beta_;
    float x[kChunk], d = 0.0f;
    __syncwarp();  // the task before is done with the warp's places
    s.eg[warp][lane] = eg;
    s.br[warp][lane] = beta * rk;
    __syncwarp();
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
      for (int i = 0; i < kChunk; i += 4) {
        const float4 e = *reinterpret_cast<const float4*>(&s.eg[warp][i]);
        const float egs[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          d = i + y == lane ? 1.0f : d * egs[y];
          x[i + y] = i + y >= lane ? d * rk * s.gram[1][i + y][lane] : 0.0f;
        }
      }
      // a row's scale: what a token has of the ones before it does not depend on later rows
      float up = 0.0f;
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        const Scale ps = scale_to_top(positive_max(fabsf(x[i])));
        x[i] *= ps.down;
        up = i == lane ? ps.up : up;
      }
      uint8_t* const mine = reinterpret_cast<uint8_t*>(s.a[warp]);
#pragma unroll
      for (int p = 0; p < kChunk / 8; ++p)
        if (p >= 2 || lane < 16)
          *reinterpret_cast<uint4*>(mine + p_at(lane, p)) =
              make_uint4(pack_f16x2(x[8 * p], x[8 * p + 1]), pack_f16x2(x[8 * p + 2], x[8 * p + 3]),
                         pack_f16x2(x[8 * p + 4], x[8 * p + 5]), pack_f16x2(x[8 * p + 6], x[8 * p + 7]));
      copy_out<kPBytes>(rec + kTBytes, mine, lane);
      const float fa = fall * rk, fc = rest * rk;
      fac[lane] = fa;
      fac[kChunk + lane] = beta;
      fac[2 * kChunk + lane] = fc;
      fac[3 * kChunk + lane] = a.scale * rq * fall;
      fac[4 * kChunk + lane] = a.scale * rq * up;
      if (lane == 0) fac[kFactors * kChunk] = all;
      continue;
    }
    // A by columns, then those of the inverse of 1 + A: as soon as a row is known it leaves the rows below
    float (*const A)[kChunk + 4] = s.a[warp];
#pragma unroll
    for (int i = 0; i < kChunk; i += 4) {
      const float4 e = *reinterpret_cast<const float4*>(&s.eg[warp][i]), f = *reinterpret_cast<const float4*>(&s.br[warp][i]);
      const float egs[4] = {e.x, e.y, e.z, e.w}, brs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        d = i + y == lane ? 1.0f : d * egs[y];
        x[i + y] = i + y > lane ? brs[y] * (d * rk) * s.gram[0][i + y][lane] : 0.0f;
      }
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
    float* const mine = &A[0][0];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (i >= 16 || lane < 16) mine[t_at(i, lane)] = round_22(x[i]);
    copy_out<kTBytes>(rec, reinterpret_cast<const uint8_t*>(mine), lane);
  }
}

// Of a chunk the chain takes k', T, the factors and its values, the outputs q',
// P and the factors; each in two places, the one in use and the one that comes.
constexpr int kChainBytes = kKeyBytes + kTBytes + kFactorBytes;
constexpr int kOutBytes = kKeyBytes + kPBytes + kFactorBytes;
// What a warp of the chain hands over: S (32 words a thread), u (16), the scales of S's rows
constexpr int kHandBytes = 12 * 32 * 16 + 64;
template <int kWarps>
constexpr int kStateSmem = 2 * (kChainBytes + kWarps * kChunk * 32 + kOutBytes + kWarps * kHandBytes);

// P's rows 16 m .., columns 16 jt .. as A: stored by columns, so that the matrices come transposed.
__device__ __forceinline__ uint32_t p_a(uint32_t tri, int m, int jt, int lane) {
  return tri + p_at(16 * jt + (lane & 7) + ((lane >> 4) << 3), 2 * m + ((lane >> 3) & 1));
}
// The values of a chunk: 2 kWarps 16-byte pieces to a row, eight rows of a piece in different banks.
template <int kWarps>
__device__ __forceinline__ int value_at(int row, int piece) {
  return (row * 2 * kWarps + (piece ^ (kWarps == 4 ? row & 7 : (row >> 1) & 3))) << 4;
}

// kWarps warps of the chain, 16 value rows each, and as many for the outputs; with two of them three CTAs fit an SM.
template <int kWarps>
__global__ void __launch_bounds__(kWarps * 64, kWarps == 2 ? 3 : 1) state_kernel(PromptArgs a, long long limit) {
  static_assert(kWarps == 2 || kWarps == 4, "the values' places in shared memory");
  constexpr int kThreads = 2 * kWarps * 32;
  constexpr int kValueBytes = kWarps * kChunk * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int never;  // 0: no role's wait ends another's
  const int th = threadIdx.x, lane = th & 31, g = lane >> 2, c = lane & 3;
  __shared__ int gave_up;  // whether a wait ran out
  if (th == 0) never = gave_up = 0;
  const bool chain = th < kWarps * 32;
  const int warp = (th >> 5) & (kWarps - 1);
  const int h = blockIdx.y, kh = h / (a.hv / a.hk);
  // Longer lanes first where a thread can have one each: the last to start decides when the call ends.
  int b = blockIdx.z;
  bool bad = false;
  {
    __shared__ int length[kThreads];
    __shared__ int mine;
    const bool sorted = a.num_lanes <= kThreads;
    for (int i = th; i < a.num_lanes; i += kThreads) {
      const int lo = a.cu[i], hi = a.cu[i + 1];
      bad |= lo < 0 || hi < lo || hi > a.total;
      if (sorted) length[i] = hi - lo;
    }
    if (__syncthreads_or(bad)) {
      if (blockIdx.x == 0 && h == 0 && b == 0 && th == 0) raise_status(a.status, SDVA_STATUS_BAD_COUNT);
      return;
    }
    if (sorted && a.num_lanes > 1) {
      if (th < a.num_lanes) {
        int rank = 0;
        for (int i = 0; i < a.num_lanes; ++i) rank += length[i] > length[th] || (length[i] == length[th] && i < th);
        if (rank == b) mine = th;
      }
      __syncthreads();
      b = mine;
    }
  }
  const bool report = blockIdx.x == 0 && h == 0 && th == 0;
  const int row0 = a.cu[b], n = a.cu[b + 1] - row0;
  if (n == 0) return;
  const int slot = a.slots[b], L = a.seq_lens != nullptr ? a.seq_lens[b] : 1;
  if (L < 0 || slot < 0 || slot >= a.num_slots) {
    if (report) raise_status(a.status, L < 0 ? SDVA_STATUS_OVERFLOW : SDVA_STATUS_BAD_PAGE);
    return;
  }
  const int chunks = (n + kChunk - 1) / kChunk, base = chunk_base(row0, b);
  uint8_t* const chain_smem = smem;                                       // k', T in two parts, factors; values
  uint8_t* const out_smem = smem + 2 * (kChainBytes + kValueBytes);       // q', P, factors
  uint8_t* const hand = out_smem + 2 * kOutBytes + warp * 2 * kHandBytes + lane * 16;
  const int row16 = (blockIdx.x * kWarps + warp) * 16;  // the warp's first value row

  if (!chain) {
    const int ot = th - kWarps * 32;
    bool dead = false;  // of thread 0: a wait ran out; no more records are copied, and what follows is undefined
    __shared__ uint64_t bars[2];
    if (ot == 0) {
      tc::mbar_init(smem_u32(&bars[0]), 1);
      tc::mbar_init(smem_u32(&bars[1]), 1);
      tc::mbar_fence_init();
    }
    const uint16_t* const vcol = a.v + (size_t)row0 * (size_t)a.v_stride + (size_t)h * kHeadDim + blockIdx.x * kWarps * 16;
    // What the next interval needs: chunk i + 1 for the chain, chunk i for the outputs.  Records by bulk copies of one
    // thread; the values' 16-byte pieces by all (those behind the lane's rows are zeros).
    const auto fetch = [&](int i, uint32_t bar) {
      if (ot == 0 && !dead) {
        const int bytes = (i + 1 < chunks ? kChainBytes : 0) + (i >= 0 && i < chunks ? kOutBytes : 0);
        if (bytes != 0) tc::mbar_arrive_expect_tx(bar, bytes);
        if (i + 1 < chunks) {
          const uint8_t* const keys = a.keys + ((size_t)(base + i + 1) * a.hk + kh) * kKeyRecord;
          const uint8_t* const heads = a.heads + ((size_t)(base + i + 1) * a.hv + h) * kHeadRecord;
          const uint32_t to = smem_u32(chain_smem) + ((i + 1) & 1) * (kChainBytes + kValueBytes);
          tc::bulk_load(to, keys, kKeyBytes, bar);
          tc::bulk_load(to + kKeyBytes, heads, kTBytes, bar);
          tc::bulk_load(to + kKeyBytes + kTBytes, heads + kTBytes + kPBytes, kFactorBytes, bar);
        }
        if (i >= 0 && i < chunks) {
          const uint32_t to = smem_u32(out_smem) + (i & 1) * kOutBytes;
          tc::bulk_load(to, a.keys + ((size_t)(base + i) * a.hk + kh) * kKeyRecord + kKeyBytes, kKeyBytes, bar);
          tc::bulk_load(to + kKeyBytes, a.heads + ((size_t)(base + i) * a.hv + h) * kHeadRecord + kTBytes,
                        kPBytes + kFactorBytes, bar);
        }
      }
      if (i + 1 < chunks) {
        const uint32_t to = smem_u32(chain_smem) + ((i + 1) & 1) * (kChainBytes + kValueBytes) + kChainBytes;
#pragma unroll
        for (int x = ot; x < kChunk * 2 * kWarps; x += kWarps * 32) {
          const int r = x / (2 * kWarps), p = x % (2 * kWarps);
          const int t = (i + 1) * kChunk + r;
          cp_async_16_or_zeros(to + value_at<kWarps>(r, p), vcol + (size_t)min(t, n - 1) * (size_t)a.v_stride + 8 * p, t < n);
        }
      }
    };
    uint16_t* const orow = a.out + ((size_t)row0 * a.hv + h) * kHeadDim + row16 + 2 * c;
    fetch(-1, smem_u32(&bars[0]));
    for (int i = 0; i <= chunks; ++i) {
      const uint32_t bar = smem_u32(&bars[i & 1]), parity = (i >> 1) & 1;
      if (ot == 0 && !dead && !copies_here(bar, parity, &never, limit)) {
        raise_status(a.status, SDVA_STATUS_TIMEOUT);
        dead = gave_up = 1;
      }
      cp_async_wait_all();
      tc::fence_proxy_async_smem();
      __syncthreads();  // chunk i is there for the chain and chunk i - 1 for the outputs, which has been handed over
      fetch(i, smem_u32(&bars[(i + 1) & 1]));
      if (i == 0) continue;
      const int ch = i - 1;
      const uint8_t* const stage = out_smem + (ch & 1) * kOutBytes;
      const uint32_t key = smem_u32(stage), tri = key + kKeyBytes;
      const float* const fac = reinterpret_cast<const float*>(stage + kKeyBytes + kPBytes);
      const uint8_t* const from = hand + (ch & 1) * kHandBytes;
      float qs[2][2][4] = {}, p[2][2][4] = {};
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        const uint4 S = *reinterpret_cast<const uint4*>(from + m * 512);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t f[4];
          ldmatrix_x4(key + key_at(16 * r + (lane & 15), 2 * m + (lane >> 4)), f[0], f[1], f[2], f[3]);
          mma_f16_16816(qs[r][0], f, S.x, S.y);
          mma_f16_16816(qs[r][1], f, S.z, S.w);
        }
      }
      // P u in one tf32 part: the k indices c and c + 4 are the tokens 2 c and 2 c + 1 in both operands
#pragma unroll
      for (int jt = 0; jt < 2; ++jt) {
        float u[2][4];  // tokens 16 jt + 2 c, + 1, + 8, + 9 of value row 8 t + g
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float4 y = *reinterpret_cast<const float4*>(from + (8 + 2 * jt + r) * 512);
          u[0][2 * r] = to_tf32(y.x), u[0][2 * r + 1] = to_tf32(y.y), u[1][2 * r] = to_tf32(y.z), u[1][2 * r + 1] = to_tf32(y.w);
        }
#pragma unroll
        for (int m = jt; m < 2; ++m) {
          uint32_t f[4];
          ldmatrix_x4_trans(p_a(tri, m, jt, lane), f[0], f[1], f[2], f[3]);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 y = f16x2_to_f32(f[2 * r]), z = f16x2_to_f32(f[2 * r + 1]);
            const float pa[4] = {y.x, z.x, y.y, z.y};
            mma_tf32_1688(p[m][0], pa, u[0][2 * r], u[0][2 * r + 1]);
            mma_tf32_1688(p[m][1], pa, u[1][2 * r], u[1][2 * r + 1]);
          }
        }
      }
      float2 up[2];  // of the value rows 8 x + 2 c, + 1
#pragma unroll
      for (int x = 0; x < 2; ++x) up[x] = *reinterpret_cast<const float2*>(from - lane * 16 + 12 * 512 + (8 * x + 2 * c) * 4);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int t = 16 * m + 8 * r + g;
          const float o1 = fac[3 * kChunk + t], o2 = fac[4 * kChunk + t];
          if (ch * kChunk + t < n)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              *reinterpret_cast<uint32_t*>(orow + ((size_t)ch * kChunk + t) * a.hv * kHeadDim + 8 * x) =
                  pack_bf16x2(fmaf(o1 * up[x].x, qs[m][x][2 * r], o2 * p[m][x][2 * r]),
                              fmaf(o1 * up[x].y, qs[m][x][2 * r + 1], o2 * p[m][x][2 * r + 1]));
        }
    }
    return;
  }

  // S[x]: value rows g (0, 1) and g + 8 (2, 3), key dims 8 x + 2 c and + 1; the state is S times the row's isig
  float S[16][4], sig[2], isig[2];
  float* const st = a.state + ((size_t)slot * a.hv + h) * kStateElems + (size_t)(row16 + g) * kHeadDim + 2 * c;
#pragma unroll
  for (int x = 0; x < 16; ++x)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 y = L > 0 ? *reinterpret_cast<const float2*>(st + i * 8 * kHeadDim + 8 * x) : make_float2(0.0f, 0.0f);
      S[x][2 * i] = y.x, S[x][2 * i + 1] = y.y;
    }
  const auto row_max = [&](float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
  };
  // A row's largest, `all`, brought into fp16's range; the row is times `was` now.
  const auto choose = [&](int t, float all, float was) {
    const Scale sc = all == 0.0f ? Scale{1.0f, 1.0f} : scale_to_top(all);
    const float by = fminf(was * sc.down, 3.0e38f);  // past fp32's range only for a row of zeros
#pragma unroll
    for (int x = 0; x < 16; ++x) S[x][2 * t] *= by, S[x][2 * t + 1] *= by;
    sig[t] = sc.down, isig[t] = sc.up;
  };
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float top = 0.0f;
#pragma unroll
    for (int x = 0; x < 16; ++x) top = max3(top, fabsf(S[x][2 * t]), fabsf(S[x][2 * t + 1]));
    choose(t, row_max(top), 1.0f);
  }

  for (int ch = 0; ch < chunks; ++ch) {
    tc::fence_proxy_async_smem();  // what was read of a place is read before the next bulk copy into it
    __syncthreads();
    const uint8_t* const stage = chain_smem + (ch & 1) * (kChainBytes + kValueBytes);
    const uint32_t key = smem_u32(stage);
    const float* const T = reinterpret_cast<const float*>(stage + kKeyBytes);
    const float* const fac = T + kTBytes / 4;
    uint8_t* const to = hand + (ch & 1) * kHandBytes;
    if (c == 0) {
      float* const up = reinterpret_cast<float*>(to - lane * 16 + 12 * 512);
      up[g] = isig[0], up[8 + g] = isig[1];
    }

    // S k' in two parts: rows are value rows g, g + 8, columns tokens 8 t + 2 c (+ 1).  A step's rows of k' are loaded
    // before the one in front of it is stored for the outputs: a load would wait for that store.
    float x[4][4] = {}, top[2] = {};
    const auto keys = [&](int m, uint32_t (&b)[4][2]) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        ldmatrix_x4(key + key_at(16 * i + (lane & 7) + ((lane >> 4) << 3), 2 * m + ((lane >> 3) & 1)), b[2 * i][0], b[2 * i][1],
                    b[2 * i + 1][0], b[2 * i + 1][1]);
    };
    uint32_t b[2][4][2];
    keys(0, b[0]);
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      uint32_t hi[4], lo[4];
      if (m < 7) keys(m + 1, b[(m + 1) & 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) split_f16(S[2 * m + (i >> 1)][2 * (i & 1)], S[2 * m + (i >> 1)][2 * (i & 1) + 1], hi[i], lo[i]);
#pragma unroll
      for (int t = 0; t < 4; ++t) mma_f16_16816(x[t], hi, b[m & 1][t][0], b[m & 1][t][1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) mma_f16_16816(x[t], lo, b[m & 1][t][0], b[m & 1][t][1]);
      *reinterpret_cast<uint4*>(to + m * 512) = make_uint4(hi[0], hi[2], hi[1], hi[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) top[i & 1] = max3(top[i & 1], fabsf(S[2 * m + (i >> 1)][2 * (i & 1)]), fabsf(S[2 * m + (i >> 1)][2 * (i & 1) + 1]));
    }
    // values of the tokens 8 t + 2 c, + 1
    uint32_t v[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
      ldmatrix_x4_trans(key + kChainBytes + value_at<kWarps>(lane, 2 * warp + r), v[r][0], v[r][1], v[r][2], v[r][3]);
    // x as it is, in tf32: the tokens' values, and T's entries, have sizes of their own, which fp16 would need a scale for
    float xl[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float2 fa = *reinterpret_cast<const float2*>(fac + 8 * t + 2 * c);
      const float2 be = *reinterpret_cast<const float2*>(fac + kChunk + 8 * t + 2 * c);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        x[t][2 * r] = be.x * (bf16_lo(v[r][t]) - fa.x * (isig[r] * x[t][2 * r]));
        x[t][2 * r + 1] = be.y * (bf16_hi(v[r][t]) - fa.y * (isig[r] * x[t][2 * r + 1]));
        split_tf32(x[t][2 * r], x[t][2 * r], xl[t][2 * r]);
        split_tf32(x[t][2 * r + 1], x[t][2 * r + 1], xl[t][2 * r + 1]);
      }
    }
    // u' = x' T': 8 x 8 pieces of T up to its diagonal.  The k indices c and c + 4 of a product are the tokens 2 c and
    // 2 c + 1 in both operands, so that x is A as it came.
    float2 Th[10], Tl[10];
#pragma unroll
    for (int i = 0, y = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j <= i; ++j, ++y) {
        const float2 z = *reinterpret_cast<const float2*>(T + t_at(8 * i + g, 8 * j + 2 * c));
        split_22(z.x, Th[y].x, Tl[y].x);
        split_22(z.y, Th[y].y, Tl[y].y);
      }
    float u[4][4] = {};
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int o = 0; o < 10; ++o) {
        // rows of T in an order that leaves an accumulator two other products' time
        constexpr int kRow[10] = {3, 2, 0, 3, 1, 3, 2, 3, 1, 2}, kCol[10] = {0, 0, 0, 1, 0, 2, 1, 3, 1, 2};
        const int i = kRow[o], j = kCol[o];
        const float(&y)[4] = p == 1 ? xl[j] : x[j];
        const float xa[4] = {y[0], y[2], y[1], y[3]};
        const float2 z = (p == 0 ? Tl : Th)[i * (i + 1) / 2 + j];
        mma_tf32_1688(u[i], xa, z.x, z.y);
      }
    const float fall = fac[kFactors * kChunk];
    // u for the outputs; with its factors, in two parts, for the state
    float most[2] = {};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      *reinterpret_cast<float4*>(to + (8 + t) * 512) = make_float4(u[t][0], u[t][1], u[t][2], u[t][3]);
      const float2 fc = *reinterpret_cast<const float2*>(fac + 2 * kChunk + 8 * t + 2 * c);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        u[t][2 * r] *= fc.x, u[t][2 * r + 1] *= fc.y;
        most[r] = max3(most[r], fabsf(u[t][2 * r]), fabsf(u[t][2 * r + 1]));
      }
    }
    // the rows' scales behind the chunk: 32 updates, elements of k' below 4
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float was = fall * isig[r];
      choose(r, fmaf(row_max(top[r]), was, 4.0f * kChunk * row_max(most[r])), was);
    }
    uint32_t uh[2][4], ul[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float (&y)[4] = u[2 * j + (i >> 1)];
        split_f16(y[2 * (i & 1)] * sig[i & 1], y[2 * (i & 1) + 1] * sig[i & 1], uh[j][i], ul[j][i]);
      }
    // the state behind the chunk
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t b0[2], b1[2];
        ldmatrix_x4_trans(key + key_at(16 * j + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * m + (lane >> 4)), b0[0], b1[0],
                          b0[1], b1[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma_f16_16816(S[2 * m + i], uh[j], b0[i], b1[i]);
          mma_f16_16816(S[2 * m + i], ul[j], b0[i], b1[i]);
        }
      }
  }
  __syncthreads();  // the last chunk is handed over
  if (gave_up) return;  // the state stays as it was
#pragma unroll
  for (int x = 0; x < 16; ++x)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float2*>(st + i * 8 * kHeadDim + 8 * x) = make_float2(S[x][2 * i] * isig[i], S[x][2 * i + 1] * isig[i]);
}

template <int kWarps>
int launch_as(const PromptArgs& a, cudaStream_t s) {
  const auto kernel = state_kernel<kWarps>;
  constexpr int bytes = kStateSmem<kWarps>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return SDVA_ERR_CUDA;
  kernel<<<dim3(kHeadDim / (16 * kWarps), a.hv, a.num_lanes), kWarps * 64, bytes, s>>>(a, wait_limit());
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}

int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

// Two warps of the chain to a CTA, up to three CTAs on an SM, or four warps and one CTA.  A chunk takes the chain 21
// parts with one CTA of two on the SM, 40 with two, 47 with three, and 29 in a CTA of four: whichever ends first by how
// many rounds its grid makes, lanes being of one length.  Of 2,048 tokens a lane, us with two and with four: 16 heads, two
// lanes 98 and 119, three 160 and 124, four 167 and 131, six 206 and 244; 32 heads, four lanes 285 and 257, eight 486
// and 507.  Short lanes make many short rounds, of which those of three CTAs an SM overlap: 60 lanes of 100 tokens, 16
// heads, 142 and 151.
int launch_state(const PromptArgs& a, cudaStream_t s) {
  const int64_t sms = num_sms() > 0 ? num_sms() : 1, twos = (int64_t)a.hv * a.num_lanes * (kHeadDim / 32);
  const int64_t rest = twos % (3 * sms);
  const int64_t with_two = twos / (3 * sms) * 47 + (rest == 0 ? 0 : rest <= sms ? 21 : rest <= 2 * sms ? 40 : 47);
  const int64_t with_four = (twos / 2 + sms - 1) / sms * 29;
  return with_two <= with_four || a.total < (int64_t)a.num_lanes * 256 ? launch_as<2>(a, s) : launch_as<4>(a, s);
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
  return launch_state(a, s);
}
