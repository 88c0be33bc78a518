// kv_append_rope.cu -- kv_append_rope and kv_append_packed_rope: queries and
// keys turned to their positions, keys and values quantised into the paged
// cache, in one launch.
//
// A pair (x1, x2) of a head's rotated dims becomes (x1 c - x2 s, x2 c + x1 s)
// with the position's cosine and sine out of the caller's table; fp32, every
// product and sum rounded (no contraction), then bf16.  The cache gets what
// kv_append_quant writes for those bf16 keys, byte for byte.
//
// Bound by memory: 512 bytes per q head and 512 + codes per kv head and token,
// and 4 bytes of the table per rotated dim and token.  Grid: page slots by
// (kv heads, then groups of four q heads).  A kv head's CTA holds its page's K
// and V (kv_page.cuh); a q CTA gives one warp a token's four heads, eight
// threads each, so that the heads share the loads of the table's row.
// 41,175 tokens of 8 lanes, 24 / 4 heads: FP8, 128 dims turned, 122 us (5.7 TB/s);
// INT4, 64 dims, 123 by halves and 116 by neighbours.  64 lanes of up to 16 rows,
// INT8: 6.7 us; one token: 3.3.
#include "kv_page.cuh"

namespace sdva {
namespace {

using kvpage::kItems;
using kvpage::kThreads;
using kvpage::slot_base;

constexpr int kQHeads = 4;  // q heads of a CTA
constexpr int kAhead = 2;   // tokens of a thread whose loads are under way together

struct RopeArgs {
  const uint16_t* q;
  const uint16_t* k_new;
  const uint16_t* v_new;
  uint8_t* k_codes;
  uint8_t* v_codes;
  void* k_scales;
  void* v_scales;
  const float* rope;        // [num_positions][rot]: cosines, then sines
  const int32_t* positions;  // nullable [B][n_new] (windows)
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* cu;      // packed rows; null: a window of n_new rows per lane
  const int32_t* n_lane;  // nullable [B] (windows)
  uint16_t* q_out;
  uint16_t* k_out;  // nullable
  int32_t* status;
  long long q_stride, k_stride, v_stride;
  int num_pages, num_q_heads, num_kv_heads, max_pages, num_lanes, total, n_new, lane_slots, num_positions, rot;
};

// Sixteen dims of a row: [8 sub, 8 sub + 8) of the lower and the upper half.
struct Piece {
  uint4 lo, hi;
};

__device__ __forceinline__ Piece load_piece(const uint16_t* row, int sub) {
  return {__ldcs(reinterpret_cast<const uint4*>(row + sub * 8)), __ldcs(reinterpret_cast<const uint4*>(row + sub * 8 + 64))};
}
__device__ __forceinline__ void store_piece(uint16_t* row, int sub, const Piece& p) {
  *reinterpret_cast<uint4*>(row + sub * 8) = p.lo;
  *reinterpret_cast<uint4*>(row + sub * 8 + 64) = p.hi;
}

// a c - b s and a c + b s without contraction
__device__ __forceinline__ float turn_minus(float a, float c, float b, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_plus(float a, float c, float b, float s) {
  return __fadd_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}

// Eight dims x whose partners are the dims y of another place: this thread's
// half of the pairs is the first (x c - y s) or the second (x c + y s).
__device__ __forceinline__ uint4 turn_pairs(uint4 x, uint4 y, const float4 (&c)[2], const float4 (&s)[2], bool first) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
  const float cs[8] = {c[0].x, c[0].y, c[0].z, c[0].w, c[1].x, c[1].y, c[1].z, c[1].w};
  const float sn[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[1].x, s[1].y, s[1].z, s[1].w};
  uint32_t r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a0 = bf16_lo(a[j]), a1 = bf16_hi(a[j]), b0 = bf16_lo(b[j]), b1 = bf16_hi(b[j]);
    // x c + y (-s) has the same products and the same sum
    const float s0 = first ? -sn[2 * j] : sn[2 * j], s1 = first ? -sn[2 * j + 1] : sn[2 * j + 1];
    r[j] = pack_bf16x2(turn_plus(a0, cs[2 * j], b0, s0), turn_plus(a1, cs[2 * j + 1], b1, s1));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// Eight dims that are four pairs side by side.
__device__ __forceinline__ uint4 turn_neighbours(uint4 x, float4 c, float4 s) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w};
  const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
  uint32_t r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x1 = bf16_lo(a[j]), x2 = bf16_hi(a[j]);
    r[j] = pack_bf16x2(turn_minus(x1, cs[j], x2, sn[j]), turn_plus(x2, cs[j], x1, sn[j]));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// The piece turned by the table's row `t` (8 threads of a row call it together;
// rot = 16, 32, 64 or 128).
template <bool kNeighbours>
__device__ __forceinline__ void turn(Piece& p, const float* t, int rot, int sub) {
  const int half = rot / 2;
  const float4* const c4 = reinterpret_cast<const float4*>(t);
  const float4* const s4 = reinterpret_cast<const float4*>(t + half);
  if constexpr (kNeighbours) {
    if (sub * 8 < rot) p.lo = turn_neighbours(p.lo, __ldg(c4 + sub), __ldg(s4 + sub));
    if (rot == kHeadDim) p.hi = turn_neighbours(p.hi, __ldg(c4 + 8 + sub), __ldg(s4 + 8 + sub));
  } else if (rot == kHeadDim) {  // the pairs are this thread's two halves
    const float4 c[2] = {__ldg(c4 + 2 * sub), __ldg(c4 + 2 * sub + 1)};
    const float4 s[2] = {__ldg(s4 + 2 * sub), __ldg(s4 + 2 * sub + 1)};
    const uint4 lo = p.lo;
    p.lo = turn_pairs(lo, p.hi, c, s, true);
    p.hi = turn_pairs(p.hi, lo, c, s, false);
  } else {  // the partner is the thread rot / 16 away
    const int away = rot / 16;
    const unsigned row = 0xFFu << (threadIdx.x & 24);
    uint4 y;
    y.x = __shfl_xor_sync(row, p.lo.x, away);
    y.y = __shfl_xor_sync(row, p.lo.y, away);
    y.z = __shfl_xor_sync(row, p.lo.z, away);
    y.w = __shfl_xor_sync(row, p.lo.w, away);
    if (sub < 2 * away) {
      const int at = 2 * (sub & (away - 1));
      const float4 c[2] = {__ldg(c4 + at), __ldg(c4 + at + 1)};
      const float4 s[2] = {__ldg(s4 + at), __ldg(s4 + at + 1)};
      p.lo = turn_pairs(p.lo, y, c, s, !(sub & away));
    }
  }
}

// Four CTAs to an SM and two tokens ahead: of the batch above 121 us; three CTAs and one token 132, three and four 122,
// four and one 123, five and two 124.
template <int KVT, bool kNeighbours>
__global__ void __launch_bounds__(kThreads, 4) append_rope_kernel(RopeArgs a) {
  const int slot = blockIdx.x, th = threadIdx.x;
  bool bad = false;
  int b, page, n;
  size_t row0;
  if (a.cu != nullptr) {
    // the slot's lane, the last whose base is at or before it, and whether all offsets are in order
    __shared__ uint32_t s_found[kThreads / 32];
    constexpr uint32_t kBad = 1u << 20;  // above every count: the host refuses more lanes than 65,535
    uint32_t found = 0;
    for (int i = th; i < a.num_lanes; i += kThreads) {
      const int lo = a.cu[i], hi = a.cu[i + 1];
      bad |= lo < 0 || hi < lo || hi > a.total;
      found += slot_base(lo, i) <= slot;
    }
    found = __reduce_add_sync(0xffffffffu, found + (bad ? kBad : 0u));
    if ((th & 31) == 0) s_found[th >> 5] = found;
    __syncthreads();
    found = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) found += s_found[w];
    if (found >= kBad) {
      if (slot == 0 && blockIdx.y == 0 && th == 0) raise_status(a.status, SDVA_STATUS_BAD_COUNT);
      return;
    }
    if (found == 0) return;
    b = (int)found - 1;
    row0 = (size_t)a.cu[b];
    n = a.cu[b + 1] - (int)row0;
    page = slot - slot_base((int)row0, b);
  } else {
    b = slot / a.lane_slots;
    page = slot - b * a.lane_slots;
    row0 = (size_t)b * a.n_new;
    n = a.n_lane != nullptr ? a.n_lane[b] : a.n_new;
  }
  const bool report = page == 0 && blockIdx.y == 0 && th == 0;
  if (n < 0 || (a.cu == nullptr && n > a.n_new)) {
    if (report) raise_status(a.status, SDVA_STATUS_BAD_COUNT);
    return;
  }
  if (n == 0) return;  // nothing to write: the lane is not examined
  const int L = a.seq_lens[b];
  const long long end = (long long)L + n;
  // positions are int32, and those of the rotation rows of the table
  if (L < 0 || end > min((long long)a.max_pages * kPage, 0x7fffffffLL) ||
      (a.positions == nullptr && end > a.num_positions)) {
    if (report) raise_status(a.status, SDVA_STATUS_OVERFLOW);
    return;
  }
  const int lp = L / kPage + page;
  if ((long long)lp * kPage >= end) return;
  const int t0 = max(L, lp * kPage), start = t0 - lp * kPage;
  const int count = (int)(min(end, (long long)lp * kPage + kPage) - t0);
  row0 += (size_t)(t0 - L);  // the page's first token

  // every page and position of the lane has to be valid before anything of it is written
  const int32_t* const table = a.page_table + (size_t)b * a.max_pages;
  const int last = (int)((end - 1) / kPage);
  int wrong = 0;
  for (int p = L / kPage + th; p <= last; p += kThreads) {
    const int id = table[p];
    if (id < 0 || id >= a.num_pages) wrong |= SDVA_STATUS_BAD_PAGE;
  }
  const int32_t* const positions = a.positions == nullptr ? nullptr : a.positions + (size_t)b * a.n_new;
  if (positions != nullptr)
    for (int i = th; i < n; i += kThreads)
      if (positions[i] < 0 || positions[i] >= a.num_positions) wrong |= SDVA_STATUS_OVERFLOW;
  const int pid = table[lp], sub = th & 7;
  // the table's row of the page's token t
  const auto turns = [&](int t) {
    return a.rope + (size_t)(positions != nullptr ? positions[t0 - L + t] : t0 + t) * a.rot;
  };
  const bool stop = __syncthreads_or(wrong);
  if (stop) {
    if (page == 0 && blockIdx.y == 0 && wrong) raise_status(a.status, wrong);
    return;
  }

  if ((int)blockIdx.y < a.num_kv_heads) {
    const int hk = blockIdx.y, is_v = (th >> 3) & 1;
    const uint16_t* const src = (is_v ? a.v_new : a.k_new) + (size_t)hk * kHeadDim;
    const size_t stride = (size_t)(is_v ? a.v_stride : a.k_stride);
    uint4 x[kItems][2];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int t = (th >> 4) + i * (kThreads / 16);
      x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (t < count) {
        const Piece p = load_piece(src + (row0 + t) * stride, sub);
        x[i][0] = p.lo;
        x[i][1] = p.hi;
      }
    }
    if (!is_v) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int t = (th >> 4) + i * (kThreads / 16);
        if (t < count) {
          Piece p = {x[i][0], x[i][1]};
          turn<kNeighbours>(p, turns(t), a.rot, sub);
          x[i][0] = p.lo;
          x[i][1] = p.hi;
          if (a.k_out != nullptr)
            store_piece(a.k_out + ((row0 + t) * a.num_kv_heads + hk) * kHeadDim, sub, p);
        }
      }
    }
    const size_t ph = (size_t)pid * a.num_kv_heads + hk;
    kvpage::write_page<KVT>(x, th, start, count, ph, is_v ? a.v_codes : a.k_codes, is_v ? a.v_scales : a.k_scales);
    return;
  }
  const int head = ((int)blockIdx.y - a.num_kv_heads) * kQHeads + ((th >> 3) & (kQHeads - 1));
  if (head >= a.num_q_heads) return;
  const uint16_t* const src = a.q + (size_t)head * kHeadDim;
  // a thread's tokens t, t + 8, ..: kAhead loads in flight
  constexpr int kStep = kThreads / 32;
  for (int t = th >> 5; t < count; t += kAhead * kStep) {
    Piece p[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (t + i * kStep < count) p[i] = load_piece(src + (row0 + t + i * kStep) * (size_t)a.q_stride, sub);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (t + i * kStep < count) {
        turn<kNeighbours>(p[i], turns(t + i * kStep), a.rot, sub);
        store_piece(a.q_out + ((row0 + t + i * kStep) * a.num_q_heads + head) * kHeadDim, sub, p[i]);
      }
  }
}

template <bool kNeighbours>
void launch(int dtype, dim3 grid, cudaStream_t s, const RopeArgs& a) {
  const auto kernel = dtype == SDVA_KV_FP8_E4M3   ? append_rope_kernel<SDVA_KV_FP8_E4M3, kNeighbours>
                      : dtype == SDVA_KV_INT4_G32 ? append_rope_kernel<SDVA_KV_INT4_G32, kNeighbours>
                      : dtype == SDVA_KV_INT8_G64 ? append_rope_kernel<SDVA_KV_INT8_G64, kNeighbours>
                                                  : append_rope_kernel<SDVA_KV_FP8_ROW, kNeighbours>;
  kernel<<<grid, kThreads, 0, s>>>(a);
}

// What both calls check; the rows' and lanes' counts are the caller's.
int rope_launch(const sdva_kv_cache* cache, RopeArgs& a, int64_t slots, int pairing, sdva_stream_t stream) {
  if (const int rc = append_launch(cache, a.k_new, a.v_new, a.num_lanes, 1, nullptr, a.page_table, a.max_pages,
                                   a.seq_lens, a.status, stream, true))
    return rc;
  if (a.q == nullptr || a.q_out == nullptr || a.rope == nullptr || a.num_q_heads <= 0 || a.num_positions <= 0 ||
      a.num_q_heads % cache->num_kv_heads != 0)
    return SDVA_ERR_INVALID;
  const int64_t q_width = (int64_t)a.num_q_heads * kHeadDim, width = (int64_t)cache->num_kv_heads * kHeadDim;
  if (a.q_stride < q_width || a.k_stride < width || a.v_stride < width || ((a.q_stride | a.k_stride | a.v_stride) & 7) ||
      ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new) |
        reinterpret_cast<uintptr_t>(a.q_out) | reinterpret_cast<uintptr_t>(a.k_out) |
        reinterpret_cast<uintptr_t>(a.rope)) &
       15u))
    return SDVA_ERR_INVALID;
  if ((a.rot != 16 && a.rot != 32 && a.rot != 64 && a.rot != 128) ||
      (pairing != SDVA_ROPE_HALVES && pairing != SDVA_ROPE_NEIGHBOURS))
    return SDVA_ERR_UNSUPPORTED;
  const int64_t heads = (int64_t)cache->num_kv_heads + (a.num_q_heads + kQHeads - 1) / kQHeads;
  if (slots > 0x7fffffff || heads > 65535) return SDVA_ERR_UNSUPPORTED;
  a.k_codes = static_cast<uint8_t*>(cache->k_codes);
  a.v_codes = static_cast<uint8_t*>(cache->v_codes);
  a.k_scales = cache->k_scales;
  a.v_scales = cache->v_scales;
  a.num_pages = cache->num_pages;
  a.num_kv_heads = cache->num_kv_heads;
  const dim3 grid((unsigned)slots, (unsigned)heads);
  (pairing == SDVA_ROPE_NEIGHBOURS ? launch<true> : launch<false>)(cache->dtype, grid,
                                                                   reinterpret_cast<cudaStream_t>(stream), a);
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}

RopeArgs rope_args(const void* q, const void* k_new, const void* v_new, int64_t q_stride, int64_t k_stride,
                   int64_t v_stride, int num_q_heads, int num_lanes, const float* rope, int num_positions, int rot_dim,
                   const int32_t* page_table, int max_pages_per_lane, const int32_t* seq_lens, void* q_out,
                   void* k_out, int32_t* status) {
  RopeArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.num_q_heads = num_q_heads;
  a.num_lanes = num_lanes;
  a.rope = rope;
  a.num_positions = num_positions;
  a.rot = rot_dim;
  a.page_table = page_table;
  a.max_pages = max_pages_per_lane;
  a.seq_lens = seq_lens;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_out = static_cast<uint16_t*>(k_out);
  a.status = status;
  return a;
}

}  // namespace
}  // namespace sdva

using namespace sdva;

extern "C" int kv_append_rope(const sdva_kv_cache* cache, const void* q, const void* k_new, const void* v_new,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride, int num_q_heads, int num_lanes,
                              int n_new, const int32_t* n_lane, const float* rope, int num_positions, int rot_dim,
                              int pairing, const int32_t* positions, const int32_t* page_table,
                              int max_pages_per_lane, const int32_t* seq_lens, void* q_out, void* k_out,
                              int32_t* status, sdva_stream_t stream) {
  if (n_new <= 0) return SDVA_ERR_INVALID;
  RopeArgs a = rope_args(q, k_new, v_new, q_stride, k_stride, v_stride, num_q_heads, num_lanes, rope, num_positions,
                         rot_dim, page_table, max_pages_per_lane, seq_lens, q_out, k_out, status);
  a.n_new = n_new;
  a.n_lane = n_lane;
  a.positions = positions;
  a.lane_slots = (int)(((int64_t)n_new + kPage - 2) / kPage + 1);  // pages that n_new tokens can touch
  return rope_launch(cache, a, (int64_t)num_lanes * a.lane_slots, pairing, stream);
}

extern "C" int kv_append_packed_rope(const sdva_kv_cache* cache, const void* q, const void* k_new, const void* v_new,
                                     int64_t q_stride, int64_t k_stride, int64_t v_stride, int num_q_heads,
                                     int total_tokens, const int32_t* cu_tokens, int num_lanes, const float* rope,
                                     int num_positions, int rot_dim, int pairing, const int32_t* page_table,
                                     int max_pages_per_lane, const int32_t* seq_lens, void* q_out, void* k_out,
                                     int32_t* status, sdva_stream_t stream) {
  if (total_tokens == 0) return SDVA_OK;
  if (cu_tokens == nullptr || total_tokens < 0) return SDVA_ERR_INVALID;
  RopeArgs a = rope_args(q, k_new, v_new, q_stride, k_stride, v_stride, num_q_heads, num_lanes, rope, num_positions,
                         rot_dim, page_table, max_pages_per_lane, seq_lens, q_out, k_out, status);
  a.cu = cu_tokens;
  a.total = total_tokens;
  return rope_launch(cache, a, (int64_t)total_tokens / kPage + 2 * (int64_t)num_lanes, pairing, stream);
}
