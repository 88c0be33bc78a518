// kv_append_packed.cu -- kv_append_quant for lanes packed one behind the
// other: a prompt batch's K/V into the paged, quantised cache.
//
// What is written is what kv_append_quant writes (sdva.h).  The call is bound
// by memory: 512 bytes in and 128 to 264 out per token and kv head (65,536
// tokens, 4 kv heads: FP8 36.3 us, 5.5 TB/s; FP8 rows 35.5, 5.7; INT8 39.5, 5.1;
// INT4 37.2, 4.6, which issues more instructions).  One CTA
// per (touched page, kv head) takes K and V together: eight threads per token
// row, each with dims [8 t, 8 t + 8) of both 64-dim halves, so that a row's
// loads and stores are whole 128- and 64-byte runs; all of a thread's loads
// are issued before the lane's page ids are checked.  The grid is flat over
// page slots, found from the offsets alone (slot_base).
#include "kv_page.cuh"

namespace sdva {
namespace {

using kvpage::kItems;
using kvpage::kRowThreads;
using kvpage::kThreads;
using kvpage::slot_base;

struct PackedArgs {
  const uint16_t* k_new;
  const uint16_t* v_new;
  uint8_t* k_codes;
  uint8_t* v_codes;
  void* k_scales;
  void* v_scales;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* cu;
  int32_t* status;
  long long k_stride, v_stride;
  int num_pages, num_kv_heads, max_pages, num_lanes, total;
};

template <int KVT>
__global__ void __launch_bounds__(kThreads, 4) append_packed_kernel(PackedArgs a) {
  const int slot = blockIdx.x, hk = blockIdx.y, th = threadIdx.x;
  // the slot's lane, the last whose base is at or before it, and whether all offsets are in order
  __shared__ uint32_t s_found[kThreads / 32];
  constexpr uint32_t kBad = 1u << 20;  // above every count: the host refuses more lanes than 65,535
  uint32_t found = 0, bad = 0;
  for (int b = th; b < a.num_lanes; b += kThreads) {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    bad |= lo < 0 || hi < lo || hi > a.total;
    found += slot_base(lo, b) <= slot;
  }
  found = __reduce_add_sync(0xffffffffu, found + (bad ? kBad : 0u));
  if ((th & 31) == 0) s_found[th >> 5] = found;
  __syncthreads();
  found = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) found += s_found[w];
  if (found >= kBad) {
    if (slot == 0 && hk == 0 && th == 0) raise_status(a.status, SDVA_STATUS_BAD_COUNT);
    return;
  }
  const int below = (int)found;
  if (below == 0) return;
  const int b = below - 1, row0 = a.cu[b], n = a.cu[b + 1] - row0, page = slot - slot_base(row0, b);
  if (n == 0) return;  // nothing to write: the lane is not examined
  const int L = a.seq_lens[b];
  const long long end = (long long)L + n;
  const bool report = page == 0 && hk == 0 && th == 0;
  if (L < 0 || end > min((long long)a.max_pages * kPage, 0x7fffffffLL)) {  // positions are int32
    if (report) raise_status(a.status, SDVA_STATUS_OVERFLOW);
    return;
  }
  const int lp = L / kPage + page;
  if ((long long)lp * kPage >= end) return;
  const int t0 = max(L, lp * kPage), start = t0 - lp * kPage;
  const int count = (int)(min(end, (long long)lp * kPage + kPage) - t0);

  // rows (token, K|V) it / 8 of items it = th, th + 256, ...; dims 8 sub .. and 64 + 8 sub ..
  const int sub = th & (kRowThreads - 1), is_v = (th >> 3) & 1;
  const uint16_t* const src = (is_v ? a.v_new : a.k_new) + (size_t)hk * kHeadDim + sub * 8;
  const size_t stride = (size_t)(is_v ? a.v_stride : a.k_stride);
  uint4 x[kItems][2];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int t = (th >> 4) + i * (kThreads / 16);
    x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
    if (t < count) {
      const uint16_t* r = src + ((size_t)row0 + (t0 - L) + t) * stride;
      x[i][0] = __ldcs(reinterpret_cast<const uint4*>(r));
      x[i][1] = __ldcs(reinterpret_cast<const uint4*>(r + 64));
    }
  }
  // every page of the lane's range has to be valid before one is written
  const int32_t* const row = a.page_table + (size_t)b * a.max_pages;
  const int last = (int)((end - 1) / kPage), pid = row[lp];
  for (int p = L / kPage + th; p <= last; p += kThreads) {
    const int id = row[p];
    bad |= id < 0 || id >= a.num_pages;
  }
  if (__syncthreads_or(bad)) {
    if (report) raise_status(a.status, SDVA_STATUS_BAD_PAGE);
    return;
  }
  const size_t ph = (size_t)pid * a.num_kv_heads + hk;
  uint8_t* const codes = is_v ? a.v_codes : a.k_codes;
  void* const scales = is_v ? a.v_scales : a.k_scales;

  kvpage::write_page<KVT>(x, th, start, count, ph, codes, scales);
}

}  // namespace
}  // namespace sdva

using namespace sdva;

extern "C" int kv_append_packed(const sdva_kv_cache* cache, const void* k_new, const void* v_new, int64_t k_stride,
                                int64_t v_stride, int total_tokens, const int32_t* cu_tokens, int num_lanes,
                                const int32_t* page_table, int max_pages_per_lane, const int32_t* seq_lens,
                                int32_t* status, sdva_stream_t stream) {
  if (total_tokens == 0) return SDVA_OK;
  if (cu_tokens == nullptr || total_tokens < 0) return SDVA_ERR_INVALID;
  if (const int rc = append_launch(cache, k_new, v_new, num_lanes, 1, nullptr, page_table, max_pages_per_lane,
                                   seq_lens, status, stream, true))
    return rc;
  const int64_t width = (int64_t)cache->num_kv_heads * kHeadDim;
  if (k_stride < width || v_stride < width || ((k_stride | v_stride) & 7) ||
      ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15u))
    return SDVA_ERR_INVALID;
  PackedArgs a;
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.k_codes = static_cast<uint8_t*>(cache->k_codes);
  a.v_codes = static_cast<uint8_t*>(cache->v_codes);
  a.k_scales = cache->k_scales;
  a.v_scales = cache->v_scales;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.cu = cu_tokens;
  a.status = status;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.num_pages = cache->num_pages;
  a.num_kv_heads = cache->num_kv_heads;
  a.max_pages = max_pages_per_lane;
  a.num_lanes = num_lanes;
  a.total = total_tokens;
  const dim3 grid(total_tokens / kPage + 2 * num_lanes, cache->num_kv_heads);
  const auto kernel = cache->dtype == SDVA_KV_FP8_E4M3   ? append_packed_kernel<SDVA_KV_FP8_E4M3>
                      : cache->dtype == SDVA_KV_INT4_G32 ? append_packed_kernel<SDVA_KV_INT4_G32>
                      : cache->dtype == SDVA_KV_INT8_G64 ? append_packed_kernel<SDVA_KV_INT8_G64>
                                                         : append_packed_kernel<SDVA_KV_FP8_ROW>;
  kernel<<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}
