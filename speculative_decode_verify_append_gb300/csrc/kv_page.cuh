// kv_page.cuh -- the rows of one (page, kv head), K and V together, quantised
// into the paged cache: what kv_append_packed and the rotated appends share.
// A CTA of kThreads threads holds up to 64 tokens; eight threads per token
// row, each with dims [8 t, 8 t + 8) of both 64-dim halves, so that a row's
// loads and stores are whole 128- and 64-byte runs.
//
// Division.  A code comes from fp32 x / s, rounded to nearest, and a scale
// from amax / 448, / 127 or / 7.  With r = 1 / s rounded, q = x r, the
// remainder e = x - q s by one fused multiply-add is exact and q + e r,
// rounded once, is the rounded quotient (Markstein, IBM Journal of Research
// and Development 34, 1990).  r comes from the hardware's approximation by one
// such step.  For every bf16 significand over every fp32 one but all ones, and
// an approximation within two units in the last place, the result was
// compared with the division (all 2^30 pairs), while nothing under- or
// overflows: with s in [2^-80, 2^80] the quotients that matter (2^-10 and more
// for E4M3, 1/2 for the integers) have exact remainders.  Elsewhere the
// division itself is used.  With -r for r the same steps give the negative
// quotient, and a zero keeps its sign; two at a time they are one and a half
// instructions an element, where the encoding of a row by divisions and
// conversions made the call bound by instructions (19 an element for INT8).
#pragma once

#include "sdva_internal.cuh"
#include "tc_primitives.cuh"

namespace sdva {
namespace kvpage {

constexpr int kThreads = 256;
constexpr int kRowThreads = 8;  // threads per token row
constexpr int kItems = kPage * 2 * kRowThreads / kThreads;  // (token, K|V) rows per thread

// First page slot of a lane whose rows start at row `at`.  A lane of n tokens
// touches at most n / 64 + 2 pages wherever it starts in a page, and the next
// lane's base is at least n / 64 + 2 further, so no prefix sum is needed.
__device__ __forceinline__ int slot_base(int at, int lane) { return at / kPage + 2 * lane; }

using tc::f2_pack;
using tc::f2_unpack;
using tc::ffma2;
using tc::fmul2;

// -(x / s) of two values, nr = -1 / s (see above)
__device__ __forceinline__ float2 minus_quotients(float x0, float x1, float s, float nr) {
  const unsigned long long x = f2_pack(x0, x1), n = f2_pack(nr, nr), q = fmul2(x, n);
  return f2_unpack(ffma2(ffma2(q, f2_pack(s, s), x), n, q));
}
struct Divisor {
  float s, nr;
  bool plain;  // not for the short form
  __device__ explicit Divisor(float s_) : s(s_) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    nr = -__fmaf_rn(r, __fmaf_rn(-s, r, 1.0f), r);
    plain = !(s >= 0x1p-80f && s <= 0x1p80f) || (~__float_as_uint(s) & 0x7FFFFFu) == 0;
  }
};
// amax / kTop of a bf16 amax >= 0
template <int kTop>
__device__ __forceinline__ float scale_of(float amax) {
  if (amax < 0x1p-70f) return __fdiv_rn(amax, (float)kTop);
  const float n = -1.0f / kTop, q = __fmul_rn(amax, n);
  return -__fmaf_rn(__fmaf_rn(q, (float)kTop, amax), n, q);
}

__device__ __forceinline__ float amax8(uint4 w) {
  // the largest magnitude of eight bf16: their bits without the sign order as integers
  const uint32_t a = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                              __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return __uint_as_float(max(a & 0xFFFF0000u, a << 16));
}
template <int kLanes>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// The E4M3 codes of eight x / s; zeros for s = 0.
__device__ __forceinline__ uint2 e4m3x8(uint4 w, const Divisor& d) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t p[4];
  if (!d.plain) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y = minus_quotients(bf16_lo(u[j]), bf16_hi(u[j]), d.s, d.nr);
      p[j] = e4m3x2_from_f32(y.x, y.y);
    }
    // the sign bits back
    return make_uint2((p[0] | (p[1] << 16)) ^ 0x80808080u, (p[2] | (p[3] << 16)) ^ 0x80808080u);
  }
  if (d.s == 0.0f) return make_uint2(0u, 0u);
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = e4m3x2_from_f32(__fdiv_rn(bf16_lo(u[j]), d.s), __fdiv_rn(bf16_hi(u[j]), d.s));
  return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}
// Eight integer codes of x / s, halves to even, in [-kTop, kTop], as two's
// complement in the low bits of each; zeros for s = 0.  wide is the scale
// before it was rounded to fp16: a normal one is within 2^-11 of it, so that
// quotients reach kTop (1 + 2^-11) at most, which rounds to kTop; adding
// 1.5 * 2^23 rounds them and nothing is left to clamp.
template <int kTop>
__device__ __forceinline__ void int_codes(uint4 w, float s, float wide, uint32_t (&c)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  const Divisor d(s);
  if (s >= 0x1p-14f && wide <= 65504.0f) {  // fp16 significands are never all ones
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y = minus_quotients(bf16_lo(u[j]), bf16_hi(u[j]), s, d.nr);
      c[2 * j] = __float_as_uint(12582912.0f - y.x);
      c[2 * j + 1] = __float_as_uint(12582912.0f - y.y);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = (j & 1) ? bf16_hi(u[j >> 1]) : bf16_lo(u[j >> 1]);
    c[j] = s == 0.0f ? 0u : (uint32_t)max(-kTop, min(kTop, __float2int_rn(__fdiv_rn(x, s))));
  }
}

// Tokens [start, start + count) of row block ph = page * heads + head, quantised
// and written.  Thread th has rows it / 8 of items it = th, th + 256, ... (token
// it / 16, K or V by bit 3), dims 8 (th & 7) .. of both halves in x[i]; rows
// from count on are zeros.  codes and scales are the thread's, K's or V's.
// Every thread of the CTA calls it.
template <int KVT>
__device__ __forceinline__ void write_page(const uint4 (&x)[kItems][2], int th, int start, int count, size_t ph,
                                           uint8_t* codes, void* scales) {
  const int sub = th & (kRowThreads - 1), is_v = (th >> 3) & 1;
  if constexpr (KVT == SDVA_KV_FP8_E4M3) {
    // one scale for the page's K and one for its V
    __shared__ float s_amax[2][kThreads / 32];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kItems; ++i) m = fmaxf(m, fmaxf(amax8(x[i][0]), amax8(x[i][1])));
    // over the lanes of a warp with the same K|V (lane bit 3)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o != 8) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((th & 0x17) == 0) s_amax[is_v][th >> 5] = m;
    float* const scale = static_cast<float*>(scales) + ph;
    const float s_old = *scale;  // read by every thread before the barrier below
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, s_amax[is_v][w]);
    const float s_cand = scale_of<448>(m);
    const float s_new = start == 0 ? s_cand : (s_cand > s_old ? s_cand : s_old);
    uint8_t* const page_codes = codes + ph * kPage * kHeadDim;
    if (start > 0 && s_new > s_old) {
      // earlier tokens of the page move to the larger scale: 4 codes per item, by the threads of their half
      uint32_t* const old = reinterpret_cast<uint32_t*>(page_codes);
      for (int it = (th >> 4) * 8 + sub; it < start * (kHeadDim / 4); it += kThreads / 2) {
        const uint32_t c = old[it];
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __fdiv_rn(__fmul_rn(e4m3_to_f32((c >> (8 * j)) & 0xFFu), s_old), s_new);
        old[it] = (uint32_t)e4m3x2_from_f32(v[0], v[1]) | ((uint32_t)e4m3x2_from_f32(v[2], v[3]) << 16);
      }
    }
    const Divisor d(s_new);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int t = (th >> 4) + i * (kThreads / 16);
      if (t < count) {
        uint8_t* const out = page_codes + (size_t)(start + t) * kHeadDim + sub * 8;
        *reinterpret_cast<uint2*>(out) = e4m3x8(x[i][0], d);
        *reinterpret_cast<uint2*>(out + 64) = e4m3x8(x[i][1], d);
      }
    }
    if ((th & ~8) == 0) *scale = s_new;
  } else {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (i * (kThreads / 16) >= count) break;
      const int t = (th >> 4) + i * (kThreads / 16);
      const size_t at = ph * kPage + start + t;  // (page, kv head, token) row
      float m[2] = {amax8(x[i][0]), amax8(x[i][1])};
      if constexpr (KVT == SDVA_KV_FP8_ROW) {
        const float s = scale_of<448>(lanes_max<8>(fmaxf(m[0], m[1])));
        if (t < count) {
          const Divisor d(s);
          uint8_t* const out = codes + at * kHeadDim + sub * 8;
          *reinterpret_cast<uint2*>(out) = e4m3x8(x[i][0], d);
          *reinterpret_cast<uint2*>(out + 64) = e4m3x8(x[i][1], d);
          if (sub == 0) static_cast<float*>(scales)[at] = s;
        }
      } else {
        // a 64-dim half is one group of INT8 and, by four threads each, two of INT4
        constexpr bool kInt4 = KVT == SDVA_KV_INT4_G32;
        constexpr int kTop = kInt4 ? 7 : 127;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float wide = scale_of<kTop>(lanes_max<kInt4 ? 4 : 8>(m[h]));
          const __half s16 = __float2half_rn(fminf(wide, 65504.0f));
          if (t < count) {
            uint32_t c[8], p[2] = {0u, 0u};
            int_codes<kTop>(x[i][h], __half2float(s16), wide, c);
            if constexpr (kInt4) {
#pragma unroll
              for (int j = 0; j < 8; ++j) p[0] |= (c[j] & 0xFu) << (4 * j);
            } else {
              p[0] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
              p[1] = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
            }
            __half* const sc = static_cast<__half*>(scales);
            if constexpr (kInt4) {
              *reinterpret_cast<uint32_t*>(codes + at * (kHeadDim / 2) + 32 * h + 4 * sub) = p[0];
              if ((sub & 3) == 0) sc[at * 4 + 2 * h + (sub >> 2)] = s16;
            } else {
              *reinterpret_cast<uint2*>(codes + at * kHeadDim + 64 * h + 8 * sub) = make_uint2(p[0], p[1]);
              if (sub == 0) sc[at * 2 + h] = s16;
            }
          }
        }
      }
    }
  }
}

}  // namespace kvpage
}  // namespace sdva
