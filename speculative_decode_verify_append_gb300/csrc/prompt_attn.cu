// prompt_attn.cu -- causal attention of packed prompts over their own bf16
// keys and values, before the prompts' K/V go into the quantised cache.
//
// For row t of a lane and q head h of kv head g:  s_j = scale q_t . k_j over
// the lane's rows j <= t, out = sum_j exp(s_j - lse) v_j, lse = log sum exp s_j,
// in one pass over the keys with the running maximum and sum.
//
// A tile is 2 x T consecutive rows of one kv head, T = 128 / G: each of its
// two halves fills the 128 rows of a tensor-core tile with T tokens x G q
// heads (row r = token r / G, head r % G), so that a group's heads share the
// K/V tiles and few rows are empty whatever the group.  Twelve warps:
//   * warp 8 (loader): takes the next tile, TMA-loads its Q and the K and V
//     blocks of 128 keys into a ring of five 32 KB stages;
//   * warps 9, 10 (issuers, one per half): S = Q K^T into tensor memory, then
//     per block O += P V and the next S = Q K^T back to back.  They take
//     turns, so that one half's softmax runs under the other half's products
//     and each has its waits behind it when its turn comes.  (Untied, the
//     halves' products interleave, both halves' scores come late and their
//     softmaxes run together; one issuer for both halves spends 300 cycles
//     between two halves' products, waiting: 262 against 236 us at 8,192
//     tokens, 24 / 4 heads);
//   * warp 11 (guard): V rows behind a tile's first row are hidden from some
//     of its rows, but a weight of 0 does not hide an infinity or a NaN from
//     a product; it takes such values out of the V block in shared memory
//     before the product reads it, and marks the tile, whose rows then add
//     those they do see from global memory;
//   * warps 0-3 and 4-7 (softmax, one warpgroup per half): a thread owns a
//     row: reads its 128 scores, masks the last blocks, keeps a running
//     reference (its maximum, or one near it) and sum, writes P as bf16 over
//     the scores, in two parts, so that the PV of the first runs under the
//     weights of the second.  Once the QK of a block is done, so is the PV
//     before it (one issuer, in order), so the thread may rescale its O in
//     place when the reference moves.  At the end it divides by the sum and
//     stores.
// Where there are few tiles, one of T rows has the CTA alone (kOne): one
// issuer and one softmax warpgroup, the scores in the places of both halves in
// turns, so that a block's products run under the softmax of the one before.
// Bound by the tensor cores from some thousand tokens on (16,384 tokens of 24 /
// 4 heads 845 to 990 us with the clock that power leaves, 1,660 to 1,950 TFLOP/s,
// where a library product reaches 1,690 sustained and 1,865 in a burst; 8,192
// 226 us, 1,825), below by the chain of blocks of the longest tile, a few
// hundred cycles each for the products, the scores' way to the softmax and the
// weights' way back.
// Every wait is bounded: on timeout the CTA raises SDVA_STATUS_TIMEOUT,
// drains its copies and products, frees tensor memory and returns.
#include <math.h>

#include "sdva_internal.cuh"
#include "tc_primitives.cuh"
#include "verify_attn_tc.cuh"

namespace sdva {
namespace {

using namespace tc;

constexpr int kMaxPromptLanes = 1024;
constexpr int kBlock = 128;  // keys per K or V block
constexpr int kThreads = 384;
constexpr int kLoaderWarp = 8, kIssueWarp = 9, kGuardWarp = 11;
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register split");
constexpr int kStages = 5;
constexpr uint32_t kStageBytes = kBlock * kHeadDim * 2;  // two 64-dim panels of 128 rows x 128 bytes
constexpr uint32_t kPanel = kStageBytes / 2;
constexpr uint32_t kOffKv = 2 * kStageBytes;  // behind the Q of both halves
constexpr uint32_t kOffCtl = kOffKv + kStages * kStageBytes;
constexpr int kGuardRing = 8;  // barriers of the guard's blocks, more than there are stages
// A row's reference is the maximum of its first block of keys, and moves to a
// later maximum where that lies more than 2^kLag above it: the largest weight
// is then between 1 and 2^kLag, so that small values are not lost and the sum
// over n keys stays finite for values below 2^(127 - kLag) / n.  Few rows move:
// 4,550 tokens of 8 / 8 heads take 24.5 us with a few key channels eight times
// the rest and without.
constexpr float kLag = 8.0f;  // log2 units
constexpr float kLog2e = 1.4426950408889634f;
// tensor memory: S (fp32, 128 columns) of half s, overlaid by its P (bf16, 64 columns); O (fp32, 128 columns)
__device__ __forceinline__ uint32_t col_s(int s) { return 128u * s; }
__device__ __forceinline__ uint32_t col_o(int s) { return 256u + 128u * s; }
constexpr uint32_t kTmemCols = 512;
// kind::f16 with bf16 A and B (formats 1 at bits 7 and 10), fp32 D; Q K^T with both K-major, P V with V MN-major
constexpr uint32_t kBf16 = (1u << 7) | (1u << 10);
constexpr uint32_t kIdescQK = idesc_f16(128, kBlock, 0) | kBf16;
constexpr uint32_t kIdescPV = idesc_f16(128, kHeadDim, 1) | kBf16;

struct PromptArgs {
  const uint16_t* v;
  long long v_stride;
  const int32_t* cu;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int Hq, Hkv, G, T, span, total, num_lanes;
  float scale, scale_log2;
  long long wait_limit;
};

struct Tile {
  int row0, len;  // the lane's first row and rows; len 0: no more tiles
  int t0, hk;     // first row of the tile inside the lane, kv head
  int dirty;      // the guard took values out that some of the tile's rows see
};

// What the loader has issued: stage fills, those of them that the guard looks
// at first (bit i of recent: the fill i before the last one), Q loads, requests
// for another CTA's place and their answers.
struct Issued {
  long long fills, guarded;
  uint32_t recent, q_loads[2], asks, answers;
};

struct Ctl {
  uint64_t q_full[2], q_free[2], full[kStages], empty[kStages];
  uint64_t s_full[2], p_full[2][2], o_full[2], o_free[2], turn[2], drain[2];
  uint64_t guard[kGuardRing];
  uint64_t tile_full[2], tile_free[2], tile_guarded[2];
  alignas(16) uint32_t next_cta[4];  // the answer to a request for another CTA's place
  uint64_t next_full;
  Tile tile[2];
  Issued issued;
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kSmemBytes = 1024 + kOffCtl + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "shared memory budget");

// K/V blocks of a half whose rows end before row `end` of the lane.
__device__ __forceinline__ int blocks_to(int end) { return (end + kBlock - 1) / kBlock; }

struct Shape {
  int end, n[2], total;  // the tile's last row + 1; blocks of each half; blocks loaded
  __device__ Shape(const Tile& t, int T, int span) {
    end = (int)min((long long)t.t0 + span, (long long)t.len);
    n[0] = blocks_to(min(t.t0 + T, t.len));
    n[1] = end - t.t0 > T ? blocks_to(end) : 0;
    total = max(n[0], n[1]);
  }
};

// The first V block with rows that some row of the tile does not see.
__device__ __forceinline__ int guard_from(const Tile& t) { return (t.t0 + 1) / kBlock; }

// Which tile comes r-th.  Tiles are ordered with the longest rows first over
// all lanes (a tile's work grows with its position); the grid has a CTA per
// tile, and a CTA that runs takes over the next one that has not started, so
// that the work is dealt as it is done and ends with the shortest tiles.  A
// lane with n tiles has one at each position below n; between two successive
// tile counts of the batch the number of lanes that reach a position stays the
// same, which turns a rank into a position by one division per distinct count.
// The ranks a CTA gets grow, so it keeps its place.  (Where the longest chain
// of blocks outlasts the rest, halves that share T rows and take every other
// block would halve it, but each block then serves half as many rows: 2,048
// tokens 37.5 against 26.8 us.)
struct Order {
  const int32_t* cu;
  int B, span, lane;
  int cur, next;         // tile counts: the largest not yet passed, the one below
  uint32_t count, base;  // lanes that reach `cur`, tiles of longer positions

  __device__ int tiles(int b) const { return (int)((uint32_t)(cu[b + 1] - cu[b] + span - 1) / (uint32_t)span); }
  __device__ void scan() {
    uint32_t c = 0;
    int m = 0;
    for (int b = lane; b < B; b += 32) {
      const int n = tiles(b);
      if (n >= cur) ++c;
      else m = max(m, n);
    }
    count = __reduce_add_sync(0xffffffffu, c);
    next = __reduce_max_sync(0xffffffffu, m);
  }
  __device__ void init(const int32_t* cu_, int B_, int span_, int lane_) {
    cu = cu_;
    B = B_;
    span = span_;
    lane = lane_;
    base = 0;
    cur = 0x7fffffff;
    scan();
    cur = next;
    if (cur > 0) scan();
  }
  // lane and position of tile r; false when there is none
  __device__ bool find(uint32_t r, int* b_out, int* pos) {
    if (r < base) init(cu, B, span, lane);
    while (cur > 0 && r - base >= count * (uint32_t)(cur - next)) {
      base += count * (uint32_t)(cur - next);
      cur = next;
      if (cur > 0) scan();
    }
    if (cur <= 0) return false;
    const uint32_t o = r - base;
    *pos = cur - 1 - (int)(o / count);
    uint32_t k = o % count;  // the k-th lane of those that reach cur
    for (int b = 0; b < B; b += 32) {
      const bool mine = b + lane < B && tiles(min(b + lane, B - 1)) >= cur;
      const uint32_t has = __ballot_sync(0xffffffffu, mine), c = __popc(has);
      if (k < c) {
        *b_out = b + __ffs(__ballot_sync(0xffffffffu, mine && __popc(has & ((1u << lane) - 1u)) == k)) - 1;
        return true;
      }
      k -= c;
    }
    return false;
  }
};

__device__ __forceinline__ void give_up(Ctl* ctl, int32_t* status) {
  if ((threadIdx.x & 31) == 0) {
    ctl->abort = 1;
    raise_status(status, SDVA_STATUS_TIMEOUT);
  }
}

// One barrier with its phase, as one role sees it.
struct Phase {
  uint32_t bit = 0;
  __device__ uint32_t take() {
    const uint32_t b = bit;
    bit ^= 1u;
    return b;
  }
};

// A place in the ring of stages and the parity its fill completes with.
struct Ring {
  uint32_t st = 0, phase = 0;
  __device__ void next() {
    if (++st == kStages) {
      st = 0;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Bits 15 and 31 of the result: whether some bf16 of the words has an exponent
// of all ones (the addition carries into those bits).
__device__ __forceinline__ uint32_t nonfinite_bits(uint4 w) {
  return ((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u) |
         ((w.z & 0x7F807F80u) + 0x00800080u) | ((w.w & 0x7F807F80u) + 0x00800080u);
}

// Lane q of four holds the 16-byte units 0 .. 3 of its row q and gets unit q of the four rows.
__device__ __forceinline__ uint4 shfl_xor4(uint4 v, int m) {
  return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, m), __shfl_xor_sync(0xffffffffu, v.y, m),
                    __shfl_xor_sync(0xffffffffu, v.z, m), __shfl_xor_sync(0xffffffffu, v.w, m));
}
__device__ __forceinline__ void quad_transpose(uint4 (&u)[4]) {
#pragma unroll
  for (int m = 1; m <= 2; m *= 2) {
    const bool high = threadIdx.x & m;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (!(k & m)) {
        const uint4 got = shfl_xor4(high ? u[k] : u[k + m], m);
        if (high) u[k] = got;
        else u[k + m] = got;
      }
  }
}

template <bool kOne>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const PromptArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const gen = smem_raw + (base - smem_u32(smem_raw));
  Ctl* const ctl = reinterpret_cast<Ctl*>(gen + kOffCtl);
  // broadcast: the compiler then knows it, and what follows from it, to be the same for the whole warp
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  Order order;  // the loader's; safe to set up from offsets that turn out bad
  if (warp == kLoaderWarp) {
    if (lane < 3) prefetch_tmap(lane == 0 ? &mq : lane == 1 ? &mk : &mv);
    order.init(a.cu, a.num_lanes, a.span, lane);
  } else if (warp == kGuardWarp) {
    tmem_alloc(smem_u32(&ctl->tmem_base), kTmemCols);
  } else if (threadIdx.x == kIssueWarp * 32) {
    mbar_init(smem_u32(&ctl->next_full), 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&ctl->full[i]), 1);
      mbar_init(smem_u32(&ctl->empty[i]), kOne ? 1 : 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl->q_full[i]), 1);
      mbar_init(smem_u32(&ctl->q_free[i]), 1);
      mbar_init(smem_u32(&ctl->turn[i]), 1);
      mbar_init(smem_u32(&ctl->drain[i]), 1);
      mbar_init(smem_u32(&ctl->s_full[i]), 1);
      mbar_init(smem_u32(&ctl->p_full[i][0]), 4);
      mbar_init(smem_u32(&ctl->p_full[i][1]), 4);
      mbar_init(smem_u32(&ctl->o_full[i]), 1);
      mbar_init(smem_u32(&ctl->o_free[i]), 4);
      mbar_init(smem_u32(&ctl->tile_full[i]), 1);
      mbar_init(smem_u32(&ctl->tile_free[i]), kOne ? 6 : 11);  // the issuers, the guard, the softmax warps
      mbar_init(smem_u32(&ctl->tile_guarded[i]), 1);
    }
    for (int i = 0; i < kGuardRing; ++i) mbar_init(smem_u32(&ctl->guard[i]), 1);
    ctl->abort = 0;
    mbar_fence_init();
    mbar_arrive(smem_u32(&ctl->turn[0]));  // the first half begins
  }
  int bad = 0;
  for (int i = threadIdx.x; i < a.num_lanes; i += kThreads) {
    const int lo = a.cu[i], hi = a.cu[i + 1];
    bad |= lo < 0 || hi < lo || hi > a.total;
  }
  fence_before_sync();
  bad = __syncthreads_or(bad);
  fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  volatile int* const abort_flag = &ctl->abort;
  const long long limit = a.wait_limit;
  // A warp's lanes test one barrier, one flag and one clock together and so go
  // on or give up together (a vote on it costs 2%, 1,004 against 980 us at
  // 16,384 tokens of 24 / 4 heads).
  // (spinning instead of sleeping takes issue slots from the softmax: 1,496
  // against 1,524 TFLOP/s at 32,768 tokens)
  auto wait = [&](uint64_t& bar, uint32_t parity) {
    return mbar_wait<false>(smem_u32(&bar), parity, abort_flag, limit);
  };

  if (bad) {  // the same for the whole CTA
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_status(a.status, SDVA_STATUS_BAD_COUNT);
  } else if (warp >= kLoaderWarp) {
    regs_decrease<kRegsOther>();
    bool ok = true;
    if (warp == kLoaderWarp) {
      const uint32_t half_bytes = (uint32_t)(a.G * a.T) * 128u;  // one 64-dim panel of one half's Q
      long long fills = 0;  // stage fills issued
      uint32_t q_loads[2] = {0, 0};
      long long guard0 = 0;  // guarded blocks issued
      uint32_t recent = 0;   // bit i: whether the fill i before the last one was such a block
      // a V block that the guard looks at first lands on the guard's barrier; the guard passes it on
      auto load = [&](const CUtensorMap* map, int hk, int row, bool guarded) {
        const int s = (int)(fills % kStages);
        if (fills >= kStages && !wait(ctl->empty[s], (uint32_t)((fills / kStages - 1) & 1))) return false;
        if (lane == 0) {
          const uint32_t bar = smem_u32(guarded ? &ctl->guard[guard0 % kGuardRing] : &ctl->full[s]);
          const uint32_t dst = base + kOffKv + s * kStageBytes;
          mbar_arrive_expect_tx(bar, kStageBytes);
          tma_load_3d(dst, map, 0, hk, row, bar);
          tma_load_3d(dst + kPanel, map, 64, hk, row, bar);
        }
        __syncwarp();
        ++fills;
        guard0 += guarded;
        recent = recent << 1 | (uint32_t)guarded;
        return true;
      };
      uint32_t r = blockIdx.x;
      Tile t;
      auto locate = [&]() {
        int b, pos;
        t = {0, 0, 0, (int)(r % (uint32_t)a.Hkv), 0};
        if (!order.find(r / (uint32_t)a.Hkv, &b, &pos)) return false;
        t.row0 = a.cu[b];
        t.len = a.cu[b + 1] - t.row0;
        t.t0 = pos * a.span;
        return true;
      };
      uint32_t asks = 0, answers = 0;
      auto ask = [&]() {
        if (lane == 0) take_over_next(smem_u32(ctl->next_cta), smem_u32(&ctl->next_full));
        __syncwarp();
        ++asks;
      };
      bool more = locate();
      for (int i = 0;; ++i) {
        const int slot = i & 1;
        if (i >= 2 && !(ok = wait(ctl->tile_free[slot], (uint32_t)((i / 2 - 1) & 1)))) break;
        if (lane == 0) {
          ctl->tile[slot] = t;
          mbar_arrive(smem_u32(&ctl->tile_full[slot]));
        }
        __syncwarp();
        if (!more) break;
        const Shape sh(t, a.T, a.span);
        const int halves = sh.n[1] ? 2 : 1;
        if (lane < 4 && (lane >> 1) < halves)  // Q waits for its place: into L2 meanwhile
          tma_prefetch_3d(&mq, 64 * (lane & 1), t.hk * a.G, t.row0 + t.t0 + (lane >> 1) * a.T);
        __syncwarp();
        // the first K and V do not wait for the tile before
        if (!(ok = load(&mk, t.hk, t.row0, false) && load(&mv, t.hk, t.row0, guard_from(t) == 0))) break;
        for (int s = 0; s < halves; ++s) {
          if (q_loads[s] > 0 && !(ok = wait(ctl->q_free[s], (q_loads[s] - 1) & 1u))) break;
          if (lane == 0) {
            const uint32_t bar = smem_u32(&ctl->q_full[s]);
            mbar_arrive_expect_tx(bar, half_bytes * 2u);
            for (int p = 0; p < 2; ++p)
              tma_load_3d(base + s * kStageBytes + p * kPanel, &mq, 64 * p, t.hk * a.G, t.row0 + t.t0 + s * a.T, bar);
          }
          __syncwarp();
          ++q_loads[s];
        }
        if (!ok) break;
        for (int j = 1; j < sh.total && ok; ++j)
          ok = load(&mk, t.hk, t.row0 + j * kBlock, false) &&
               load(&mv, t.hk, t.row0 + j * kBlock, j >= guard_from(t));
        if (!ok) break;
        // The next tile, asked for when the last blocks of this one are on
        // their way (asked for at its start, the CTAs with the longest tiles
        // take a second one before others are free: 8,192 tokens of 8 / 8
        // heads 124 against 92 us).  Places behind the last tile are taken
        // over too, so that no CTA starts for them.
        ask();
        t = {0, 0, 0, 0, 0};
        more = false;
        while (!more && (ok = wait(ctl->next_full, answers & 1u))) {
          ++answers;
          if (!taken_over(smem_u32(ctl->next_cta), &r)) break;
          fence_proxy_async_smem();  // the answer is read before the next one is written
          __syncwarp();
          if (!(more = locate())) ask();
        }
        if (!ok) break;
      }
      if (!ok) give_up(ctl, a.status);
      if (lane == 0) ctl->issued = {fills, guard0, recent, {q_loads[0], q_loads[1]}, asks, answers};
      __syncwarp();
    } else if (kOne ? warp == kIssueWarp : warp == kIssueWarp || warp == kIssueWarp + 1) {
      const int s = warp - kIssueWarp;
      // Descriptors differ in their start address alone: the low words are
      // added up from constants, so that a product costs few instructions
      // here (stage numbers by 64-bit remainders held the tensor core up by
      // 700 cycles a block: 1,566 against 1,731 TFLOP/s at 32,768 tokens).
      const uint64_t q_desc = sdesc_sw128(base + s * kStageBytes, 1024, 1024);
      const uint64_t k_desc = sdesc_sw128(base + kOffKv, 1024, 1024);
      const uint64_t v_desc = sdesc_sw128(base + kOffKv, kPanel, 1024);
      constexpr uint64_t kStage16 = kStageBytes >> 4, kPanel16 = kPanel >> 4;
      const uint32_t d_o = tmem + col_o(s);
      Ring ring;
      Phase p_phase, o_phase, q_phase, turn_phase;
      bool used = false;
      // S of place b = Q K^T with the K block of stage st
      auto qk = [&](uint32_t st, int b) {
        const uint32_t d_s = tmem + col_s(b);
        const uint64_t kd = k_desc + st * kStage16;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_f16_ss(d_s, q_desc + kPanel16 * (k >> 2) + 2 * (k & 3), kd + kPanel16 * (k >> 2) + 2 * (k & 3), kIdescQK,
                     k != 0);
        mma_commit(smem_u32(&ctl->s_full[b]));
        mma_commit(smem_u32(&ctl->empty[st]));
      };
      // O (+)= P V with keys 64 part .. + 63 of the V block of stage st
      auto pv = [&](uint32_t st, int b, int part, bool add) {
        const uint32_t d_s = tmem + col_s(b);
        const uint64_t vd = v_desc + st * kStage16;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_ts(d_o, d_s + 32 * part + 8 * k, vd + 512 * part + 128 * k, kIdescPV, add || k != 0);
      };
      auto take_turn = [&]() { return wait(ctl->turn[s], turn_phase.take()); };
      auto pass_turn = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->turn[s ^ 1]));
      };
      // a stage that only the other half reads
      auto leave = [&](Ring r) {
        if (!wait(ctl->full[r.st], r.phase)) return false;
        if (lane == 0) mbar_arrive(smem_u32(&ctl->empty[r.st]));
        return true;
      };
      // One half: its scores go to the places of both halves in turns, so that
      // the next ones are there when a block's weights are.
      uint32_t places = 0;  // bit b: the parity of place b's next weights
      for (int i = 0; kOne && ok; ++i) {
        const int slot = i & 1;
        if (!(ok = wait(ctl->tile_full[slot], (uint32_t)((i / 2) & 1)))) break;
        const Tile t = ctl->tile[slot];
        if (t.len == 0) break;
        const Shape sh(t, a.T, a.span);
        const int n = __shfl_sync(0xffffffffu, sh.n[0], 0);
        Ring k = ring, v = ring;
        v.next();
        // the scores of block j
        auto scores = [&](int j) {
          if (!wait(ctl->full[k.st], k.phase)) return false;
          fence_after_sync();
          if (elect_one()) {
            qk(k.st, j & 1);
            if (j + 1 == n) mma_commit(smem_u32(&ctl->q_free[0]));
          }
          __syncwarp();
          k.next();
          k.next();
          return true;
        };
        if (!(ok = wait(ctl->q_full[0], q_phase.take()) && scores(0) && (n == 1 || scores(1)))) break;
        for (int j = 0; j < n; ++j) {
          const int b = j & 1;
          const uint32_t phase = (places >> b) & 1u;
          places ^= 1u << b;
          if (!(ok = wait(ctl->full[v.st], v.phase) && (j > 0 || !used || wait(ctl->o_free[0], o_phase.take())) &&
                     wait(ctl->p_full[b][0], phase)))
            break;
          fence_after_sync();
          if (elect_one()) pv(v.st, b, 0, j > 0);
          __syncwarp();
          if (!(ok = wait(ctl->p_full[b][1], phase))) break;
          fence_after_sync();
          if (elect_one()) {
            pv(v.st, b, 1, true);
            mma_commit(smem_u32(&ctl->empty[v.st]));
            mma_commit(smem_u32(&ctl->o_full[1]));  // O holds the blocks so far
            if (j + 1 == n) mma_commit(smem_u32(&ctl->o_full[0]));
          }
          __syncwarp();
          v.next();
          v.next();
          if (j + 2 < n && !(ok = scores(j + 2))) break;
        }
        if (!ok) break;
        used = true;
        ring = k;
        if (lane == 0) mbar_arrive(smem_u32(&ctl->tile_free[slot]));
        __syncwarp();
      }
      for (int i = 0; !kOne && ok; ++i) {
        const int slot = i & 1;
        if (!(ok = wait(ctl->tile_full[slot], (uint32_t)((i / 2) & 1)))) break;
        const Tile t = ctl->tile[slot];
        if (t.len == 0) break;
        const Shape sh(t, a.T, a.span);
        const int n = __shfl_sync(0xffffffffu, sh.n[s], 0), total = __shfl_sync(0xffffffffu, sh.total, 0);
        if (n > 0 && !(ok = wait(ctl->q_full[s], q_phase.take()) && wait(ctl->full[ring.st], ring.phase))) break;
        if (!(ok = take_turn())) break;
        if (n > 0) {
          fence_after_sync();
          if (elect_one()) {
            qk(ring.st, s);
            if (n == 1) mma_commit(smem_u32(&ctl->q_free[s]));
          }
        }
        pass_turn();
        if (n == 0 && !(ok = leave(ring))) break;
        ring.next();
        for (int j = 0; j < total && ok; ++j) {
          const Ring v = ring;  // V of block j, K of block j + 1
          ring.next();
          const Ring k = ring;
          if (j + 1 < total) ring.next();
          if (j >= n) {
            if (!(ok = take_turn())) break;
            pass_turn();
            ok = leave(v) && (j + 1 == total || leave(k));
            continue;
          }
          const bool more = j + 1 < n;
          const uint32_t phase = p_phase.take();
          if (!(ok = wait(ctl->full[v.st], v.phase) && (!more || wait(ctl->full[k.st], k.phase)) &&
                     (j > 0 || !used || wait(ctl->o_free[s], o_phase.take())) && wait(ctl->p_full[s][0], phase) &&
                     take_turn()))
            break;
          fence_after_sync();
          if (elect_one()) pv(v.st, s, 0, j > 0);
          __syncwarp();
          if (!(ok = wait(ctl->p_full[s][1], phase))) break;
          fence_after_sync();
          if (elect_one()) {
            pv(v.st, s, 1, true);
            mma_commit(smem_u32(&ctl->empty[v.st]));
            if (more) {
              qk(k.st, s);
              if (j + 2 == n) mma_commit(smem_u32(&ctl->q_free[s]));
            } else {
              mma_commit(smem_u32(&ctl->o_full[s]));
            }
          }
          pass_turn();
          if (!more && j + 1 < total) ok = leave(k);
        }
        if (!ok) break;
        used |= n > 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->tile_free[slot]));
      }
      if (!ok) give_up(ctl, a.status);
      // the tensor core is done with everything this warp issued (bounded)
      if (elect_one()) mma_commit(smem_u32(&ctl->drain[s]));
      __syncwarp();
      int none = 0;
      mbar_wait<false>(smem_u32(&ctl->drain[s]), 0, &none, 400000000LL);
    } else if (warp == kGuardWarp) {
      long long stage0 = 0, guard0 = 0;
      for (int i = 0; ok; ++i) {
        const int slot = i & 1;
        if (!(ok = wait(ctl->tile_full[slot], (uint32_t)((i / 2) & 1)))) break;
        const Tile t = ctl->tile[slot];
        if (t.len == 0) break;
        const Shape sh(t, a.T, a.span);
        for (int j = guard_from(t); j < sh.total; ++j, ++guard0) {
          const long long f = stage0 + 2 * j + 1;
          if (!(ok = wait(ctl->guard[guard0 % kGuardRing], (uint32_t)((guard0 / kGuardRing) & 1)))) break;
          uint8_t* const vt = gen + kOffKv + (uint32_t)(f % kStages) * kStageBytes;
          const int from = max(0, t.t0 + 1 - j * kBlock) * 128;  // bytes of the rows every row of the tile sees
          uint32_t found = 0;
#pragma unroll 4
          for (int o = from + 16 * lane; o < (int)kPanel; o += 512)
            found |= nonfinite_bits(*reinterpret_cast<const uint4*>(vt + o)) |
                     nonfinite_bits(*reinterpret_cast<const uint4*>(vt + kPanel + o));
          if (__any_sync(0xffffffffu, (found & 0x80008000u) != 0)) {
            bool seen = false;
            for (int o = from + 2 * lane; o < (int)kPanel; o += 64)
              for (int p = 0; p < 2; ++p) {
                uint16_t* const x = reinterpret_cast<uint16_t*>(vt + p * kPanel + o);
                if ((*x & 0x7F80u) == 0x7F80u) {
                  *x = 0;
                  seen |= j * kBlock + o / 128 < sh.end;
                }
              }
            if (__any_sync(0xffffffffu, seen) && lane == 0) ctl->tile[slot].dirty = 1;
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(smem_u32(&ctl->full[f % kStages]));
          __syncwarp();
        }
        if (!ok) break;
        stage0 += 2 * sh.total;
        if (lane == 0) {
          mbar_arrive(smem_u32(&ctl->tile_guarded[slot]));
          mbar_arrive(smem_u32(&ctl->tile_free[slot]));
        }
        __syncwarp();
      }
      if (!ok) give_up(ctl, a.status);
    }
  } else if (!kOne || warp < 4) {
    regs_increase<kRegsSoftmax>();
    const int s = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // TMEM lane 32 * (warp % 4) in bits 16 and up
    const uint32_t t_o = tmem + lane_base + col_o(s);
    const int r_tok = row / a.G, r_head = row % a.G;
    const int w_tok = (row & ~31) / a.G;  // the warp's first token
    const float ninf = __int_as_float(0xff800000);
    Phase s_phase, o_phase;
    uint32_t places = 0;  // bit b: the parity of place b's next scores
    uint32_t before = 0;  // blocks of the tiles before
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const int slot = i & 1;
      if (!(ok = wait(ctl->tile_full[slot], (uint32_t)((i / 2) & 1)))) break;
      const Tile t = ctl->tile[slot];
      if (t.len == 0) break;
      const Shape sh(t, a.T, a.span);
      const int n = sh.n[s], first = t.t0 + s * a.T;
      const int tok = first + r_tok;
      const bool valid = r_tok < a.T && tok < t.len;
      // The largest weight of a row with few keys is 1, and rounding it to bf16
      // costs nothing, which is most of the error there (against fp64, of the
      // output's norm: one key 0 instead of 1.4e-3, four 1.4e-3 instead of
      // 2.1e-3, 1.3e-3 of it from rounding the output).
      float m = ninf, l = 0.0f;
      for (int j = 0; j < n; ++j) {
        const int b = kOne ? j & 1 : s;  // the place of the block's scores and weights
        const uint32_t t_s = tmem + lane_base + col_s(b);
        const uint32_t s_parity = kOne ? (places >> b) & 1u : s_phase.take();
        places ^= 1u << b;
        if (!(ok = wait(ctl->s_full[b], s_parity))) break;
        fence_after_sync();
        uint32_t x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, x[c]);
        tmem_wait_ld();
        if ((j + 1) * kBlock > first + w_tok + 1) {  // some row of the warp does not see the whole block
          const int seen = tok - j * kBlock + 1;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int left = min(max(seen - 32 * c, 0), 32);
            const uint32_t hidden = left == 32 ? 0u : 0xffffffffu << left;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (hidden & (1u << k)) x[c][k] = 0xff800000u;
          }
        }
        // The weights of the first 64 keys are taken about the reference that
        // the row has, beside this block's maximum (64 three-way maxima are a
        // third of the work on a block); only where that lies too far off, as in
        // the first block, are they taken again.
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = fmaxf(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]));
#pragma unroll
          for (int k = 2; k < 32; k += 2)
            mx[c] = fmax3(mx[c], __uint_as_float(x[c][k]), __uint_as_float(x[c][k + 1]));
        }
        const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
        uint32_t p[32];
        unsigned long long sum0, sum1;
        // weights of the 64 keys of chunks c0 and c0 + 1, added to the sums
        auto weights = [&](int c0) {
          // no reference yet, or all scores -inf so far: weights of 0
          const float shift = m == ninf ? 0.0f : -m * a.scale_log2;
          const unsigned long long sc2 = f2_pack(a.scale_log2, a.scale_log2), sh2 = f2_pack(shift, shift);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float2 e = f2_unpack(
                  ffma2(f2_pack(__uint_as_float(x[c0 + c][k]), __uint_as_float(x[c0 + c][k + 1])), sc2, sh2));
              const float e0 = fast_exp2(e.x), e1 = fast_exp2(e.y);
              if (k & 2) sum1 = fadd2(sum1, f2_pack(e0, e1));
              else sum0 = fadd2(sum0, f2_pack(e0, e1));
              p[16 * c + k / 2] = pack_bf16x2(e0, e1);
            }
        };
        auto hand_over = [&](int part) {
          tmem_st32(t_s + 32 * part, p);
          tmem_wait_st();
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl->p_full[b][part]));
        };
        sum0 = sum1 = 0ull;
        weights(0);
        // from -inf, at j = 0, any maximum is far; no NaN moves the reference
        const bool move = (top - m) * a.scale_log2 > kLag;
        if (__any_sync(0xffffffffu, move && valid)) {
          const float f = move ? fast_exp2((m - top) * a.scale_log2) : 1.0f;
          if (move) m = top;
          if (j > 0) {
            // with one half the scores run ahead of O
            if (kOne && !(ok = wait(ctl->o_full[1], (before + j - 1) & 1u))) break;
            if (kOne) fence_after_sync();
            l *= f;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tmem_ld16(t_o + 16 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(t_o + 16 * c, o);
            }
          }
          sum0 = sum1 = 0ull;
          weights(0);
        }
        hand_over(0);
        weights(2);
        const float2 sum = f2_unpack(fadd2(sum0, sum1));
        l += sum.x + sum.y;
        hand_over(1);
      }
      if (!ok) break;
      before += n;
      if (!(ok = wait(ctl->tile_guarded[slot], (uint32_t)((i / 2) & 1)))) break;
      const bool dirty = ctl->tile[slot].dirty != 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->tile_free[slot]));
      if (n == 0) continue;
      if (!(ok = wait(ctl->o_full[s], o_phase.take()))) break;
      fence_after_sync();
      const float inv = 1.0f / l;
      // where this lane's four rows of the tile lie behind its first (-1: nowhere)
      const int own_at = valid ? r_tok * a.Hq + r_head : -1;
      int at4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) at4[k] = __shfl_sync(0xffffffffu, own_at, (lane & ~3) + k);
      uint16_t* const tile_out = a.out + ((size_t)(t.row0 + first) * a.Hq + (size_t)t.hk * a.G) * kHeadDim;
      const size_t at = (size_t)(t.row0 + tok) * a.Hq + (size_t)t.hk * a.G + r_head;
      uint32_t all[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_o + 32 * c, all[c]);
      tmem_wait_ld();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->o_free[s]));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t(&o)[32] = all[c];
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * inv);
        if (dirty && valid) {
          // infinities and NaN that the guard took out, from the rows this one sees
          for (int key = t.t0 + 1; key <= tok; ++key) {
            const uint16_t* v = a.v + (size_t)(t.row0 + key) * a.v_stride + (size_t)t.hk * kHeadDim + 32 * c;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const uint32_t w = v[k];
              if ((w & 0x7F80u) == 0x7F80u)
                o[k] = __float_as_uint(__uint_as_float(o[k]) + __uint_as_float(w << 16));
            }
          }
        }
        // A row's 64 bytes go out by four lanes: of its own row a lane would
        // write 16 bytes into a line of its own each time, 32 lines to a store,
        // and every shared-memory access of the SM queues behind them (228
        // prompts of 42 rows, 24 / 4 heads, 45.5 against 36.4 us; three of 4,096
        // with 32 / 8 heads 254 against 243).
        uint4 u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          u[k] = make_uint4(pack_bf16x2(__uint_as_float(o[8 * k]), __uint_as_float(o[8 * k + 1])),
                            pack_bf16x2(__uint_as_float(o[8 * k + 2]), __uint_as_float(o[8 * k + 3])),
                            pack_bf16x2(__uint_as_float(o[8 * k + 4]), __uint_as_float(o[8 * k + 5])),
                            pack_bf16x2(__uint_as_float(o[8 * k + 6]), __uint_as_float(o[8 * k + 7])));
        quad_transpose(u);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (at4[k] >= 0) *reinterpret_cast<uint4*>(tile_out + at4[k] * kHeadDim + 32 * c + 8 * (lane & 3)) = u[k];
      }
      if (valid && a.lse != nullptr) a.lse[at] = m * a.scale + logf(l);
    }
    if (!ok) give_up(ctl, a.status);
  }

  fence_before_sync();
  __syncthreads();
  if (warp == kGuardWarp) {
    fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  } else if (warp == kLoaderWarp && ctl->abort) {
    // No copy outlives the CTA, whichever warp gave up (bounded; where none
    // did, all were waited for).  A block that the guard has not passed on
    // completes the guard's barrier alone.
    const Issued n = ctl->issued;
    int none = 0;
    long long g = n.guarded;
    for (long long f = n.fills - 1; f >= 0 && f >= n.fills - kStages; --f) {
      const bool guarded = n.recent >> (n.fills - 1 - f) & 1u;
      g -= guarded;
      mbar_wait<false>(smem_u32(guarded ? &ctl->guard[g % kGuardRing] : &ctl->full[f % kStages]),
                       (uint32_t)((guarded ? g / kGuardRing : f / kStages) & 1), &none, 400000000LL);
    }
    if (n.asks > n.answers) mbar_wait<false>(smem_u32(&ctl->next_full), n.answers & 1u, &none, 400000000LL);
    for (int s = 0; s < 2; ++s)
      if (n.q_loads[s]) mbar_wait<false>(smem_u32(&ctl->q_full[s]), (n.q_loads[s] - 1) & 1u, &none, 400000000LL);
  }
}

// rows x heads x 128 bf16 with `stride` elements between rows, loaded in boxes
// of 64 dims x `heads` heads x `rows` rows with the 128-byte swizzle
bool encode_rows(CUtensorMap* m, const void* p, int64_t stride, int num_heads, int total, int heads, int rows) {
  EncodeTiledFn enc = encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)num_heads, (cuuint64_t)total};
  cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)rows};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace sdva

using namespace sdva;

extern "C" int prompt_attn(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, int num_q_heads, int num_kv_heads, int total_tokens,
                           const int32_t* cu_tokens, int num_lanes, float sm_scale, void* out, float* lse,
                           int32_t* status, sdva_stream_t stream) {
  if (total_tokens == 0) return SDVA_OK;
  if (q == nullptr || k == nullptr || v == nullptr || cu_tokens == nullptr || out == nullptr) return SDVA_ERR_INVALID;
  if (total_tokens < 0 || num_lanes <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_q_heads % num_kv_heads != 0 || !(sm_scale > 0.0f) || !isfinite(sm_scale))
    return SDVA_ERR_INVALID;
  const int64_t qw = (int64_t)num_q_heads * kHeadDim, kw = (int64_t)num_kv_heads * kHeadDim;
  if (q_stride < qw || k_stride < kw || v_stride < kw || ((q_stride | k_stride | v_stride) & 7) ||
      ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
        reinterpret_cast<uintptr_t>(out)) &
       15u))
    return SDVA_ERR_INVALID;
  const int G = num_q_heads / num_kv_heads;
  if (num_lanes > kMaxPromptLanes || G > 128 || num_kv_heads > 65535) return SDVA_ERR_UNSUPPORTED;
  PromptArgs a;
  a.v = static_cast<const uint16_t*>(v);
  a.v_stride = v_stride;
  a.cu = cu_tokens;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = status;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.G = G;
  a.T = 128 / G;
  a.total = total_tokens;
  a.num_lanes = num_lanes;
  a.scale = sm_scale;
  a.scale_log2 = sm_scale * kLog2e;
  a.wait_limit = wait_limit();
  CUtensorMap mq, mk, mv;
  if (!encode_rows(&mq, q, q_stride, num_q_heads, total_tokens, G, a.T) ||
      !encode_rows(&mk, k, k_stride, num_kv_heads, total_tokens, 1, kBlock) ||
      !encode_rows(&mv, v, v_stride, num_kv_heads, total_tokens, 1, kBlock))
    return SDVA_ERR_CUDA;
  // One half to a tile where two would not give each SM a tile (a lane counted
  // with half a tile for its ragged end): its chain of blocks is the shorter
  // one, 1,200 to 1,900 cycles a block against 2,150 for two halves, whose blocks
  // serve twice the rows.  2,048 tokens of 8 / 8 heads 20.4 against 26.4 us, 4,096
  // 33.2 / 45.0, 16,384 of 2 / 1 104 / 149, 1,200 of 32 / 8 (154 tiles on 152 SMs)
  // 19.5 / 20.2, 512 of 24 / 4 10.1 / 12.0; 1,300 of 32 / 8 (166) 23.2 / 21.1, 2,048 of
  // 24 / 4 (197) 31.5 / 27.8, eight ragged prompts (447) 49.1 / 39.0.
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SDVA_ERR_CUDA;
  const long long rows = (long long)total_tokens + (long long)a.T * num_lanes;
  a.span = 20 * rows * num_kv_heads <= 21LL * sms * 2 * a.T ? a.T : 2 * a.T;
  // at most this many tiles: one per span of rows and a ragged one per lane
  const long long tiles = ((long long)total_tokens / a.span + num_lanes) * num_kv_heads;
  if (tiles > 0x7fffffffLL) return SDVA_ERR_UNSUPPORTED;  // more rows of K and V than memory holds
  // the shared-memory limit is a per-device attribute of the function: set it
  // on every call, for the device current now
  const auto kernel = a.span == a.T ? prompt_attn_kernel<true> : prompt_attn_kernel<false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes) !=
      cudaSuccess)
    return SDVA_ERR_CUDA;
  kernel<<<(unsigned)tiles, kThreads, kSmemBytes,
                       reinterpret_cast<cudaStream_t>(stream)>>>(mq, mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? SDVA_OK : SDVA_ERR_CUDA;
}
