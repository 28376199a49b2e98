// What the attention kernels of the bf16 pool share (sm_103a): their arguments,
// how a tile's rows and keys are found, the warp role of decode, tensor maps of
// a pool, tcgen05 issue helpers.  attention_tc.cu has the plain kernels,
// attention_mod.cu those with modified scores (MOD).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>

#include "ptx_util.cuh"
#include "rx.h"
#include "rx_internal.h"
#include "tc_util.cuh"

// Of each file that includes this.  Bit 0: a slot outside [0, num_slots) was
// read (slot 0 used instead); bit 1: a barrier wait timed out; bit 2: a tile
// found its dynamic shared memory off a 1024-byte boundary and did nothing.
// Read by rx_device_check().
static __device__ int32_t g_tc_error;

namespace {

using bf16 = __nv_bfloat16;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr long long kWaitLimit = 4000000000LL;  // clock cycles (~2 s)
constexpr float kRescaleThreshold = 8.0f;       // log2 units
constexpr uint32_t kSleepNs = 0;                // MMA / loader waits: plain try_wait polling
constexpr float kMasked = -1.0e30f;             // raw score of a masked key
constexpr int kExtendInterleaveWaves = 8;
// Extend CTA order: heads interleaved also when one request's keys over all
// KV heads (K and V, bf16) take at most this much: the row tiles in flight
// then read a few requests' keys, which stay in L2 for every head at once.
constexpr int64_t kExtendInterleaveKvBytes = 32ll << 20;
constexpr int BM = 128;

// Division of 0 <= n < 2^31 by a constant d >= 1 of the launch: (n * mul) >> shift
// with mul = ceil(2^shift / d) and shift = 31 + ceil(log2 d) is exact there (mul d
// - 2^shift <= 2^(shift - 31)).  A division by a value the compiler does not know
// is a chain of some thirty instructions, and a tile's description, its rows' offsets
// and each unit's start hold several: when the tile took 217 us for a prompt of
// 8,191 tokens in a window of 1,024 and 108 for 5 prompts of 1,500 to 2,500 tokens in
// documents of 400, the operator made them 222 and 113.
struct Div {
  uint32_t mul, shift;
  __device__ __forceinline__ int operator()(int n) const {
    return int((uint64_t(uint32_t(n)) * mul) >> shift);
  }
};
inline Div make_div(int d) {
  int s = 0;
  while ((1ll << s) < d) ++s;
  const uint64_t two = 1ull << (31 + s);
  return Div{uint32_t((two + uint64_t(d) - 1) / uint64_t(d)), uint32_t(31 + s)};
}

struct TcArgs {
  const bf16* q;
  const bf16* kpool;  // layer base, [Hkv][num_slots][D]
  const bf16* vpool;
  int64_t head_stride;
  int64_t num_slots;
  const int32_t* table;
  int64_t row_stride;
  int hq;
  int group;
  float scale_log2;
  // extend
  const int32_t* req_rows;
  const int32_t* prefix_len;
  const int32_t* qo_indptr;
  const int32_t* tile_indptr;
  int num_req;
  int num_tiles;
  int heads_interleaved;   // extend CTA order: 1 = tile-major over heads, 0 = head-major
  float* out;
  float* lse;
  int64_t tma_row_base;  // row of (layer, KV head 0, slot 0) in the tensor maps
  int64_t tma_head_rows; // rows per KV head (num_slots)
  // decode
  const int32_t* work;     // tensor-core items
  const int32_t* members;
  float* ws_o;
  float* ws_lse;
  // fused decode: warp-role items (<= 16 rows) and the step's new tokens
  const int32_t* work_small;
  int n_small_units;       // warp-role (item, KV head) units
  int n_tc_ctas;           // tensor-core CTAs
  int n_warp_first;        // warp-role-only CTAs placed before them
  int* unit_counter;       // next warp-role unit to take (0 at launch)
  int tiles_leave;         // decode: tile CTAs exit after their tile
  int early_inputs;        // decode: the tiles may read Q and shared-segment keys
                           // before griddepcontrol.wait (see decode_fused)
  int step;                // step index within a multi-step plan
  const bf16* k_new;       // bf16 [B][Hkv][D] of the step's tokens, or NULL
  const bf16* v_new;
  const int32_t* slots_new;
  // modified scores (the MOD kernels only; rx_score_mod)
  float cap_in;            // scale / softcap, 0: no cap
  float cap_out;           // softcap * log2(e)
  float cap_poly[7];       // of tanh (kTanh), times cap_out
  float2 cap_fold2[5];     // of kTanhNear with cap_in and cap_out in it, twice: a raw
  float cap_near;          // score of at most this magnitude times a polynomial in its
                           // square
  float cap_ref;           // the reference of every row's weights, or -inf: none fits
  int window;              // 0: none
  const float* slopes;
  const int32_t* key_begin;
  const int32_t* bidir_end;
  const int32_t* ctx_len;
  int out_bf16;
  int q_boxes;             // Q's whole row tiles are loaded by boxes
  int hkv;
  Div by_group, by_hkv;    // division by them
};

// A loader's mark, in a slot's place, for a key outside its range.  MOD: not -1, which
// a table may hold by mistake and which is flagged as any slot outside the pool.
template <bool MOD>
constexpr int32_t kNoKey = MOD ? INT32_MIN : -1;

struct TileDesc {
  const int32_t* trow;
  int key_begin, key_end, nomask_end, n_rows;
  int gr0, q_base, prefix;
  int member_off, part_base;
  // MOD: rows see no key before key_lo (key_begin is the multiple of 16 at or
  // before it, where the 16-key groups of the loads start), and every key
  // before bidir
  int key_lo, bidir;
  int kvh;
};

// n / group, n / KV heads
template <bool MOD>
__device__ __forceinline__ int over_group(const TcArgs& a, int n) {
  if constexpr (MOD) return a.by_group(n);
  return n / a.group;
}
template <bool MOD>
__device__ __forceinline__ int over_hkv(const TcArgs& a, int n) {
  if constexpr (MOD) return a.by_hkv(n);
  return n / (a.hq / a.group);
}

template <bool DECODE, bool MOD>
__device__ __forceinline__ TileDesc describe(const TcArgs& a, int bx) {
  TileDesc t;
  t.kvh = t.key_lo = t.bidir = 0;
  if constexpr (DECODE) {
    const int32_t* w = a.work + int64_t(bx) * RX_WORK_WORDS;
    t.trow = a.table + int64_t(w[0]) * a.row_stride;
    t.key_begin = w[1];
    t.key_end = w[7] > 0 ? min(w[2], w[7] + a.step) : w[2];
    t.member_off = w[3];
    t.part_base = w[5];
    t.n_rows = w[6];
    t.nomask_end = t.key_end;
    t.gr0 = t.q_base = t.prefix = 0;
  } else {
    const int tile = a.num_tiles - 1 - bx;  // heaviest first
    // the request of this tile: the last r with tile_indptr[r] <= tile, found
    // by the warp in rounds of 32 samples (each round one load per lane and
    // a ballot) instead of a binary search's chain of dependent loads, which
    // held every CTA's start-up for several microseconds
    const int ln = int(threadIdx.x & 31);
    int lo = 0, hi = a.num_req;
    while (hi - lo > 32) {
      const int step = (hi - lo + 31) >> 5;
      const int p = lo + ln * step;
      const bool le = p < hi && __ldg(a.tile_indptr + p) <= tile;
      const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));  // lane 0's sample is <= tile
      lo = lo + k * step;
      hi = min(hi, lo + step);
    }
    {
      const int p = lo + ln;
      const bool le = p < hi && __ldg(a.tile_indptr + p) <= tile;
      lo += 31 - __clz(__ballot_sync(0xffffffffu, le));
    }
    const int G = a.group;
    t.q_base = a.qo_indptr[lo];
    const int s_r = a.qo_indptr[lo + 1] - t.q_base;
    t.prefix = a.prefix_len[lo];
    t.trow = a.table + int64_t(a.req_rows[lo]) * a.row_stride;
    t.gr0 = (tile - a.tile_indptr[lo]) * BM;
    t.n_rows = min(BM, s_r * G - t.gr0);
    t.key_begin = 0;
    t.key_end = t.prefix + over_group<MOD>(a, t.gr0 + t.n_rows - 1) + 1;
    t.nomask_end = t.prefix + over_group<MOD>(a, t.gr0) + 1;
    t.member_off = t.part_base = 0;
    if constexpr (MOD) {
      // the keys that some row of the tile sees lie in [key_begin, key_end)
      const int tok0 = t.nomask_end - 1 - t.prefix, tok1 = t.key_end - 1 - t.prefix;
      t.bidir = a.bidir_end ? min(__ldg(a.bidir_end + lo), t.prefix + s_r) : 0;
      t.key_end = max(t.key_end, t.bidir);
      if (a.window > 0) t.key_begin = max(0, t.prefix + tok0 - a.window + 1);
      if (a.key_begin) {
        int least = INT32_MAX;
        for (int tok = tok0 + ln; tok <= tok1; tok += 32)
          least = min(least, __ldg(a.key_begin + t.q_base + tok));
        t.key_begin = max(t.key_begin, __reduce_min_sync(0xffffffffu, least));
      }
    }
  }
  if constexpr (MOD) {
    t.key_lo = t.key_begin;
    t.key_begin &= ~15;
  }
  return t;
}

// row i -> (query index, head, part index for decode, causal limit)
template <bool DECODE, bool MOD = false>
__device__ __forceinline__ void row_info(const TcArgs& a, const TileDesc& t, int kvh, int i,
                                         int64_t& qi, int& head, int64_t& part, int& lim) {
  const int G = a.group;
  if constexpr (DECODE) {
    const int unit = over_group<MOD>(a, i);
    qi = a.members[t.member_off + unit];
    head = kvh * G + (i - unit * G);
    part = int64_t(t.part_base) + unit;
    lim = t.key_end;
  } else {
    const int gr = t.gr0 + i;
    const int tok = over_group<MOD>(a, gr);
    qi = int64_t(t.q_base) + tok;
    head = kvh * G + (gr - tok * G);
    part = 0;
    lim = t.prefix + tok + 1;
  }
}

// 128-byte-swizzled tile of `rows` rows, stored as column blocks of 64 bf16:
// byte address of 16-byte chunk `ch` (of the full row) of row r.
__device__ __forceinline__ uint32_t sw128(uint32_t base, int rows, int r, int ch) {
  return base + uint32_t((ch >> 3) * rows * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

// D(tmem) (+)= A * B(smem), A from shared memory (ss) or TMEM (ts), issued
// by a single thread, with the shared-memory descriptors passed as 32-bit
// halves: the high half (stride between 8-row groups, version, swizzle) is
// common to every operand of the tile, and the low half (start address >> 4
// and leading-byte offset) moves by compile-time steps, so the issuing thread
// spends one add per operand instead of rebuilding 64-bit descriptors.
__device__ __forceinline__ void mma_ss_split(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                             uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 ad, bd;\n setp.ne.b32 p, %5, 0;\n"
      " mov.b64 ad, {%1, %3};\n mov.b64 bd, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %4, p;\n}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts_split(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                             uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 bd;\n setp.ne.b32 p, %5, 0;\n"
      " mov.b64 bd, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %4, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 16 columns of 32-bit values from registers (thread t: lane t).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// What a row adds to its scores (rx_score_mod, in log2 units), and the first
// key that it sees.
struct RowMod {
  int lo = 0;
  float slope = 0.f;  // slope of the row's head times log2(e)
  int pos = 0;        // the query's position
};

// of the query at index qi and position pos
__device__ __forceinline__ RowMod row_mod(const TcArgs& a, int64_t qi, int head, int pos) {
  RowMod r;
  if (a.window > 0) r.lo = max(0, pos - a.window + 1);
  if (a.key_begin) r.lo = max(r.lo, __ldg(a.key_begin + qi));
  if (a.slopes) r.slope = __ldg(a.slopes + head) * kLog2e;
  r.pos = pos;
  return r;
}

// tanh(u) / u for |u| <= 1 as a polynomial in u^2 of degree 6, the nearest to it
// there by relative error (Remez exchange): 5e-8 in exact arithmetic, 1.6e-7
// in fp32.
constexpr int kTanhTerms = 7;
constexpr float kTanh[kTanhTerms] = {0.99999994f, -0.3333284f,   0.13325204f,  -0.05345703f,
                                     0.02028998f, -0.006203379f, 0.0010410226f};
// The same for |u| <= 0.6, of degree 4: 7e-8, 1.8e-7 in fp32.
constexpr int kTanhNearTerms = 5;
constexpr float kTanhNear[kTanhNearTerms] = {0.99999994f, -0.3333231f, 0.13310173f, -0.05210148f,
                                             0.015475428f};
// tanh(u) = 1 - 2 / (1 + e^2u), off by some 2^-22 at most: for |u| above 0.6, where that is
// less than 2^-20 of it
__device__ __forceinline__ float tanh_exp(float u) {
  return fmaf(-2.f, __fdividef(1.f, 1.f + rxk::fast_exp2(u * (2.f * kLog2e))), 1.f);
}
// softcap * tanh(scale * s / softcap) * log2(e) of a lane's scores: all by the polynomial
// first (branches for each one would put their chains one behind the other), and where some
// score of the warp lies beyond its range, those that do by the exponential.
template <int N>
__device__ __forceinline__ void cap_all(const TcArgs& a, float (&x)[N][4]) {
  float u[4 * N], v[4 * N], p[4 * N];
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) {
    u[i] = x[i >> 2][i & 3] * a.cap_in;
    most = fmaxf(most, fabsf(u[i]));
    v[i] = u[i] * u[i];
    p[i] = a.cap_poly[kTanhTerms - 1];
  }
#pragma unroll
  for (int d = kTanhTerms - 2; d >= 0; --d)
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) p[i] = fmaf(p[i], v[i], a.cap_poly[d]);
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) x[i >> 2][i & 3] = u[i] * p[i];
  if (!__all_sync(0xffffffffu, most <= 1.f)) {
#pragma unroll
    for (int i = 0; i < 4 * N; ++i)
      if (!(fabsf(u[i]) <= 1.f)) x[i >> 2][i & 3] = a.cap_out * tanh_exp(u[i]);
  }
}

// ---------------------------------------------------------------------------
// Warp role of the fused decode kernel: work items of <= 16 query rows at
// head_dim 128, <= 8 at 256 (a request's private tail, or a shared segment
// chunk with few rows).  One warp owns one (item, KV head) unit and streams its keys
// in steps of 16.  With few query rows per item the products are computed transposed,
// keys in the M dimension of mma.sync m16n8k16 and query rows in N (8 or 16
// rows, NR n-tiles), so no MMA row is wasted on keys:
//   S^T (16 keys x 8 rows)  = K (16 x D, ldmatrix)        . Q^T (registers)
//   O^T (D x 8 rows)       += V^T (16 d x 16 keys per m-tile, ldmatrix.trans)
//                             . P^T (the S^T accumulators, bf16, moved into
//                               operand layout with four shuffles)
// A thread of the S^T accumulators holds keys g, g+8 of rows 2c, 2c+1 (g =
// lane/4, c = lane%4): the running max and sum of a row live in the 8 lanes
// that share c.  K and V rows of a step are gathered by slot with 16-byte
// cp.async into a ring of PipeCfg<D>::STAGES stages (one fewer steps in
// flight) whose rows are padded by 16 B, so ldmatrix reads all 32 banks.
// The max is rescaled lazily: O and the sum are rescaled only when a row's
// max grows by more than 2^8.
constexpr int kPipeWarps = 6;                    // warps of a CTA in the warp role
constexpr int kSlotBuf = 128;                    // key slots per slot block (x 16 B aligned)
constexpr int kSlotRegs = kSlotBuf / 32;         // slots of a block per lane
template <int D>
struct PipeCfg {
  static constexpr int STAGES = D == 128 ? 4 : 2;     // ring stages per warp
  static constexpr int PITCH = 2 * D + 16;            // shared bytes per K/V row
  static constexpr int STAGE_BYTES = 32 * PITCH;      // 16 K rows, then 16 V rows
  // the ring, then two slot blocks (the one in use and the next)
  static constexpr int WARP_BYTES = STAGES * STAGE_BYTES + 2 * kSlotBuf * 4;
};

// A warp's next warp-role unit, fetched in stages while the current one
// streams, so that the counter, work-item and slot-table round trips are off
// the path: stage 1 takes an index from the counter (lane 0), stage 2 loads
// the item's work words (lane k < 8 holds word k), stage 3 its first block
// of key slots (lane l holds keys l + 32 i).  idx >= n_small_units: none left.
struct NextUnit {
  int idx;  // lane 0 only until stage 2
  int32_t wk;
  int32_t s[kSlotRegs];
  int stage;
  __device__ __forceinline__ int32_t word(int k) const { return __shfl_sync(0xffffffffu, wk, k); }
};

template <bool BACK = false, bool MOD = false>
__device__ __forceinline__ void next_unit_step(const TcArgs& a, NextUnit& n) {
  const int lane = threadIdx.x & 31;
  if (n.stage == 0) {
    n.idx = lane == 0 ? atomicAdd(a.unit_counter, 1) : 0;
  } else if (n.stage == 1) {
    n.idx = __shfl_sync(0xffffffffu, n.idx, 0);
    n.wk = 0;
    if (n.idx < a.n_small_units && lane < RX_WORK_WORDS)
      n.wk = __ldg(a.work_small + int64_t(over_hkv<MOD>(a, n.idx)) * RX_WORK_WORDS + lane);
  } else if (n.stage == 2) {
    const int32_t row = n.word(0), kb = n.word(1), kend = n.word(2), grow = n.word(7);
    if (n.idx < a.n_small_units) {
      const int32_t* trow = a.table + int64_t(row) * a.row_stride;
      const int ke = grow > 0 ? min(kend, grow + a.step) : kend;
#pragma unroll
      for (int i = 0; i < kSlotRegs; ++i) {
        const int at = lane + 32 * i;
        n.s[i] = at < ke - kb ? __ldg(trow + (BACK ? ke - 1 - at : kb + at)) : kNoKey<MOD>;
      }
    }
  }
  if (n.stage < 3) ++n.stage;
}

// MOD, CAP, SLOPES: modified scores (with neither of the last two, masks alone).
template <int NR, int D, bool MOD = false, bool CAP = false, bool SLOPES = false>
__device__ __forceinline__ void pipe_unit(const TcArgs& a, uint32_t ring, int32_t* slot_buf,
                                          uint32_t& gstep, const NextUnit& cur, NextUnit& nxt) {
  using Cfg = PipeCfg<D>;
  constexpr int S = Cfg::STAGES;
  constexpr int kRowPitch = Cfg::PITCH;
  constexpr int kStageBytes = Cfg::STAGE_BYTES;
  constexpr int NK = D / 16;  // k-steps of S^T, m-tiles of O^T
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int n_heads_kv = MOD ? a.hkv : a.hq / a.group;
  const int unit = cur.idx;
  const int kvh = unit - over_hkv<MOD>(a, unit) * n_heads_kv;
  const int G = a.group;
  const int32_t w_row = cur.word(0), w_kend = cur.word(2), w_grow = cur.word(7);
  const int32_t* trow = a.table + int64_t(w_row) * a.row_stride;
  const int kb = cur.word(1), member_off = cur.word(3), part_base = cur.word(5),
            n_rows = cur.word(6);
  // a private tail of a multi-step plan ends at its step-0 end + step
  const int ke = w_grow > 0 ? min(w_kend, w_grow + a.step) : w_kend;
  const bf16* kbase = a.kpool + int64_t(kvh) * a.head_stride;
  const bf16* vbase = a.vpool + int64_t(kvh) * a.head_stride;

  // The unit whose chunk holds this step's newest token (the end of a growing
  // private tail) stores that token's K/V row for its KV head first, so no
  // separate store launch is needed; the bulk copies below then see the row.
  if (a.k_new && w_grow > 0 && ke == w_grow + a.step && kb < ke) {
    const int64_t b = a.members[member_off];
    const int64_t sl = a.slots_new[b];
    if (sl >= 1 && sl < a.num_slots) {
      const int half = lane >> 4, ch = lane & 15;  // lanes 0-15: K, 16-31: V
      const bf16* src = (half ? a.v_new : a.k_new) + (b * n_heads_kv + kvh) * D;
      bf16* dst = const_cast<bf16*>(half ? vbase : kbase) + sl * D;
#pragma unroll
      for (int h = 0; h < D / 128; ++h)
        reinterpret_cast<uint4*>(dst)[ch + 16 * h] =
            __ldg(reinterpret_cast<const uint4*>(src) + ch + 16 * h);
    } else {
      atomicOr(&g_tc_error, 1);
    }
    // only this warp reads the row back (cp.async below): order the lanes'
    // stores before those reads within the CTA
    __threadfence_block();
    __syncwarp();
  }

  const int n_steps = ke > kb ? (ke - kb + 15) >> 4 : 0;
  // Key slots go through two shared blocks of kSlotBuf: block b (keys
  // [kb + 128 b, ..)) sits in half b % 2.  Block 0 comes prefetched with the
  // unit; block b + 1 is loaded into registers when block b is stored, and
  // stored when the first step of block b + 1 is issued, so no table read
  // waits.  kNoKey past the key range; a slot outside the pool is flagged and
  // read as slot 0.
  int32_t blk[kSlotRegs];
  auto store_block = [&](const int32_t (&r)[kSlotRegs], int half) {
#pragma unroll
    for (int i = 0; i < kSlotRegs; ++i) {
      int32_t sl = r[i];
      if ((sl < 0 && sl != kNoKey<MOD>) || sl >= a.num_slots) {
        atomicOr(&g_tc_error, 1);
        sl = 0;
      }
      slot_buf[half * kSlotBuf + lane + 32 * i] = sl;
    }
    __syncwarp();
  };
  auto load_block = [&](int base) {
#pragma unroll
    for (int i = 0; i < kSlotRegs; ++i) {
      const int at = base + lane + 32 * i;
      blk[i] = at < ke - kb ? __ldg(trow + (SLOPES ? ke - 1 - at : kb + at)) : kNoKey<MOD>;
    }
  };
  if (n_steps > 0) {
    store_block(cur.s, 0);
    load_block(kSlotBuf);
  }
  // step st of this unit: 16 K rows and 16 V rows of 2D bytes, gathered by
  // slot with 16-byte cp.async (lane: chunks lane % 16 (+ 16 h) of rows
  // 8 (lane / 16) + i); rows past the key range are zero-filled (P is 0
  // there, and 0 * V must be 0)
  const int r0 = (lane >> 4) * 8;
  const char* ksrc = reinterpret_cast<const char*>(kbase) + (lane & 15) * 16;
  const int64_t v_minus_k = reinterpret_cast<const char*>(vbase) - reinterpret_cast<const char*>(kbase);
  auto issue = [&](int st) {
    const int block = (st * 16) / kSlotBuf;
    if (block > 0 && st * 16 == block * kSlotBuf) {
      store_block(blk, block & 1);
      load_block((block + 1) * kSlotBuf);
    }
    const uint32_t dst = ring + ((gstep + uint32_t(st)) % S) * kStageBytes +
                         uint32_t(r0 * kRowPitch + (lane & 15) * 16);
    const int4* sp = reinterpret_cast<const int4*>(
        slot_buf + ((block & 1) * kSlotBuf + st * 16 - block * kSlotBuf + r0));
    const int4 s0 = sp[0], s1 = sp[1];
    const int32_t sl[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool ok = sl[i] >= 0;
      const char* src = ksrc + int64_t(ok ? sl[i] : 0) * (D * 2);
#pragma unroll
      for (int h = 0; h < D / 128; ++h) {
        rxk::cp_async_16(dst + uint32_t(i * kRowPitch + 256 * h), src + 256 * h, ok);
        rxk::cp_async_16(dst + uint32_t((16 + i) * kRowPitch + 256 * h), src + 256 * h + v_minus_k,
                         ok);
      }
    }
  };

  float o[NR][NK][4];
#pragma unroll
  for (int nt = 0; nt < NR; ++nt)
#pragma unroll
    for (int mt = 0; mt < NK; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
  // (MOD: l_run is the sum of the weights before their rounding, for lse, and l_bf the sum
  // of those that the product with V takes, for o: the rounding of a weight that is nearly
  // all of a row's then cancels)
  float m_ref[NR][2], l_run[NR][2], l_bf[NR][2];
#pragma unroll
  for (int nt = 0; nt < NR; ++nt) {
    m_ref[nt][0] = m_ref[nt][1] = -INFINITY;
    l_run[nt][0] = l_run[nt][1] = l_bf[nt][0] = l_bf[nt][1] = 0.f;
  }

#pragma unroll 1
  for (int p = 0; p < S - 1; ++p) {
    if (p < n_steps) issue(p);
    rxk::cp_async_commit();
  }

  // Q^T operand, loaded while the first steps' keys are in flight: n-tile nt,
  // k-step kk: (d 16kk + 2c, +1 | 16kk + 2c + 8, +9) of row nt*8 + g
  uint32_t qb[NR][NK][2];
#pragma unroll
  for (int nt = 0; nt < NR; ++nt) {
    const int r = nt * 8 + g;
    const bool ok = r < n_rows;
    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(a.q);
    if (ok) {
      const int u = over_group<MOD>(a, r);
      const int64_t b = a.members[member_off + u];
      qrow = reinterpret_cast<const uint32_t*>(a.q + (b * a.hq + kvh * G + (r - u * G)) * D);
    }
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
      qb[nt][kk][0] = ok ? __ldg(qrow + 8 * kk + c) : 0u;
      qb[nt][kk][1] = ok ? __ldg(qrow + 8 * kk + c + 4) : 0u;
    }
  }

  // MOD: what the scores of rows nt*8 + 2c + e add, and the first key they see
  RowMod rm[NR][2];
  if constexpr (MOD) {
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * c + e;
        if (r < n_rows) {
          const int u = over_group<MOD>(a, r);
          const int64_t b = a.members[member_off + u];
          const int pos = a.ctx_len ? __ldg(a.ctx_len + b) + a.step - 1 : 0;
          rm[nt][e] = row_mod(a, b, kvh * G + (r - u * G), pos);
        }
      }
  }

  // ldmatrix lane addresses: K (A of S^T, keys x d) and V^T (A of O^T, d x keys)
  const uint32_t k_lane = uint32_t(((lane & 7) + ((lane >> 3) & 1) * 8) * kRowPitch + (lane >> 4) * 16);
  const uint32_t v_lane =
      uint32_t((16 + (lane & 7) + (lane >> 4) * 8) * kRowPitch + ((lane >> 3) & 1) * 16);

  // Two steps at a time where the ring has the stages and rows the registers: a step's
  // products, modification and exponentials are chains of some 1,200 cycles that hardly
  // fill a warp's issue slots, two together take little more than one.
  constexpr bool TWO = MOD && NR == 1 && S >= 4;
  if constexpr (TWO) {
#pragma unroll 1
    for (int st = 0; st < n_steps; st += 2) {
      if (st <= 4) next_unit_step<SLOPES, MOD>(a, nxt);
      // (its stage was read in the last round)
      if (st + S - 1 < n_steps) issue(st + S - 1);
      rxk::cp_async_commit();
      rxk::cp_async_wait<S - 2>();
      __syncwarp();
      const bool two = st + 1 < n_steps;
      uint32_t stage[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
        stage[u] = ring + ((gstep + uint32_t(st + u)) % S) * kStageBytes;
      float sacc[2][4], sodd[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) sacc[u][e] = sodd[u][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < NK; ++kk)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t a0, a1, a2, a3;
          rxk::ldsm_x4(stage[u] + k_lane + uint32_t(kk * 32), a0, a1, a2, a3);
          rxk::mma_bf16((kk & 1) ? sodd[u] : sacc[u], a0, a1, a2, a3, qb[0][kk][0], qb[0][kk][1]);
        }
      float x[2][4];
      bool grow = false;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e)  // (what an absent step's stage holds decides nothing)
          x[u][e] = u == 0 || two ? sacc[u][e] + sodd[u][e] : 0.f;
      if constexpr (CAP)
        cap_all(a, x);
      else
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[u][e] *= a.scale_log2;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int key0 = SLOPES ? ke - 1 - ((st + u) * 16 + g) : kb + (st + u) * 16 + g;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = SLOPES ? key0 - 8 * (e >> 1) : key0 + 8 * (e >> 1);
          const RowMod& r = rm[0][e & 1];
          float y = x[u][e];
          if constexpr (SLOPES) y = fmaf(-r.slope, fabsf(float(key - r.pos)), y);
          x[u][e] = key >= max(kb, r.lo) && key < ke ? y : -INFINITY;
          grow |= x[u][e] > m_ref[0][e & 1] + kRescaleThreshold;
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(fmaxf(x[0][e], x[0][2 + e]), fmaxf(x[1][e], x[1][2 + e]));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          if (mx > m_ref[0][e]) {
            const float alpha = rxk::fast_exp2(m_ref[0][e] - mx);  // 0 from -inf
            m_ref[0][e] = mx;
            l_run[0][e] *= alpha;
            l_bf[0][e] *= alpha;
#pragma unroll
            for (int mt = 0; mt < NK; ++mt) {
              o[0][mt][e] *= alpha;
              o[0][mt][2 + e] *= alpha;
            }
          }
        }
      }
      uint32_t pb[2][2];
      const int src1 = 8 * c + (g >> 1), src2 = src1 + 4;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t pk[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m_use = m_ref[0][e] == -INFINITY ? 0.f : m_ref[0][e];
          const float p0 = rxk::fast_exp2(x[u][e] - m_use);
          const float p1 = rxk::fast_exp2(x[u][2 + e] - m_use);
          pk[e] = rxk::pack_bf16(p0, p1);
          l_run[0][e] += p0 + p1;
          l_bf[0][e] += __uint_as_float(pk[e] << 16) + __uint_as_float(pk[e] & 0xffff0000u);
        }
        const uint32_t v0 = __shfl_sync(0xffffffffu, pk[0], src1);
        const uint32_t v1 = __shfl_sync(0xffffffffu, pk[1], src1);
        const uint32_t w0 = __shfl_sync(0xffffffffu, pk[0], src2);
        const uint32_t w1 = __shfl_sync(0xffffffffu, pk[1], src2);
        const uint32_t s1 = (g & 1) ? v1 : v0, s2 = (g & 1) ? w1 : w0;
        pb[u][0] = __byte_perm(s1, s2, 0x5410);
        pb[u][1] = __byte_perm(s1, s2, 0x7632);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (u == 1 && !two) break;  // (nothing was loaded there)
#pragma unroll
        for (int mt = 0; mt < NK; ++mt) {
          uint32_t a0, a1, a2, a3;
          rxk::ldsm_x4_t(stage[u] + v_lane + uint32_t(mt * 32), a0, a1, a2, a3);
          rxk::mma_bf16(o[0][mt], a0, a1, a2, a3, pb[u][0], pb[u][1]);
        }
      }
      __syncwarp();  // every lane is done with these stages before they are refilled
      if (st + S < n_steps) issue(st + S);
      rxk::cp_async_commit();
    }
  } else {
#pragma unroll 1
  for (int st = 0; st < n_steps; ++st) {
    // the next unit: index at step 0, work words at step 2, slots at step 4
    if (st == 0 || st == 2 || st == 4) next_unit_step<SLOPES, MOD>(a, nxt);
    rxk::cp_async_wait<S - 2>();
    __syncwarp();
    const uint32_t stage = ring + ((gstep + uint32_t(st)) % S) * kStageBytes;
    // S^T = K . Q^T, even and odd k-steps in two accumulator chains
    float sacc[NR][4], sodd[NR][4];
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sacc[nt][e] = sodd[nt][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
      uint32_t a0, a1, a2, a3;
      rxk::ldsm_x4(stage + k_lane + uint32_t(kk * 32), a0, a1, a2, a3);
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
        rxk::mma_bf16((kk & 1) ? sodd[nt] : sacc[nt], a0, a1, a2, a3, qb[nt][kk][0], qb[nt][kk][1]);
    }
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sacc[nt][e] += sodd[nt][e];
    // online softmax over the keys of this step (rows 2c, 2c+1 of each n-tile).
    // The row reference m_ref changes only when some key of the row exceeds it
    // by more than 2^8: each lane tests its own keys, one vote per step, and
    // only then are the row maxima reduced over the 8 lanes of a row and O and
    // the sums rescaled (rare after the first step of a unit).
    // (with slopes from the newest key back, so that a row's maximum settles at once)
    const int key0 = SLOPES ? ke - 1 - (st * 16 + g) : kb + st * 16 + g;
    const bool in0 = SLOPES ? key0 >= kb : key0 < ke, in1 = SLOPES ? key0 - 8 >= kb : key0 + 8 < ke;
    float x[NR][4];
    bool grow = false;
    if constexpr (CAP) cap_all(a, sacc);
#pragma unroll
    for (int nt = 0; nt < NR; ++nt) {
      if constexpr (MOD) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = SLOPES ? key0 - 8 * (e >> 1) : key0 + 8 * (e >> 1);
          const RowMod& r = rm[nt][e & 1];
          float y = CAP ? sacc[nt][e] : sacc[nt][e] * a.scale_log2;
          if constexpr (SLOPES) y = fmaf(-r.slope, fabsf(float(key - r.pos)), y);
          x[nt][e] = (e >> 1 ? in1 : in0) && key >= r.lo ? y : -INFINITY;
        }
      } else {
      x[nt][0] = in0 ? sacc[nt][0] * a.scale_log2 : -INFINITY;
      x[nt][1] = in0 ? sacc[nt][1] * a.scale_log2 : -INFINITY;
      x[nt][2] = in1 ? sacc[nt][2] * a.scale_log2 : -INFINITY;
      x[nt][3] = in1 ? sacc[nt][3] * a.scale_log2 : -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        grow |= fmaxf(x[nt][e], x[nt][2 + e]) > m_ref[nt][e] + kRescaleThreshold;
    }
    if (__any_sync(0xffffffffu, grow)) {
      float mx[NR][2];
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) mx[nt][e] = fmaxf(x[nt][e], x[nt][2 + e]);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], off));
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (mx[nt][e] > m_ref[nt][e]) {
            const float alpha = rxk::fast_exp2(m_ref[nt][e] - mx[nt][e]);  // 0 from -inf
            m_ref[nt][e] = mx[nt][e];
            l_run[nt][e] *= alpha;
            if constexpr (MOD) l_bf[nt][e] *= alpha;
#pragma unroll
            for (int mt = 0; mt < NK; ++mt) {
              o[nt][mt][e] *= alpha;
              o[nt][mt][2 + e] *= alpha;
            }
          }
        }
    }
    uint32_t pk[NR][2];  // (key g | key g+8) of rows 2c, 2c+1 as bf16x2
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float m_use = m_ref[nt][e] == -INFINITY ? 0.f : m_ref[nt][e];
        if constexpr (MOD) {
          const float p0 = rxk::fast_exp2(x[nt][e] - m_use);
          const float p1 = rxk::fast_exp2(x[nt][2 + e] - m_use);
          pk[nt][e] = rxk::pack_bf16(p0, p1);
          l_run[nt][e] += p0 + p1;
          l_bf[nt][e] +=
              __uint_as_float(pk[nt][e] << 16) + __uint_as_float(pk[nt][e] & 0xffff0000u);
          continue;
        }
        uint32_t h;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n"
            : "=r"(h)
            : "f"(rxk::fast_exp2(x[nt][2 + e] - m_use)), "f"(rxk::fast_exp2(x[nt][e] - m_use)));
        pk[nt][e] = h;  // low half: key g, high half: key g+8
        l_run[nt][e] += __uint_as_float(h << 16) + __uint_as_float(h & 0xffff0000u);
      }
    // P^T operand for n-tile nt: b0 = (P[key 2c][row g], P[key 2c+1][row g]),
    // b1 = keys 2c+8, 2c+9; key k of row r sits in lane 4k + r/2, half r%2
    uint32_t pb[NR][2];
    const int src1 = 8 * c + (g >> 1), src2 = src1 + 4;
#pragma unroll
    for (int nt = 0; nt < NR; ++nt) {
      const uint32_t v0 = __shfl_sync(0xffffffffu, pk[nt][0], src1);
      const uint32_t v1 = __shfl_sync(0xffffffffu, pk[nt][1], src1);
      const uint32_t w0 = __shfl_sync(0xffffffffu, pk[nt][0], src2);
      const uint32_t w1 = __shfl_sync(0xffffffffu, pk[nt][1], src2);
      const uint32_t s1 = (g & 1) ? v1 : v0;
      const uint32_t s2 = (g & 1) ? w1 : w0;
      pb[nt][0] = __byte_perm(s1, s2, 0x5410);
      pb[nt][1] = __byte_perm(s1, s2, 0x7632);
    }
    // O^T += V^T . P^T
#pragma unroll
    for (int mt = 0; mt < NK; ++mt) {
      uint32_t a0, a1, a2, a3;
      rxk::ldsm_x4_t(stage + v_lane + uint32_t(mt * 32), a0, a1, a2, a3);
#pragma unroll
      for (int nt = 0; nt < NR; ++nt) rxk::mma_bf16(o[nt][mt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
    }
    __syncwarp();  // every lane is done with this stage before it is refilled
    if (st + S - 1 < n_steps) issue(st + S - 1);
    rxk::cp_async_commit();
  }
  }
  rxk::cp_async_wait<0>();
  __syncwarp();
  gstep += uint32_t(n_steps);

  // write the partial (o, lse) of rows nt*8 + 2c + e
#pragma unroll
  for (int nt = 0; nt < NR; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_run[nt][e];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      float lo = l;  // what o is divided by
      if constexpr (MOD) {
        lo = l_bf[nt][e];
        lo += __shfl_xor_sync(0xffffffffu, lo, 4);
        lo += __shfl_xor_sync(0xffffffffu, lo, 8);
        lo += __shfl_xor_sync(0xffffffffu, lo, 16);
      }
      const int r = nt * 8 + 2 * c + e;
      if (r >= n_rows) continue;
      const int uu = over_group<MOD>(a, r);
      const int head = kvh * G + (r - uu * G);
      const int64_t part = int64_t(part_base) + uu;
      float* dst = a.ws_o + (part * a.hq + head) * D;
      const float inv = lo > 0.f ? 1.f / lo : 0.f;  // an empty chunk: zero partial, lse -inf
#pragma unroll
      for (int mt = 0; mt < NK; ++mt) {
        dst[16 * mt + g] = o[nt][mt][e] * inv;
        dst[16 * mt + g + 8] = o[nt][mt][2 + e] * inv;
      }
      if (g == 0) a.ws_lse[part * a.hq + head] = l > 0.f ? m_ref[nt][e] * kLn2 + logf(l) : -INFINITY;
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() { return reinterpret_cast<EncodeTiled>(rx_internal::tensor_map_encoder()); }

// Tensor map over a whole pool [L * Hkv * num_slots rows][D] of bf16, box of
// 64 columns x BN rows, 128-byte swizzle (the shared-memory tile layout);
// false if it cannot be encoded or the pool has 2^31 rows or more.
bool make_pool_map(CUtensorMap* m, const void* pool, const rx_pool_desc* d, int BN) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  // TMA row coordinates are 32-bit signed
  if (int64_t(d->num_layers) * d->num_kv_heads * d->num_slots > INT32_MAX) return false;
  const cuuint64_t dims[2] = {cuuint64_t(d->head_dim),
                              cuuint64_t(d->num_layers) * d->num_kv_heads * d->num_slots};
  const cuuint64_t strides[1] = {cuuint64_t(d->head_dim) * 2};
  const cuuint32_t box[2] = {64, cuuint32_t(BN)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor maps of the pools last used on this thread (K and V of one pool
// descriptor): encoding them is host work repeated on every launch otherwise.
struct PoolMaps {
  const void* k = nullptr;
  const void* v = nullptr;
  int64_t num_slots = 0;
  int32_t layers = 0, heads = 0, dim = 0, box_rows = 0;
  CUtensorMap mk, mv;
};

bool pool_maps(const rx_pool_desc* d, int BN, const CUtensorMap** mk, const CUtensorMap** mv) {
  thread_local PoolMaps cache[4];
  thread_local int next = 0;
  for (PoolMaps& c : cache) {
    if (c.k == d->k_pool && c.v == d->v_pool && c.num_slots == d->num_slots &&
        c.layers == d->num_layers && c.heads == d->num_kv_heads && c.dim == d->head_dim &&
        c.box_rows == BN) {
      *mk = &c.mk;
      *mv = &c.mv;
      return true;
    }
  }
  PoolMaps& c = cache[next];
  next = (next + 1) & 3;
  c.k = nullptr;
  if (!make_pool_map(&c.mk, d->k_pool, d, BN) || !make_pool_map(&c.mv, d->v_pool, d, BN))
    return false;
  c.k = d->k_pool;
  c.v = d->v_pool;
  c.num_slots = d->num_slots;
  c.layers = d->num_layers;
  c.heads = d->num_kv_heads;
  c.dim = d->head_dim;
  c.box_rows = BN;
  *mk = &c.mk;
  *mv = &c.mv;
  return true;
}

// A kernel's dynamic shared-memory limit is an attribute of the kernel in
// the current device's context: it is raised once per device (any thread
// may do it first; setting it twice is harmless).
constexpr int kMaxDevices = 64;

template <typename K>
rx_status ensure_smem(std::atomic<bool> (&done)[kMaxDevices], K* kernel, int bytes) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
    return rx_internal::set_error(RX_ERR_CUDA, "no usable current device");
  if (done[dev].load(std::memory_order_acquire)) return RX_OK;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) {
    cudaGetLastError();  // not left for a later launch check to report
    static thread_local char buf[160];
    snprintf(buf, sizeof(buf), "raising a kernel's shared-memory limit: %s",
             cudaGetErrorString(e));
    return rx_internal::set_error(RX_ERR_CUDA, buf);
  }
  done[dev].store(true, std::memory_order_release);
  return RX_OK;
}

}  // namespace
