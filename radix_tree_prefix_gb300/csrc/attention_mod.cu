// Extend and decode attention with modified scores (rx_score_mod): a tanh cap,
// distance slopes, a window, documents, a part that is seen both ways.
//
// Query i scores key j by s = softcap tanh(scale q.k / softcap) - slope |i - j|
// and sees the keys [lo_i, lim_i): lo_i from its window and its document, lim_i =
// i + 1 or the end of the part seen both ways.  What is computed from s is the
// one-pass softmax of attention_tc.cu.
//
// One tile = 128 query rows that read one KV head over one key range, as in
// attention_tc.cu (extend: suffix tokens x heads of a group; decode: members x
// heads of a shared segment).  Modified scores cost the softmax warps several
// times what the plain ones do (a cap alone some seven operations a score), and two
// warpgroups that share a key tile wait for one another at its maximum.  So here
// three warpgroups (two with two CTAs an SM, PAIR) take whole key tiles in turn,
// thread = row, and a CTA walks over row tiles:
//   warps 0..    warpgroup j % NW takes key tile j (64 keys): scores from TMEM 32 at a
//                time, modified, masked, and at once their weights 2^(s - m) (bf16)
//                into TMEM over scores read already, under the reference m that the
//                warpgroup used last.  At the tile's end the reference of tile j - 1
//                comes from the warpgroup before through shared memory (barrier H):
//                if it is larger, this tile's weights are brought down to it, if it
//                is smaller, O (in TMEM) to m, and m goes on to tile j + 1.  Both are
//                rare: m is an integer, 0 unless a row's scores lie beyond 2^+-64,
//                and a score may exceed it by 64, so that nothing but such a row ever
//                stops for another tile.  (Under a cap of at most 52 m is one number, and
//                nothing is handed on, unless a row sees 16 keys or fewer: such a row's m
//                is its first maximum.)  Each warpgroup keeps the row sums of its own
//                tiles; they meet in the row tile's end;
//   then warp S  Q rows, and S_j = Q K_j^T into a ring of TMEM buffers;
//   K, V         loaders, the K loader also finding row tiles and their key ranges for
//                all the others.  Runs of 64 slots are one TMA box per 64 columns, runs
//                of 16 (pages of 16 slots and more) smaller ones, and the groups left
//                are gathered by 16-byte cp.async, whose completion is waited for only
//                when the next tile's loads are out;
//   PV           O += P_j V_j.
// Rows of a tile see different keys: the key range is what some row sees, and
// masks are applied only to keys that some row of the warp does not see.  A masked
// score is -inf; a row that has seen no key yet has m = -inf and weighs its masked
// keys 0, and one that never sees any gets o = 0, lse = -inf.
//
// What bounds it is the softmax warps' instructions, and fetching them: a tile takes
// some 400 of a warp without a cap and 600 with one, at a little more than half an
// issue slot a clock.  The loops are rolled, and the softmax role stands first in the
// kernel (behind the other roles agent calls under a cap took 506 us, so 458).  At
// head_dim 256 it is shared memory's bandwidth and V's ring of two tiles.  One GB300,
// 40 calls of 200 queries over 3,000 common keys, 32 / 8 heads of 128: 329 us without
// modification (1,245 TFLOP/s), 343 with slopes, 436 under a cap; 64 chat turns of 200
// queries over 2,000 to 3,800 keys, 16 / 4 heads of 256, pages of 16, slopes: 566 us
// (1,083 TFLOP/s).

#include "attention_tile.cuh"

namespace {

constexpr int kGroup = 16;  // keys of a small TMA box
// A weight exceeds its reference by 2^kRaise at most.  fp32 (and bf16, of the same
// range) then has room for sums of 2^20 keys with values up to 2^40, and a row whose
// scores all lie 64 below a reference of 0 loses nothing of them (down to values of
// 2^-60): what is raised or lowered are rows of extreme scores only.
constexpr float kRaise = 64.f;
constexpr float kMostSum = 18446744073709551616.f;  // 2^kRaise
constexpr int kFew = 16;  // keys of a row that takes a score of its own for a reference
constexpr float kOffUnit = 8388608.f;  // 2^23: of what a weight's rounding adds to its sum
// Kernels by what caps their scores: nothing, a cap of at most kLowCap, a higher one.
constexpr int kNoCap = 0, kCap = 1, kHighCap = 2;
constexpr float kLowCap = 128.f;  // in log2 units
constexpr int kPairWindow = 1024;  // widest window for two CTAs an SM

// Keys are loaded, and S computed, BS at a time (the wider product at head_dim
// 128: one of 64 keys reads Q's 16 columns from shared memory for half the
// work); the softmax and O += P V go by tiles of BN = 64 keys, SUBS to a load.
// Rings of NK and NV stages of K and V, NS of S (TMEM).
constexpr int BN = 64;
// PAIR (head_dim 128): two CTAs an SM, each with half of its TMEM and shared memory
// and 64 keys a load.
template <int D, bool PAIR>
struct Layout4 {
  static constexpr int BS = D == 128 && !PAIR ? 128 : 64;
  static constexpr int SUBS = BS / BN;
  static constexpr int KV_BYTES = BS * D * 2;
  static constexpr int NW = PAIR ? 2 : 3;  // softmax warpgroups
  static constexpr int THREADS = 128 * (NW + 1);
  static constexpr int NK = PAIR ? 2 : 3, NV = D == 128 && !PAIR ? 3 : 2;
  static constexpr int NS = PAIR ? 2 : D == 128 ? 3 : 4;
  static constexpr int NB = NS * SUBS;  // tiles of P
  // Barriers of the reference's way from tile to tile: a warpgroup of three that
  // waits for tile g - 1 did tile g - 3 itself, so a ring of two is enough.
  static constexpr int NH = 2;
  static constexpr int Q = 0;
  static constexpr int K0 = BM * D * 2;
  static constexpr int V0 = K0 + NK * KV_BYTES;
  static constexpr int REF = V0 + NV * KV_BYTES;  // rows' references
  static constexpr int MORE = REF + BM * 4;       // what their sums have more than for lse
  static constexpr int SUM = MORE + BM * 4;       // rows' sums, by the warpgroups' first tiles
  static constexpr int JOIN = V0;  // SPLIT, at the end: rows' references and both their sums
  static constexpr int NEXT = SUM + 3 * BM * 4;   // answer to a request for another row tile
  static constexpr int DESC = NEXT + 16;          // the row tile in hand and the next
  static constexpr int BAR = DESC + 2 * int(sizeof(TileDesc));
  static constexpr int NBAR = 2 * NK + 2 * NV + NS + 2 * NB + 4 * NH + 11;
  static constexpr int MISC = BAR + NBAR * 8;  // TMEM address, abort flag
  static constexpr int BYTES = MISC + 16;
  static constexpr int O_COL = NB * BN;
  static constexpr int TMEM_COLS = PAIR ? 256 : 512;
  static_assert(O_COL + D <= TMEM_COLS, "TMEM budget");
  static_assert(BAR % 8 == 0 && DESC % 8 == 0, "alignment");
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
  static_assert(PAIR || BM * (D + 4) * 4 <= JOIN, "the joined rows' room (join_rows)");
};

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(bytes)
               : "memory");
}

struct Maps4 {
  CUtensorMap k, v;      // boxes of 64 keys x 64 columns
  CUtensorMap k16, v16;  // boxes of 16 keys
  CUtensorMap q;         // boxes of 128 rows: the heads of a group of 128 / group tokens
};

// 32 bytes at a 16-byte boundary, in one store at a 32-byte one.
__device__ __forceinline__ void store_32(void* dst, const uint32_t* r, bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(dst), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(r[0], r[1], r[2], r[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Asks for a CTA of the grid that has not started, to be run by this one in its place
// (16 bytes of answer at dst, 16-byte aligned); not to be asked again after a refusal.
__device__ __forceinline__ void ask_next(uint32_t dst, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];\n" ::"r"(dst),
      "r"(bar)
      : "memory");
}
// Its index, -1: none is left.
__device__ __forceinline__ int next_tile(uint32_t answer) {
  int x;
  asm volatile(
      "{\n .reg .b128 h;\n .reg .pred p;\n ld.shared.b128 h, [%1];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n mov.b32 %0, -1;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n}\n"
      : "=r"(x)
      : "r"(answer)
      : "memory");
  return x;
}

// One lane of the warp, known to the compiler as such.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(p));
  return p != 0;
}

// Waits out of line: what a wait does when its barrier is not ready stands
// elsewhere, so that the roles' loops are short stretches of code.  (They share
// an instruction cache with the softmax, and fetch from it most of the time.)
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return tc::mbar_wait(bar, parity, abort_flag, kWaitLimit);
}
__device__ __forceinline__ bool lane_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return tc::mbar_try_wait(bar, parity) || wait_on(bar, parity, abort_flag);
}
// Barriers between warps: a warp waits as one and arrives once.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_on(bar, parity, abort_flag));
}
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}

// Where a loader stands in its ring of `stages` stages, row tile after row tile.
struct Ring {
  int stage = 0, count = 0;  // the next load's stage, and its number
  uint32_t phase = 1;        // of its wait for an empty stage (none in the first round)
};

// One warp loads the K or V tiles of a row tile into its ring; barriers full
// and empty of stage s at full0 + 8 s and empty0 + 8 s (empty: the products that
// read the stage's last keys completed).  Returns false if a wait gave up.  One piece
// of code for both warps, its loops rolled (with the roles' loops unrolled the kernel
// was 195 KB of code, and its warps, each somewhere else in it, waited for
// instructions most of the time), and runs of slots found by two votes: a loader of
// twice the instructions was what pages of 16 waited for (an agent's calls 519 us
// without modification, now 422; on 64-key runs 339).
template <int D, int BS, bool BACK>
__device__ __forceinline__ bool load_tiles(const TcArgs& a, const TileDesc& t, int n_loads,
                                           const CUtensorMap* tm, const CUtensorMap* tm16,
                                           const bf16* src_base, int row0, uint32_t smem0,
                                           uint32_t full0, uint32_t empty0, int stages,
                                           Ring& ring, volatile int* abort_flag) {
  constexpr int CPR = D / 8, CB = D / 64;
  constexpr int SPL = BS / 32;  // slots a lane: of keys SPL lane + i
  constexpr int LPG = kGroup / SPL, LPW = 64 / SPL;  // lanes of a group, of 64 keys
  constexpr uint32_t GROUPS = LPG == 4 ? 0x11111111u : 0x01010101u;  // their first lanes
  constexpr uint32_t WIDES = LPW == 16 ? 0x00010001u : 1u;           // those of 64 keys
  constexpr int AHEAD = 3;  // loads whose slots are on their way
  const int lane = threadIdx.x & 31;
  int32_t slot[SPL], next[AHEAD][SPL];
  auto load_slots = [&](int j, int32_t (&dst)[SPL]) {
    const int k0 = t.key_begin + (BACK ? n_loads - 1 - j : j) * BS + SPL * lane;
#pragma unroll
    for (int i = 0; i < SPL; ++i)
      dst[i] = j < n_loads && k0 + i >= t.key_lo && k0 + i < t.key_end ? __ldg(t.trow + k0 + i)
                                                                       : kNoKey<true>;
  };
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) load_slots(u, next[u]);
  int before = 0;        // stage of the load before
  bool pending = false;  // whose gathered rows are still on their way
  bool ok = true;
#pragma unroll 1
  for (int j = 0; j < n_loads; ++j) {
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
      slot[i] = next[0][i];
#pragma unroll
      for (int u = 0; u + 1 < AHEAD; ++u) next[u][i] = next[u + 1][i];
      if (slot[i] >= a.num_slots || (slot[i] < 0 && slot[i] != kNoKey<true>)) {
        atomicOr(&g_tc_error, 1);
        slot[i] = 0;
      }
    }
    load_slots(j + AHEAD, next[AHEAD - 1]);
    const uint32_t full = full0 + 8u * uint32_t(ring.stage);
    const uint32_t dst = smem0 + uint32_t(ring.stage * BS * D * 2);
    // Runs of slots, by the bits of their first lanes: of 64 keys (wide), and of 16 in
    // the rest.  A lane's slots are a run, and go on in the next lane's.
    bool run = true;
#pragma unroll
    for (int i = 1; i < SPL; ++i) run = run && slot[i] == slot[0] + i;
    const uint32_t runs = __ballot_sync(0xffffffffu, run && slot[0] >= 0);
    const uint32_t links = __ballot_sync(
        0xffffffffu, __shfl_down_sync(0xffffffffu, slot[0], 1) == slot[0] + SPL);
    uint32_t narrow = runs & (links | (GROUPS << (LPG - 1)));
    narrow &= narrow >> 1;
    narrow &= narrow >> 2;
    if constexpr (LPG == 8) narrow &= narrow >> 4;
    narrow &= GROUPS;
    // (groups that are runs and linked to the next one)
    uint32_t wide = narrow & ((links >> (LPG - 1)) | ((WIDES << (LPW - LPG))));
    wide &= wide >> LPG;
    wide &= wide >> (2 * LPG);
    wide &= WIDES;
    const uint32_t in_wide = wide * (GROUPS & (LPW == 16 ? 0xffffu : 0xffffffffu));
    narrow &= ~in_wide;
    uint32_t left = GROUPS & ~in_wide & ~narrow;
    if (ring.count >= stages &&
        !warp_wait(empty0 + 8u * uint32_t(ring.stage), ring.phase, abort_flag)) {
      ok = false;
      break;
    }
    if (lane == 0)
      mbar_expect_tx(full, uint32_t(__popc(wide) * 64 + __popc(narrow) * kGroup) * (D * 2));
    __syncwarp();
    // a lane a box: columns 64 (lane % CB) of 64 keys, or of a group
    const int n = lane / CB, col = lane % CB;
    if (wide) {
      const int32_t b = __shfl_sync(0xffffffffu, slot[0], (n * LPW) & 31);
      if (n < BS / 64 && (wide >> (n * LPW) & 1u))
        tc::tma_load_2d(dst + uint32_t((col * BS + n * 64) * 128), tm, col * 64, row0 + b, full);
    }
    if (narrow) {
      const int32_t b = __shfl_sync(0xffffffffu, slot[0], (n * LPG) & 31);
      if (n < BS / kGroup && (narrow >> (n * LPG) & 1u))
        tc::tma_load_2d(dst + uint32_t((col * BS + n * kGroup) * 128), tm16, col * 64, row0 + b,
                        full);
    }
    const bool gathered = left != 0;
#pragma unroll 1
    for (; left; left &= left - 1u) {
      const int first = __ffs(left) - 1;  // the group's first lane
      // lanes 0-15 and 16-31 copy chunks (lane % 16) + 16 h of rows k and k + 8
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int32_t sl = __shfl_sync(0xffffffffu, slot[k % SPL],
                                       first + k / SPL + (lane >> 4) * (LPG / 2));
        const bool there = sl >= 0;
        const bf16* src = src_base + int64_t(there ? sl : 0) * D;
        const int row = first * SPL + k + (lane >> 4) * 8;
#pragma unroll
        for (int h = 0; h < CPR / 16; ++h) {
          const int ch = (lane & 15) + 16 * h;
          rxk::cp_async_16(sw128(dst, BS, row, ch), src + ch * 8, there);
        }
      }
    }
    if (gathered)
      rxk::cp_async_commit();
    else if (lane == 0)
      tc::mbar_arrive(full);
    // the gather of the tile before has had this tile's issue to land in
    if (pending) {
      if (gathered)
        rxk::cp_async_wait<1>();
      else
        rxk::cp_async_wait<0>();
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(full0 + 8u * uint32_t(before));
    }
    pending = gathered;
    before = ring.stage;
    ++ring.count;
    if (++ring.stage == stages) {
      ring.stage = 0;
      ring.phase ^= 1u;
    }
  }
  if (pending) {
    rxk::cp_async_wait<0>();
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(full0 + 8u * uint32_t(before));
  }
  return ok;
}

// What the cap multiplies the raw scores sr[at .. at + 15] by, a polynomial in their
// squares.
__device__ __forceinline__ void cap_factors(const TcArgs& a, const uint32_t (&sr)[32], int at,
                                            float2 (&p)[8]) {
  float2 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 x = make_float2(__uint_as_float(sr[at + 2 * k]),
                                 __uint_as_float(sr[at + 2 * k + 1]));
    v[k] = __fmul2_rn(x, x);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    p[k] = __ffma2_rn(a.cap_fold2[kTanhNearTerms - 1], v[k], a.cap_fold2[kTanhNearTerms - 2]);
#pragma unroll
  for (int d = kTanhNearTerms - 3; d >= 0; --d)
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = __ffma2_rn(p[k], v[k], a.cap_fold2[d]);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 2^sr in bf16, and their sum before the rounding; the largest of them and of top into top.
__device__ __forceinline__ float weights_of(const uint32_t (&sr)[32], uint32_t (&pk)[16],
                                            float& top) {
  float2 l4[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) l4[u] = make_float2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float2 p = make_float2(rxk::fast_exp2(__uint_as_float(sr[e])),
                                 rxk::fast_exp2(__uint_as_float(sr[e + 1])));
    l4[(e >> 1) & 3] = __fadd2_rn(l4[(e >> 1) & 3], p);
    pk[e >> 1] = rxk::pack_bf16(p.x, p.y);
    top = max3(top, p.x, p.y);
  }
  const float2 lt = __fadd2_rn(__fadd2_rn(l4[0], l4[1]), __fadd2_rn(l4[2], l4[3]));
  return lt.x + lt.y;
}
// Raw scores capped in place, in log2 units, less m.
__device__ __forceinline__ void cap_scores(const TcArgs& a, uint32_t (&sr)[32], bool near,
                                           float m) {
  if (near) {
    const float2 neg2 = make_float2(-m, -m);
#pragma unroll
    for (int e = 0; e < 32; e += 16) {
      float2 p[8];
      cap_factors(a, sr, e, p);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 y = __ffma2_rn(make_float2(__uint_as_float(sr[e + 2 * k]),
                                                __uint_as_float(sr[e + 2 * k + 1])), p[k], neg2);
        sr[e + 2 * k] = __float_as_uint(y.x);
        sr[e + 2 * k + 1] = __float_as_uint(y.y);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      sr[e] = __float_as_uint(fmaf(a.cap_out, tanh_exp(__uint_as_float(sr[e]) * a.cap_in), -m));
  }
}
// The same score by score: the exponential's error is one of the cap, which the scores of
// other rows and keys must not bear that are far below it.  (Under caps of at most 88 it is
// below 2^-15, nothing beside a weight's rounding, and scores go the one way or the other
// together: a prompt in a window under a cap of 30, whose scores come near it, takes 184 us
// so and 230 score by score.  Kernels of their own, because as a third way in the loop,
// inline or not, it cost calls that never take it 3 %.)
__device__ __forceinline__ void cap_each(const TcArgs& a, uint32_t (&sr)[32], float m) {
#pragma unroll
  for (int e = 0; e < 32; e += 16) {
    float2 p[8];
    cap_factors(a, sr, e, p);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float x = __uint_as_float(sr[e + k]);
      const float far = a.cap_out * tanh_exp(x * a.cap_in);
      const float near = x * (k & 1 ? p[k >> 1].y : p[k >> 1].x);
      sr[e + k] = __float_as_uint((fabsf(x) <= a.cap_near ? near : far) - m);
    }
  }
}
// sr * scale - slope |away + e| - m; behind: no key lies after the row's query, and
// the bias is linear in the key.
__device__ __forceinline__ void add_slopes(uint32_t (&sr)[32], float scale, float slope,
                                           float away, bool behind, float m) {
  if (behind) {
    const float2 scale2 = make_float2(scale, scale);
    float2 in8[4];  // within a group of eight keys
#pragma unroll
    for (int u = 0; u < 4; ++u)
      in8[u] = make_float2(slope * float(2 * u), slope * float(2 * u + 1));
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
      const float b = fmaf(slope, away + float(e), -m);
      const float2 b2 = make_float2(b, b);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 x = make_float2(__uint_as_float(sr[e + 2 * u]),
                                     __uint_as_float(sr[e + 2 * u + 1]));
        const float2 y = __ffma2_rn(x, scale2, __fadd2_rn(b2, in8[u]));
        sr[e + 2 * u] = __float_as_uint(y.x);
        sr[e + 2 * u + 1] = __float_as_uint(y.y);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      sr[e] = __float_as_uint(fmaf(-slope, fabsf(away + float(e)),
                                   fmaf(__uint_as_float(sr[e]), scale, -m)));
  }
}
// sr * scale - m
__device__ __forceinline__ void scale_scores(uint32_t (&sr)[32], float scale, float m) {
  const float2 scale2 = make_float2(scale, scale), neg2 = make_float2(-m, -m);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])),
                                scale2, neg2);
    sr[e] = __float_as_uint(x.x);
    sr[e + 1] = __float_as_uint(x.y);
  }
}
// -inf but for keys [from, to) of the 32, either of which may lie outside them.
__device__ __forceinline__ void mask_scores(uint32_t (&sr)[32], int from, int to) {
  // (a shift by 32 gives 0)
  const uint32_t seen = __funnelshift_lc(0u, ~0u, uint32_t(max(from, 0))) &
                        ~__funnelshift_lc(0u, ~0u, uint32_t(max(to, 0)));
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!(seen >> e & 1u)) sr[e] = 0xff800000u;
}
// 32 lanes x 16 columns of 32-bit values into registers.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// A tile's bf16 weights (32 columns of pairs) times f, a power of two or 0: exact.
__device__ __forceinline__ void scale_weights(uint32_t taddr, float f) {
  tc::tmem_st_wait();  // the warp's own stores
#pragma unroll 1
  for (int c = 0; c < BN / 2; c += 16) {
    uint32_t r[16];
    tmem_ld16(taddr + uint32_t(c), r);
    tc::tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      r[e] = rxk::pack_bf16(__uint_as_float(r[e] << 16) * f,
                            __uint_as_float(r[e] & 0xffff0000u) * f);
    tmem_st16(taddr + uint32_t(c), r);
  }
  tc::tmem_st_wait();
}

// SPLIT: the CTAs of a cluster share one row tile's keys.
__device__ __forceinline__ int cluster_rank() {
  int r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_size() {
  int n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(n));
  return n;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;\n" ::: "memory");
}
// The address of what lies at a shared-memory address of this CTA in CTA `rank`.
__device__ __forceinline__ uint32_t of_rank(uint32_t addr, int rank) {
  uint32_t x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(x) : "r"(addr), "r"(rank));
  return x;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(addr)
               : "memory");
  return x;
}

// The keys of this CTA's share, and in t.member_off how many CTAs have one: shares of
// kLeastShare keys and more, in whole loads.
constexpr int kLeastShare = 512;
__device__ __forceinline__ void cut_keys(TileDesc& t) {
  const int n = cluster_size(), rank = cluster_rank();
  const int keys = max(0, t.key_end - t.key_begin);
  const int share = max(kLeastShare, ((keys + n - 1) / n + 127) & ~127);
  t.member_off = (keys + share - 1) / share;
  const int begin = t.key_begin + rank * share;
  t.key_end = min(t.key_end, begin + share);
  t.key_lo = max(t.key_lo, begin);
  t.key_begin = begin;
}

// The end of a row tile whose keys were shared: every CTA's O, under its rows' references
// m (ref[i]) and sums (ref[BM + i] what O is divided by, ref[2 BM + i] of the weights before
// their rounding), is brought to the common reference and sum and put
// into shared memory, and CTA r adds up and writes the r-th part of the rows.  All
// threads; nothing of the roles is under way.
template <int D>
__device__ __forceinline__ void join_rows(const TcArgs& a, const TileDesc& t, uint8_t* gbase,
                                          const float* ref, uint32_t o_tmem, int threads,
                                          bool mine) {
  if (t.member_off <= 1) return;  // (the same in the whole cluster)
  constexpr int PITCH = D + 4;    // floats a row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = cluster_size(), rank = cluster_rank(), part = BM / n;
  const uint32_t stage = rxk::smem_addr(gbase), refs = rxk::smem_addr(ref);
  const bool m64 = t.n_rows <= 64;
  auto row_of = [&](int i, int64_t& out_row) {
    const int row = m64 ? (((i >> 5) << 4) | (i & 15)) : i;
    if ((m64 && (i & 16)) || row >= t.n_rows) return false;
    int64_t qi = 0, p = 0;
    int head = 0, lim = 0;
    row_info<false, true>(a, t, t.kvh, row, qi, head, p, lim);
    out_row = qi * a.hq + head;
    return true;
  };
  cluster_barrier();
  if (warp < 8) {
    const int i = (warp & 3) * 32 + lane, half = warp >> 2;
    float m = -INFINITY, l = 0.f, lo = 0.f;
    for (int r = 0; r < n; ++r) m = fmaxf(m, ld_cluster(of_rank(refs + 4u * i, r)));
    for (int r = 0; r < n; ++r) {
      const float mr = ld_cluster(of_rank(refs + 4u * i, r));
      if (!(mr > -INFINITY)) continue;
      const float to = rxk::fast_exp2(mr - m);
      lo = fmaf(ld_cluster(of_rank(refs + 4u * (BM + i), r)), to, lo);
      l = fmaf(ld_cluster(of_rank(refs + 4u * (2 * BM + i), r)), to, l);
    }
    const float f = lo == 0.f || ref[i] == -INFINITY ? 0.f : rxk::fast_exp2(ref[i] - m) / lo;
    const uint32_t tl = o_tmem + (uint32_t((warp & 3) * 32) << 16);
#pragma unroll 1
    for (int oc = half * (D / 2); oc < (half + 1) * (D / 2); oc += 16) {
      uint32_t x[16];
      if (mine) {
        tmem_ld16(tl + uint32_t(oc), x);
        tc::tmem_ld_wait();
      }
#pragma unroll
      for (int e = 0; e < 16; ++e)
        x[e] = mine && !(f == 0.f) ? __float_as_uint(__uint_as_float(x[e]) * f) : 0u;
      uint4* dst = reinterpret_cast<uint4*>(gbase + (i * PITCH + oc) * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        dst[e] = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
    }
    int64_t out_row = 0;
    if (half == 0 && i / part == rank && row_of(i, out_row))
      a.lse[out_row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
  }
  cluster_barrier();
  for (int k = tid; k < part * (D / 4); k += threads) {
    const int i = rank * part + k / (D / 4), c = k % (D / 4) * 4;
    int64_t out_row = 0;
    if (!row_of(i, out_row)) continue;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < n; ++r) {
      const float4 y = ld_cluster4(of_rank(stage + uint32_t((i * PITCH + c) * 4), r));
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    if (a.out_bf16)
      *reinterpret_cast<uint2*>(reinterpret_cast<bf16*>(a.out) + out_row * D + c) =
          make_uint2(rxk::pack_bf16(x.x, x.y), rxk::pack_bf16(x.z, x.w));
    else
      *reinterpret_cast<float4*>(a.out + out_row * D + c) = x;
  }
  cluster_barrier();  // (no CTA leaves while its rows are read)
}

// A CTA's row tiles one after another: `first`, and (extend) whatever CTAs of the grid
// have not started when its K loader asks for another, so that tiles of different
// lengths spread over the SMs without a counter (dealt out in turn, agent calls under a
// cap took 434 us, so 425, a prompt of 8,191 395 and 375, documents 97 and 95; row tiles
// of four key tiles, a window of 200, 60 and 64).  The loaders and the issuing warps run
// ahead into the next row tile while the softmax warps finish one and write it.  (One CTA
// a row tile left its SM idle for some 9 us of start and end.)
// CAP, SLOPES: what modifies the scores (with neither, masks alone).  Each is a
// kernel of its own: jumps over the code of what a call does not use cost its
// warps more in instruction fetches than the work.
template <int D, bool PAIR, bool DECODE, int CAP, bool SLOPES, bool SPLIT = false>
__device__ __forceinline__ void row_tiles(const TcArgs& a, const Maps4& maps, uint8_t* gbase,
                                          int first) {
  using Lo = Layout4<D, PAIR>;
  constexpr int NW = Lo::NW, NK = Lo::NK, NV = Lo::NV, NS = Lo::NS, NB = Lo::NB, BS = Lo::BS;
  constexpr int SUBS = Lo::SUBS, NH = Lo::NH;
  constexpr bool DIRECT = CAP == kNoCap && D == 128 && (SLOPES || !PAIR);
  static_assert(NW <= 3, "reference barriers and sums");
  constexpr int SW = 4 * NW;  // softmax warps; behind them S, K, V and PV
  const uint32_t base = rxk::smem_addr(gbase);
  if (base & 1023u) {  // uniform over the CTA: nothing initialised yet
    if (threadIdx.x == 0) atomicOr(&g_tc_error, 4);
    return;
  }
  const uint32_t sQ = base + Lo::Q;
  const uint32_t KF = base + Lo::BAR, KE = KF + 8u * NK, VF = KE + 8u * NK, VE = VF + 8u * NV;
  const uint32_t BAR_S = VE + 8u * NV, BAR_P = BAR_S + 8u * NS;
  // PV of tile g completes phase g / NB of its buffer's barrier: S may overwrite P
  const uint32_t BAR_PF = BAR_P + 8u * NB;
  // the reference of tile g is set for a quadrant's rows: 4 (g % NH) + quadrant
  const uint32_t BAR_H = BAR_PF + 8u * NB;
  const uint32_t BAR_FIN = BAR_H + 32u * NH;   // a row tile's products are done
  const uint32_t BAR_X = BAR_FIN + 8u;    // its warpgroups' sums are written
  const uint32_t BAR_OE = BAR_X + 8u;     // its O has been read
  const uint32_t BAR_QE = BAR_OE + 8u;    // its Q has
  const uint32_t BAR_DF = BAR_QE + 8u;    // descriptors of even and odd row tiles: written,
  const uint32_t BAR_DE = BAR_DF + 16u;   // read
  const uint32_t BAR_END = BAR_DE + 16u;  // every product issued is done
  const uint32_t BAR_QF = BAR_END + 8u;   // a row tile's Q has landed, where a box brings it
  const uint32_t BAR_NEXT = BAR_QF + 8u;  // the answer to a request for another row tile has
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Lo::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + Lo::MISC + 4);
  TileDesc* descs = reinterpret_cast<TileDesc*>(gbase + Lo::DESC);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == SW && lane == 0) {
    for (int s = 0; s < 2 * NK + 2 * NV + NS; ++s) tc::mbar_init(KF + 8u * s, 1);
    for (int b = 0; b < NB; ++b) {
      tc::mbar_init(BAR_P + 8u * b, 4);
      tc::mbar_init(BAR_PF + 8u * b, 1);
    }
    for (int b = 0; b < 4 * NH; ++b) tc::mbar_init(BAR_H + 8u * b, 1);
    tc::mbar_init(BAR_FIN, 1);
    tc::mbar_init(BAR_X, SW);
    tc::mbar_init(BAR_OE, 8);
    tc::mbar_init(BAR_QE, 1);
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(BAR_DF + 8u * b, 1);
      tc::mbar_init(BAR_DE + 8u * b, SW + 3);
    }
    tc::mbar_init(BAR_END, 2);  // one commit per issuing thread
    tc::mbar_init(BAR_QF, 1);
    tc::mbar_init(BAR_NEXT, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == SW) {
    tc::tmem_alloc(rxk::smem_addr(tmem_slot), Lo::TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // the k-th row tile's descriptor, as the K loader wrote it
  auto read_desc = [&](int k, TileDesc& t) -> bool {
    if (!warp_wait(BAR_DF + 8u * uint32_t(k & 1), uint32_t(k >> 1) & 1u, abort_flag)) return false;
    t = descs[k & 1];
    warp_arrive(BAR_DE + 8u * uint32_t(k & 1));
    return true;
  };
  // Loads of BS keys, and tiles of BN among them that hold keys.  With slopes the
  // loads go from the newest keys back: scores fall with distance, so a row's first
  // reference is its last, where the other way round almost every tile would raise it
  // (an agent loop's calls under slopes of 2^(-8 h / 32): 810 us forwards, 344).
  auto loads_of = [](const TileDesc& t) {
    return t.key_lo >= t.key_end ? 0 : (t.key_end - t.key_begin + BS - 1) / BS;
  };
  auto tiles_of = [](const TileDesc& t, int n_loads) {
    return SLOPES || n_loads == 0 ? n_loads * SUBS : (t.key_end - t.key_begin + BN - 1) / BN;
  };

  if (warp < SW) {
    // ------------------------------------------------------------ softmax
    // (fences of the tcgen05 proxy are each lane's, before its warp arrives)
    const int wg = warp >> 2;
    const int i = (warp & 3) * 32 + lane;  // TMEM lane
    const uint32_t tl = tmem + (uint32_t((warp & 3) * 32) << 16);
    float* ref = reinterpret_cast<float*>(gbase + Lo::REF);   // [BM]
    int16_t* more = reinterpret_cast<int16_t*>(gbase + Lo::MORE);  // [BM][2]
    float* sums = reinterpret_cast<float*>(gbase + Lo::SUM);  // [NW][BM]
    float* join = reinterpret_cast<float*>(gbase + Lo::JOIN);  // [3][BM]
    int g0 = 0;    // the row tile's first tile among all of the CTA's
    int used = 0;  // row tiles with keys before it
#pragma unroll 1
    for (int k = 0;; ++k) {
    TileDesc t;
    if (!read_desc(k, t) || t.kvh < 0) break;
    const int n_loads = loads_of(t), n_tiles = tiles_of(t, n_loads);
    // the tile row in lane i: row i, or with M = 64 products (at most 64 rows) row
    // 16 (i / 32) + i % 16 in the first 16 lanes of each quadrant
    const bool m64 = t.n_rows <= 64;
    const int row = m64 ? (((i >> 5) << 4) | (i & 15)) : i;
    const bool valid = (!m64 || (i & 16) == 0) && row < t.n_rows;
    int64_t out_row = 0;  // of the outputs, or of the partial ones
    int lim = t.key_end;
    RowMod rm;
    if (valid) {
      int64_t qi = 0, part = 0;
      int head = 0;
      row_info<DECODE, true>(a, t, t.kvh, row, qi, head, part, lim);
      const int pos = DECODE ? (a.ctx_len ? __ldg(a.ctx_len + qi) + a.step - 1 : 0) : lim - 1;
      if (!DECODE) lim = max(lim, t.bidir);
      rm = row_mod(a, qi, head, pos);
      rm.lo = max(rm.lo, t.key_lo);
      out_row = (DECODE ? part : qi) * a.hq + head;
    } else {
      // a lane without a row: nothing it holds is masked or counts
      rm.lo = t.key_lo;
      rm.pos = INT32_MAX;
    }
    const bool narrow = !DECODE && a.out_bf16;
    if (n_loads == 0) {
      // no row of the tile sees a key (decode: at this step of the plan)
      if (SPLIT && t.member_off > 1) {
        if (wg == 0) join[i] = -INFINITY, join[BM + i] = join[2 * BM + i] = 0.f;
      } else if (valid && wg < 2 && (!SPLIT || cluster_rank() == 0)) {
        const int64_t at = out_row * D + wg * (D / 2);
        uint4* dst = narrow ? reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(a.out) + at)
                            : reinterpret_cast<uint4*>((DECODE ? a.ws_o : a.out) + at);
        const int n = narrow ? D / 16 : D / 8;
#pragma unroll 1
        for (int u = 0; u < n; ++u) dst[u] = make_uint4(0u, 0u, 0u, 0u);
        if (wg == 0) (DECODE ? a.ws_lse : a.lse)[out_row] = -INFINITY;
      }
      continue;
    }
    // what the rows of this warp have in common: keys [lo_max, lim_min) are seen
    // by all of them, and keys up to pos_min lie behind all of them
    const int lo_max = __reduce_max_sync(0xffffffffu, rm.lo);
    const int lim_min = __reduce_min_sync(0xffffffffu, lim);
    const int pos_min = __reduce_min_sync(0xffffffffu, rm.pos);
    // The product with V takes rounded weights, and the rounding of one that is nearly all
    // of its row's sum must not be the output's.  O is therefore divided by a sum in which the
    // heaviest weight of each warpgroup counts as it was rounded (top): that weight's rounding
    // then cancels as it would if all of them did (its share of the rest's is small: with a
    // heaviest weight of 0.05 to 0.4 of the sum the outputs' errors are the same within 2 %),
    // for an instruction in place of three a pair of weights.  (Agent calls under a cap 433 us
    // without it and 442; a sum of all rounded weights takes 33 us more than none, as products
    // of mma.sync with ones 97.)  A row of few keys, where such a sum could double the error of the light
    // ones, takes the first maximum it meets for a reference instead, so that a single key's
    // weight is 1 and its value comes out as it is.  All other references are integers, and
    // what brings weights from one to another a power of two.
    const bool few = valid && lim - rm.lo <= kFew;
    // No score can leave the reach of one reference, and the tiles need not agree on it.
    // (The same for the warps of a quadrant in every warpgroup.)
    const bool bounded =
        CAP == kCap && !SLOPES && a.cap_ref > -INFINITY && !__any_sync(0xffffffffu, few);
    // reference of the row's weights, log2 units
    float m_ref = !valid ? 0.f : bounded ? a.cap_ref : -INFINITY;
    float l = 0.f;            // sum of this warpgroup's weights under it, before their
    float top = 0.f;          // rounding, and the largest of them
    bool easy = false;  // every row has a reference
    bool ok = true;
    int j = (wg + NW - g0 % NW) % NW;
    // tile j's buffer of P, and the phase of the buffer's barriers
    int s = (g0 + j) % NB;
    uint32_t phase = uint32_t((g0 + j) / NB) & 1u;
#pragma unroll 1
    for (; j < n_loads * SUBS; j += NW, s += NW) {
      const int g = g0 + j;
      if (s >= NB) {
        s -= NB;
        phase ^= 1u;
      }
      const uint32_t h_bar = BAR_H + 8u * uint32_t(4 * (g & 1) + (warp & 3));
      const uint32_t h_before = BAR_H + 8u * uint32_t(4 * ((g + 1) & 1) + (warp & 3));
      const uint32_t h_parity = uint32_t((g - 1) >> 1) & 1u;
      if (j >= n_tiles) {
        // the half of the last load without keys; it takes its turn all the same, so
        // that no barrier is arrived at before its last phase is done
        if ((!bounded && !warp_wait(h_before, h_parity, abort_flag)) ||
            (g >= NB && !warp_wait(BAR_PF + 8u * uint32_t(s), phase ^ 1u, abort_flag))) {
          ok = false;
          break;
        }
        warp_arrive(h_bar);
        warp_arrive(BAR_P + 8u * s);
        continue;
      }
      if (!warp_wait(BAR_S + 8u * uint32_t(s / SUBS), phase, abort_flag)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const int k0 = t.key_begin +
                     (SLOPES ? (n_loads - 1 - j / SUBS) * BS + (j % SUBS) * BN : j * BN);
      const bool behind = k0 + BN - 1 <= pos_min;
      const uint32_t p_col = tl + uint32_t(s * BN);
      // ---- scores, 32 at a time: modified, and at once their weights under the
      // reference this warpgroup used last (bf16 into TMEM over scores read already,
      // their sum in fp32 before the rounding: lse is then good to fp32, and o to the
      // roundings of its weights)
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        const bool masked = k0 + c < lo_max || k0 + c + 32 > lim_min;
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        uint32_t sr[32], pk[16];
        float sum = 0.f;
        tc::tmem_ld32(p_col + uint32_t(c), sr);
        tc::tmem_ld_wait();
        // DIRECT: where every key is seen and every row has its reference, weights at
        // once.  One beyond the reference's reach shows in their sum; then the scores,
        // still in TMEM, are taken again step by step.  (At head_dim 128 agent calls with
        // slopes take 344 us so and 361 without, unmodified ones 330 and 338, a prompt with
        // slopes in a window of 1,024 144 and 155.  Under a cap, whose range has to be
        // looked at before, 472 and 459; at head_dim 256 slopes 564 and 557; two CTAs an
        // SM without slopes, documents, 98.6 and 97.4.)
        bool done = false;
        if constexpr (DIRECT) {
          if (easy && !masked && (!SLOPES || behind)) {
            if constexpr (SLOPES)
              add_slopes(sr, a.scale_log2, rm.slope, float(k0 + c - rm.pos), true, m_use);
            else
              scale_scores(sr, a.scale_log2, m_use);
            float t = top;
            sum = weights_of(sr, pk, t);
            done = __all_sync(0xffffffffu, !valid || sum <= kMostSum);
            if (done) {
              top = t;
            } else {
              tc::tmem_ld32(p_col + uint32_t(c), sr);
              tc::tmem_ld_wait();
            }
          }
        }
        if (!done) {
          if constexpr (CAP != kNoCap) {
            float am[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 32; e += 8)
#pragma unroll
              for (int u = 0; u < 4; ++u)
                am[u] = fmaxf(am[u], fmaxf(fabsf(__uint_as_float(sr[e + 2 * u])),
                                           fabsf(__uint_as_float(sr[e + 2 * u + 1]))));
            const float most = fmaxf(fmaxf(am[0], am[1]), fmaxf(am[2], am[3]));
            const bool near = __all_sync(0xffffffffu, !valid || most <= a.cap_near);
            if (CAP == kHighCap && !near)
              cap_each(a, sr, SLOPES ? 0.f : m_use);
            else
              cap_scores(a, sr, CAP == kHighCap || near, SLOPES ? 0.f : m_use);
          }
          if constexpr (SLOPES)
            add_slopes(sr, CAP ? 1.f : a.scale_log2, rm.slope, float(k0 + c - rm.pos), behind,
                       m_use);
          else if constexpr (CAP == kNoCap)
            scale_scores(sr, a.scale_log2, m_use);
          if (masked) mask_scores(sr, rm.lo - (k0 + c), lim - (k0 + c));
          if (!bounded) {
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; e += 8)
#pragma unroll
              for (int u = 0; u < 4; ++u)
                mx4[u] = fmaxf(mx4[u], fmaxf(__uint_as_float(sr[e + 2 * u]),
                                             __uint_as_float(sr[e + 2 * u + 1])));
            const float mx = valid ? fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) : 0.f;
            const bool unset = m_ref == -INFINITY;
            const bool grow = mx > (unset ? -INFINITY : kRaise);
            if (__any_sync(0xffffffffu, grow)) {
              // a row without a reference takes 0 if its scores are about that (tiles of other
              // warpgroups that meet the row first then agree)
              float by = 0.f;
              if (grow && !(unset && !few && fabsf(mx) <= kRaise))
                by = unset && few ? mx : rintf(mx);
              if (grow) m_ref = m_use + by;
              const float f = unset ? 1.f : rxk::fast_exp2(-by);  // (unset: no weights yet)
              l *= f;
              top *= f;
              if (c > 0 && __any_sync(0xffffffffu, f != 1.f)) scale_weights(p_col, f);
              if (__any_sync(0xffffffffu, by != 0.f)) scale_scores(sr, 1.f, by);
            }
          }
          sum = weights_of(sr, pk, top);
          if constexpr (DIRECT) easy = !__any_sync(0xffffffffu, m_ref == -INFINITY);
        }
        tmem_st16(p_col + uint32_t(c / 2), pk);
        l += sum;
      }
      tc::tmem_st_wait();
      // ---- the row's reference: that of tile g - 1 unless O has to be raised
      if (j > 0 && !bounded) {
        if (!warp_wait(h_before, h_parity, abort_flag)) {
          ok = false;
          break;
        }
        const float m_prev = ref[i];
        if (!__all_sync(0xffffffffu, m_prev == m_ref)) {
          float down = 1.f, up = 1.f;  // what the tile's weights and O are multiplied by
          if (m_prev != -INFINITY) {
            float m = fmaxf(m_prev, m_ref);
            // (few keys: weights go down by a power of two, beyond which O does)
            if (few && m_ref > -INFINITY && m_ref < m_prev)
              m = fmaxf(m_prev, m_ref + ceilf(m_prev - m_ref));
            if (m_ref > -INFINITY) down = rxk::fast_exp2(m_ref - m);
            up = rxk::fast_exp2(m_prev - m);
            l *= down;
            top *= down;
            m_ref = m;
          }
          if (__any_sync(0xffffffffu, down != 1.f)) scale_weights(p_col, down);
          if (__any_sync(0xffffffffu, up != 1.f)) {
            // O is rescaled once PV of tile g - 1 has written it.  (Its barrier cannot be
            // a phase behind: that tile's scores were issued after PV of tile g - 1 - NB
            // completed, and are done.)
            if (!warp_wait(BAR_PF + 8u * uint32_t(s == 0 ? NB - 1 : s - 1),
                           s == 0 ? phase ^ 1u : phase, abort_flag)) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
#pragma unroll 1
            for (int oc = 0; oc < D; oc += 16) {
              uint32_t r[16];
              tmem_ld16(tl + uint32_t(Lo::O_COL + oc), r);
              tc::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * up);
              tmem_st16(tl + uint32_t(Lo::O_COL + oc), r);
            }
            tc::tmem_st_wait();
          }
        }
      }
      // (its reader, this thread of the next tile's warpgroup, waits for barrier H)
      if (!bounded) ref[i] = m_ref;
      warp_arrive(h_bar);  // (always, so that its phases are counted alike)
      tc::tc_fence_before();
      warp_arrive(BAR_P + 8u * s);
    }
    // Once the row tile's products are done, O stands under the last reference; the
    // warpgroups bring there and exchange their sums as O is divided by them, and what these
    // have more than for lse (16 bits, in 2^-23 of a sum: there is no room for second sums).
    // From here on a warpgroup is known by its first tile: summed by warpgroup, a call's last
    // bits would hang on which row tiles the CTA came to take over.
    if (!ok || !warp_wait(BAR_FIN, uint32_t(used) & 1u, abort_flag)) break;
    tc::tc_fence_after();
    const float m_fin = bounded ? m_ref : ref[i];
    const int first = (wg + NW - g0 % NW) % NW;
    const float wide = few ? 0.f : __uint_as_float(rxk::pack_bf16(0.f, top)) - top;
    const int off = min(max(__float2int_rn(__fdividef(wide * kOffUnit, l)), -32768), 32767);
    if (first > 0) more[2 * i + first - 1] = int16_t(off);
    sums[first * BM + i] =
        m_ref == -INFINITY ? 0.f : (l + wide) * rxk::fast_exp2(m_ref - m_fin);
    warp_arrive(BAR_X);
    if (!warp_wait(BAR_X, uint32_t(used) & 1u, abort_flag)) break;
    g0 += n_loads * SUBS;
    ++used;
    if (first < 2) {
      float l_all = 0.f, l_more = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float x = sums[w * BM + i];
        l_all += x;
        if (first == 0)
          l_more = fmaf(x, float(w == 0 ? off : int(more[2 * i + w - 1])), l_more);
      }
      const float l_lse = fmaf(l_more, -1.f / kOffUnit, l_all);
      if constexpr (SPLIT) {
        if (t.member_off > 1) {  // (read by all of the cluster once every role has ended)
          if (first == 0) join[i] = m_fin, join[BM + i] = l_all, join[2 * BM + i] = l_lse;
          continue;
        }
      }
      const float inv = l_all == 0.f ? 0.f : 1.f / l_all;
      // Warpgroup w < 2 writes columns [w D/2, (w+1) D/2) of the rows, 32 bytes (a
      // sector) a thread and store: the rows need no trip through shared memory.
      constexpr int HC = D / 2;
      const int64_t at = out_row * D + first * HC;
      const bool whole = (reinterpret_cast<uintptr_t>(DECODE ? a.ws_o : a.out) & 31) == 0;
#pragma unroll 1
      for (int oc = 0; oc < HC; oc += 16) {
        uint32_t r[16];
        tmem_ld16(tl + uint32_t(Lo::O_COL + first * HC + oc), r);
        tc::tmem_ld_wait();
        if (oc + 16 >= HC) {  // the next row tile's products may overwrite O
          tc::tc_fence_before();
          warp_arrive(BAR_OE);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * inv);
        if (!valid) continue;
        if (narrow) {
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            h[e] = rxk::pack_bf16(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
          store_32(reinterpret_cast<bf16*>(a.out) + at + oc, h, whole);
        } else {
          float* dst = (DECODE ? a.ws_o : a.out) + at + oc;
          store_32(dst, &r[0], whole);
          store_32(dst + 8, &r[8], whole);
        }
      }
      if (valid && first == 0)
        (DECODE ? a.ws_lse : a.lse)[out_row] =
            l_all == 0.f ? -INFINITY : m_fin * kLn2 + logf(l_lse);
    }
    }
  } else if (warp == SW + 1 || warp == SW + 2) {
    // ------------------------------------------------------------- loaders
    const bool v = warp == SW + 2;
    Ring ring;
    int c = first;  // -1: no row tile is left
#pragma unroll 1
    for (int k = 0;; ++k) {
      TileDesc t;
      if (!v) {
        if (c >= 0) {
          int bx = over_hkv<true>(a, c), kvh = c - bx * a.hkv;
          if (!DECODE && !a.heads_interleaved) {
            kvh = c / a.num_tiles;
            bx = c - kvh * a.num_tiles;
          }
          t = describe<DECODE, true>(a, bx);
          t.kvh = kvh;
          if constexpr (SPLIT) cut_keys(t);
        } else {
          t.kvh = -1;
        }
        if (k >= 2 && !warp_wait(BAR_DE + 8u * uint32_t(k & 1), uint32_t((k >> 1) - 1) & 1u,
                                 abort_flag))
          break;
        if (lane == 0) descs[k & 1] = t;
        warp_arrive(BAR_DF + 8u * uint32_t(k & 1));
        if (c < 0) break;
        if (!DECODE && !SPLIT && lane == 0) {
          tc::mbar_arrive_expect_tx(BAR_NEXT, 16);
          ask_next(base + Lo::NEXT, BAR_NEXT);
        }
      } else if (!read_desc(k, t) || t.kvh < 0) {
        break;
      }
      const bool ok = load_tiles<D, BS, SLOPES>(
          a, t, loads_of(t), v ? &maps.v : &maps.k, v ? &maps.v16 : &maps.k16,
          (v ? a.vpool : a.kpool) + int64_t(t.kvh) * a.head_stride,
          int(a.tma_row_base + int64_t(t.kvh) * a.tma_head_rows), base + (v ? Lo::V0 : Lo::K0),
          v ? VF : KF, v ? VE : KE, v ? NV : NK, ring, abort_flag);
      if (!v) {
        c = -1;
        if constexpr (!DECODE && !SPLIT) {
          // (waited for after a failure too: it is written into shared memory)
          int drain_abort = 0;
          if (!tc::mbar_wait(BAR_NEXT, uint32_t(k) & 1u, &drain_abort, kWaitLimit)) {
            *abort_flag = 1;
            break;
          }
          c = next_tile(base + Lo::NEXT);
          tc::fence_proxy_async_smem();
          __syncwarp();
        }
      }
      if (!ok) break;
    }
    // Before the CTA gives up its shared memory the last load of every stage has
    // landed: at once on the normal path; after a wait of another warp gave up, one
    // more bounded wait that does not look at the abort flag.
    if (lane == 0) {
      const int stages = v ? NV : NK;
      int drain_abort = 0;
#pragma unroll 1
      for (int n = max(0, ring.count - stages); n < ring.count; ++n)
        tc::mbar_wait((v ? VF : KF) + 8u * uint32_t(n % stages), uint32_t(n / stages) & 1u,
                      &drain_abort, kWaitLimit);
    }
    __syncwarp();
  } else if (warp == SW) {
    // --------------------------------------------------- Q, and S = Q K^T
    // descriptors as in attention_tc.cu: 128-byte swizzle, 1024 bytes between
    // 8-row groups in the high half
    constexpr uint32_t DHI = (1024u >> 4) | (1u << 14) | (2u << 29);
    constexpr uint32_t KV_STEP = uint32_t(Lo::KV_BYTES) >> 4;
    static_assert(Lo::REF < (1 << 18), "descriptor address field");
    const uint32_t q_lo = ((sQ & 0x3FFFFu) >> 4) | (1u << 16);
    const uint32_t k_lo0 = (((base + Lo::K0) & 0x3FFFFu) >> 4) | (1u << 16);
    int sk = 0, sb = 0, count = 0, used = 0;  // used: row tiles with keys so far
    uint32_t k_phase = 0, b_phase = 1, q_phase = 0;
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      TileDesc t;
      if (!read_desc(k, t) || t.kvh < 0) break;
      const int n_loads = loads_of(t);
      if (n_loads == 0) continue;
      // Q rows into shared memory once the last row tile's products have read theirs: a
      // whole tile by a box per 64 columns, else gathered (zeros past the tile's rows; a
      // lane finds four rows, and the warp copies whole rows, whose pieces lie together)
      if (used > 0 && !warp_wait(BAR_QE, uint32_t(used - 1) & 1u, abort_flag)) break;
      ++used;
      if (!DECODE && a.q_boxes && t.n_rows == BM) {
        if (lane == 0) tc::mbar_arrive_expect_tx(BAR_QF, uint32_t(BM * D * 2));
        __syncwarp();
        if (lane < D / 64)
          tma_load_3d(sQ + uint32_t(lane * BM * 128), &maps.q, lane * 64, t.kvh * a.group,
                      t.q_base + over_group<true>(a, t.gr0), BAR_QF);
        if (!warp_wait(BAR_QF, q_phase, abort_flag)) {
          // (it has landed before the CTA gives up its shared memory)
          int drain_abort = 0;
          tc::mbar_wait(BAR_QF, q_phase, &drain_abort, kWaitLimit);
          break;
        }
        q_phase ^= 1u;
      } else {
        constexpr int CPR = D / 8, RPI = 32 / CPR;  // chunks a row, rows an instruction
#pragma unroll 1
        for (int r0 = 0; r0 < BM; r0 += 32) {
          const bf16* src = nullptr;
          if (r0 + lane < t.n_rows) {
            int64_t qi = 0, part = 0;
            int head = 0, lim = 0;
            row_info<DECODE, true>(a, t, t.kvh, r0 + lane, qi, head, part, lim);
            src = a.q + (qi * a.hq + head) * D;
          }
#pragma unroll
          for (int r = 0; r < 32; r += RPI) {
            const bf16* from = reinterpret_cast<const bf16*>(__shfl_sync(
                0xffffffffu, reinterpret_cast<unsigned long long>(src), r + lane / CPR));
            rxk::cp_async_16(sw128(sQ, BM, r0 + r + lane / CPR, lane % CPR),
                             (from ? from : a.q) + lane % CPR * 8, from != nullptr);
          }
        }
        rxk::cp_async_commit();
        rxk::cp_async_wait<0>();
        tc::fence_proxy_async_smem();
        __syncwarp();
      }
      if (elect_one()) {
        const uint32_t idesc = t.n_rows <= 64 ? tc::idesc_bf16(64, BS, 0)
                                              : tc::idesc_bf16(BM, BS, 0);
#pragma unroll 1
        for (int j = 0; j < n_loads; ++j) {
          // (products complete in order: the last tile of the buffer's P is enough)
          if ((count >= NS &&
               !lane_wait(BAR_PF + 8u * (sb * SUBS + SUBS - 1), b_phase, abort_flag)) ||
              !lane_wait(KF + 8u * sk, k_phase, abort_flag)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t k_lo = k_lo0 + uint32_t(sk) * KV_STEP;
          const uint32_t d_s = tmem + uint32_t(sb * BS);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t a_off = uint32_t(((ks >> 2) * (BM * 128) + (ks & 3) * 32) >> 4);
            const uint32_t b_off = uint32_t(((ks >> 2) * (BS * 128) + (ks & 3) * 32) >> 4);
            mma_ss_split(d_s, q_lo + a_off, k_lo + b_off, DHI, idesc, ks > 0 ? 1u : 0u);
          }
          tc::mma_commit(BAR_S + 8u * sb);
          tc::mma_commit(KE + 8u * sk);
          ++count;
          if (++sk == NK) sk = 0, k_phase ^= 1u;
          if (++sb == NS) sb = 0, b_phase ^= 1u;
        }
        tc::mma_commit(BAR_QE);
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (elect_one()) {
      tc::mma_commit(BAR_END);
      int drain_abort = 0;
      tc::mbar_wait(BAR_END, 0, &drain_abort, kWaitLimit);
    }
    __syncwarp();
  } else if (warp == SW + 3) {
    // ------------------------------------------------------------ O += P V
    constexpr uint32_t DHI = (1024u >> 4) | (1u << 14) | (2u << 29);
    constexpr uint32_t KV_STEP = uint32_t(Lo::KV_BYTES) >> 4;
    const uint32_t v_lo0 = (((base + Lo::V0) & 0x3FFFFu) >> 4) | (uint32_t(BS * 128 / 16) << 16);
    int sv = 0, pb = 0, used = 0;
    uint32_t v_phase = 0, p_phase = 0;
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      TileDesc t;
      if (!read_desc(k, t) || t.kvh < 0) break;
      const int n_loads = loads_of(t), n_tiles = tiles_of(t, n_loads);
      if (n_loads == 0) continue;
      if (elect_one()) {
        const uint32_t idesc = t.n_rows <= 64 ? tc::idesc_bf16(64, D, 1) : tc::idesc_bf16(BM, D, 1);
#pragma unroll 1
        for (int j = 0; ok && j < n_loads * SUBS; ++j) {
          const int sub = j % SUBS;
          ok = lane_wait(BAR_P + 8u * pb, p_phase, abort_flag) &&
               (sub != 0 || lane_wait(VF + 8u * sv, v_phase, abort_flag)) &&
               (j > 0 || used == 0 || lane_wait(BAR_OE, uint32_t(used - 1) & 1u, abort_flag));
          if (!ok) break;
          tc::tc_fence_after();
          if (j < n_tiles) {
            const uint32_t v_lo =
                v_lo0 + uint32_t(sv) * KV_STEP + uint32_t(sub * (BN * 128 / 16));
            const uint32_t p_t = tmem + uint32_t(pb * BN);
#pragma unroll
            for (int ks = 0; ks < BN / 16; ++ks)
              mma_ts_split(tmem + uint32_t(Lo::O_COL), p_t + uint32_t(ks * 8),
                           v_lo + uint32_t(ks * 2048 / 16), DHI, idesc,
                           (j > 0 || ks > 0) ? 1u : 0u);
          }
          tc::mma_commit(BAR_PF + 8u * pb);
          if (sub == SUBS - 1) {
            tc::mma_commit(VE + 8u * sv);
            if (++sv == NV) sv = 0, v_phase ^= 1u;
          }
          if (++pb == NB) pb = 0, p_phase ^= 1u;
        }
        tc::mma_commit(BAR_FIN);
      }
      ++used;
      ok = __all_sync(0xffffffffu, ok);
    }
    if (elect_one()) {
      tc::mma_commit(BAR_END);
      int drain_abort = 0;
      tc::mbar_wait(BAR_END, 0, &drain_abort, kWaitLimit);
    }
    __syncwarp();
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) atomicOr(&g_tc_error, 2);
  if constexpr (SPLIT) {
    tc::tc_fence_after();
    join_rows<D>(a, descs[0], gbase, reinterpret_cast<float*>(gbase + Lo::JOIN),
                 tmem + uint32_t(Lo::O_COL), Lo::THREADS, loads_of(descs[0]) > 0);
    tc::tc_fence_before();
    __syncthreads();
  }
  if (warp == SW) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, Lo::TMEM_COLS);
  }
}

// Extend: a CTA a row tile in the grid, the heaviest first, of which one an SM (PAIR:
// two) runs and takes the others over; heads as in attention_tc.cu.
template <int D, bool PAIR, int CAP, bool SLOPES>
__global__ void __launch_bounds__(Layout4<D, PAIR>::THREADS, PAIR ? 2 : 1)
    extend_mod_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ Maps4 maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  row_tiles<D, PAIR, false, CAP, SLOPES>(a, maps, smem_raw, int(blockIdx.x));
}

// The same for calls of few row tiles over long contexts: a cluster a row tile.
template <int D, int CAP, bool SLOPES>
__global__ void __launch_bounds__(Layout4<D, false>::THREADS, 1)
    extend_mod_split_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ Maps4 maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  row_tiles<D, false, false, CAP, SLOPES, true>(a, maps, smem_raw,
                                                int(blockIdx.x) / cluster_size());
}

// Decode: the plan's large items as tiles, a CTA each, and beside them the units
// of its small ones on whatever SMs are free (two kernels: the softmax of the
// tiles has three warpgroups, and a unit more registers than those leave).
template <int D, int CAP, bool SLOPES>
__global__ void __launch_bounds__(Layout4<D, false>::THREADS, 1)
    decode_mod_tile_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ Maps4 maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  rxk::griddep_launch_dependents();
  row_tiles<D, false, true, CAP, SLOPES>(a, maps, smem_raw, int(blockIdx.x));
}

// A warp a unit (an item and a KV head): unit blockIdx.x + gridDim.x * warp when
// every unit has a warp, else from a counter, heaviest first.  n_tc_ctas > 0: the
// tiles' kernel runs beside this one, which ends only after it, so that the merge
// behind this one finds both done.
template <int D, bool CAP, bool SLOPES>
__global__ void __launch_bounds__(kPipeWarps * 32, 1)
    decode_mod_stream_kernel(const __grid_constant__ TcArgs a) {
  using Cfg = PipeCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  rxk::griddep_launch_dependents();
  const int warp = int(threadIdx.x >> 5);
  const int lane = int(threadIdx.x & 31);
  const uint32_t ring = rxk::smem_addr(smem_raw) + uint32_t(warp * Cfg::WARP_BYTES);
  int32_t* slot_buf = reinterpret_cast<int32_t*>(smem_raw + warp * Cfg::WARP_BYTES +
                                                 Cfg::STAGES * Cfg::STAGE_BYTES);
  uint32_t gstep = 0;
  NextUnit cur, nxt;
  cur.stage = 0;
  if (!a.unit_counter) {
    cur.idx = int(blockIdx.x) + int(gridDim.x) * warp;
    cur.stage = 1;  // (it has its index)
  }
  while (cur.stage < 3) next_unit_step<SLOPES, true>(a, cur);
  while (cur.idx < a.n_small_units) {
    nxt.stage = 0;
    if (!a.unit_counter) {
      nxt.idx = a.n_small_units;
      nxt.stage = 3;
    }
    if (cur.word(6) <= 8) {
      pipe_unit<1, D, true, CAP, SLOPES>(a, ring, slot_buf, gstep, cur, nxt);
    } else if constexpr (D == 128) {
      pipe_unit<2, D, true, CAP, SLOPES>(a, ring, slot_buf, gstep, cur, nxt);
    } else if (lane == 0) {
      atomicOr(&g_tc_error, 1);  // the plan gives head_dim 256 no such item
    }
    while (nxt.stage < 3) next_unit_step<SLOPES, true>(a, nxt);
    cur = nxt;
  }
  if (a.n_tc_ctas > 0) rxk::griddep_wait();
}

bool make_maps(Maps4* m, const rx_pool_desc* pool) {
  const CUtensorMap *k, *v, *k16, *v16;
  if (!pool_maps(pool, 64, &k, &v)) return false;
  m->k = *k;
  m->v = *v;
  if (!pool_maps(pool, kGroup, &k16, &v16)) return false;
  m->k16 = *k16;
  m->v16 = *v16;
  return true;
}

// Boxes over the queries: whole tiles only are read by them, whose tokens all exist, so
// the map need not know how many there are.  Groups that do not divide a tile have none.
bool make_q_map(CUtensorMap* m, const TcArgs& a, int D) {
  if (BM % a.group != 0) return false;
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(a.hq), cuuint64_t(INT32_MAX)};
  const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(a.hq) * D * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(a.group), cuuint32_t(BM / a.group)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16*>(a.q), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

void set_common(TcArgs* a, const rx_pool_desc* pool, int32_t layer, const void* d_q,
                int32_t num_q_heads, const int32_t* table, int64_t row_stride, float scale,
                const rx_score_mod& m) {
  const int D = pool->head_dim;
  const int64_t rows = int64_t(layer) * pool->num_kv_heads * pool->num_slots;
  a->q = static_cast<const bf16*>(d_q);
  a->kpool = static_cast<const bf16*>(pool->k_pool) + rows * D;
  a->vpool = static_cast<const bf16*>(pool->v_pool) + rows * D;
  a->head_stride = pool->num_slots * D;
  a->num_slots = pool->num_slots;
  a->table = table;
  a->row_stride = row_stride;
  a->hq = num_q_heads;
  a->group = num_q_heads / pool->num_kv_heads;
  a->hkv = pool->num_kv_heads;
  a->by_group = make_div(a->group);
  a->by_hkv = make_div(a->hkv);
  a->scale_log2 = scale * kLog2e;
  a->tma_row_base = rows;
  a->tma_head_rows = pool->num_slots;
  a->cap_in = m.softcap > 0.f ? scale / m.softcap : 0.f;
  a->cap_out = m.softcap * kLog2e;
  for (int i = 0; i < kTanhTerms; ++i) a->cap_poly[i] = kTanh[i] * a->cap_out;
  if (m.softcap > 0.f) {
    // kTanhNear with cap_in, a power of it and cap_out folded in.  A coefficient too
    // small for fp32 is left out, and with it the scores for which its term would
    // count (2^-27 of the sum).
    double u = 0.6;  // largest |scale s / softcap|
    for (int i = 0; i < kTanhNearTerms; ++i) {
      const double k = double(a->cap_in);
      const double c = double(kTanhNear[i]) * double(a->cap_out) * pow(k, 2 * i + 1);
      float f = float(c);
      if (fabs(c) < 1e-37) {
        f = 0.f;
        if (i > 0) u = std::min(u, pow(7e-9 / fabs(double(kTanhNear[i])), 0.5 / i));
      }
      if (fabs(c) > 1e37) u = -1.0;  // too large: no score is near
      a->cap_fold2[i] = make_float2(f, f);
    }
    // (no further than a raw score's square is in fp32)
    a->cap_near = float(std::min(u / double(a->cap_in), 1e19));
    // Capped scores lie within +-cap_out: where their weights under one reference stay
    // within 2^-88 and 2^kRaise, that is every row's, and no maximum is taken.
    a->cap_ref = a->cap_out <= 76.f ? fmaxf(0.f, ceilf(a->cap_out) - kRaise) : -INFINITY;
  }
  a->window = m.window;
  a->slopes = m.d_slopes;
  a->key_begin = m.d_key_begin;
  a->bidir_end = m.d_bidir_end;
  a->ctx_len = m.d_ctx_len;
}

template <int D, bool PAIR, int CAP, bool SLOPES>
rx_status launch_extend(TcArgs a, const rx_pool_desc* pool, unsigned ctas, cudaStream_t s) {
  using Lo = Layout4<D, PAIR>;
  static std::atomic<bool> configured[kMaxDevices];
  const rx_status cs = ensure_smem(configured, extend_mod_kernel<D, PAIR, CAP, SLOPES>, Lo::BYTES);
  if (cs != RX_OK) return cs;
  Maps4 maps;
  if (!make_maps(&maps, pool))
    return rx_internal::set_error(RX_ERR_CUDA, "could not encode the pool's TMA tensor maps");
  a.q_boxes = make_q_map(&maps.q, a, D);
  extend_mod_kernel<D, PAIR, CAP, SLOPES><<<ctas, Lo::THREADS, Lo::BYTES, s>>>(a, maps);
  return rx_internal::launch_status("rx_extend_attention_mod");
}

void split_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, unsigned ctas, int n,
                  int threads, int bytes) {
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = unsigned(n);
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
  cfg->gridDim = dim3(ctas * unsigned(n));
  cfg->blockDim = dim3(unsigned(threads));
  cfg->dynamicSmemBytes = size_t(bytes);
}

// CTAs a row tile, 8 at most: as many as have kLeastShare keys each of the longest context
// that the table holds (or the window lets see), and whose clusters all run at once.  (A
// cluster's CTAs, an SM each, lie in one GPC, whose SMs are no multiple of 8, and clusters in
// more than one wave lose to smaller ones: 16 row tiles of 8,000 keys at head_dim 128 take
// 48 us as clusters of 8 and 36 of 4, 38 row tiles 69 of 4 and 64 of 2.)  8 tokens over
// 30,000 keys 48 us and with one CTA 249, two requests of 20 to 40 over 4,000 at head_dim 256
// 27 and 63, 30 over 600, which one CTA has, 15 and 16.  Shares of 256 keys 23 us for the
// second, 17 for the third.
template <int D, int CAP, bool SLOPES>
rx_status split_of(const TcArgs& a, unsigned ctas, int* split) {
  using Lo = Layout4<D, false>;
  constexpr auto* kernel = extend_mod_split_kernel<D, CAP, SLOPES>;
  static std::atomic<bool> configured[kMaxDevices];
  static std::atomic<int> fit[kMaxDevices][4];  // clusters of 2^lg CTAs at once, + 1
  const int64_t keys = a.window > 0 ? std::min<int64_t>(a.row_stride, a.window) : a.row_stride;
  *split = 1;
  if (int64_t(ctas) * 2 > rx_internal::sm_count() || keys < kLeastShare * 2) return RX_OK;
  const rx_status st = ensure_smem(configured, kernel, Lo::BYTES);
  if (st != RX_OK) return st;
  int dev = -1;
  cudaGetDevice(&dev);
  for (int lg = 3; lg >= 1; --lg) {
    if (keys < kLeastShare << lg) continue;
    int n = fit[dev][lg].load(std::memory_order_relaxed);
    if (n == 0) {
      cudaLaunchConfig_t cfg{};
      cudaLaunchAttribute attr[1];
      split_config(&cfg, attr, 1, 1 << lg, Lo::THREADS, Lo::BYTES);
      int c = 0;
      if (cudaOccupancyMaxActiveClusters(&c, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();  // no cluster of this size
        c = 0;
      }
      n = c + 1;
      fit[dev][lg].store(n, std::memory_order_relaxed);
    }
    if (ctas <= unsigned(n - 1)) {
      *split = 1 << lg;
      break;
    }
  }
  return RX_OK;
}

template <int D, int CAP, bool SLOPES>
rx_status launch_extend_split(TcArgs a, const rx_pool_desc* pool, unsigned ctas, int n,
                              cudaStream_t s) {
  using Lo = Layout4<D, false>;
  Maps4 maps;
  if (!make_maps(&maps, pool))
    return rx_internal::set_error(RX_ERR_CUDA, "could not encode the pool's TMA tensor maps");
  a.q_boxes = make_q_map(&maps.q, a, D);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  split_config(&cfg, attr, ctas, n, Lo::THREADS, Lo::BYTES);
  cfg.stream = s;
  cudaLaunchKernelEx(&cfg, extend_mod_split_kernel<D, CAP, SLOPES>, a, maps);
  return rx_internal::launch_status("rx_extend_attention_mod: split");
}

template <int D, int CAP, bool SLOPES>
rx_status launch_extend_mod(const TcArgs& a, const rx_pool_desc* pool, unsigned ctas,
                            cudaStream_t s) {
  int n = 1;
  const rx_status st = split_of<D, CAP, SLOPES>(a, ctas, &n);
  if (st != RX_OK) return st;
  if (n > 1) return launch_extend_split<D, CAP, SLOPES>(a, pool, ctas, n, s);
  // Row tiles of few keys, one after another in a CTA, are bound by the way from one
  // to the next, which a second CTA on the SM fills (agent calls in a window of 128
  // 75 us and 56, of 512 108 and 101, documents of 400 tokens 100 and 97); over longer
  // ranges one CTA with deeper rings is faster (a window of 2,048 251 and 275, of 3,000
  // 324 and 383), and under a cap always (a prompt in a window of 1,024 196 and 205).
  if constexpr (D == 128 && CAP == kNoCap)
    if (a.key_begin || (a.window > 0 && a.window <= kPairWindow))
      return launch_extend<D, true, CAP, SLOPES>(a, pool, ctas, s);
  return launch_extend<D, false, CAP, SLOPES>(a, pool, ctas, s);
}

template <int D, int CAP, bool SLOPES>
rx_status launch_decode_mod(const TcArgs& a, const rx_pool_desc* pool, unsigned ctas,
                            cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.stream = s;
  if (a.n_tc_ctas > 0) {
    static std::atomic<bool> configured[kMaxDevices];
    const rx_status cs = ensure_smem(configured, decode_mod_tile_kernel<D, CAP, SLOPES>,
                                     Layout4<D, false>::BYTES);
    if (cs != RX_OK) return cs;
    Maps4 maps;
    if (!make_maps(&maps, pool))
      return rx_internal::set_error(RX_ERR_CUDA, "could not encode the pool's TMA tensor maps");
    using Lo = Layout4<D, false>;
    decode_mod_tile_kernel<D, CAP, SLOPES>
        <<<unsigned(a.n_tc_ctas), Lo::THREADS, Lo::BYTES, s>>>(a, maps);
    const rx_status st = rx_internal::launch_status("rx_decode_attention_mod: tiles");
    if (st != RX_OK) return st;
  }
  if (ctas > 0) {
    constexpr int bytes = kPipeWarps * PipeCfg<D>::WARP_BYTES;
    static_assert(bytes <= 227 * 1024 && PipeCfg<D>::WARP_BYTES % 16 == 0, "shared memory");
    static std::atomic<bool> configured[kMaxDevices];
    const rx_status cs =
        ensure_smem(configured, decode_mod_stream_kernel<D, CAP != kNoCap, SLOPES>, bytes);
    if (cs != RX_OK) return cs;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPipeWarps * 32);
    cfg.dynamicSmemBytes = bytes;
    cfg.numAttrs = a.n_tc_ctas > 0 ? 1 : 0;
    cudaLaunchKernelEx(&cfg, decode_mod_stream_kernel<D, CAP != kNoCap, SLOPES>, a);
    return rx_internal::launch_status("rx_decode_attention_mod: streams");
  }
  return RX_OK;
}

// By modification: none (masks), slopes; a cap, and slopes; a high cap, and slopes.
using Launch = rx_status (*)(const TcArgs&, const rx_pool_desc*, unsigned, cudaStream_t);
template <int D>
constexpr Launch kExtend[6] = {
    launch_extend_mod<D, kNoCap, false>,   launch_extend_mod<D, kNoCap, true>,
    launch_extend_mod<D, kCap, false>,     launch_extend_mod<D, kCap, true>,
    launch_extend_mod<D, kHighCap, false>, launch_extend_mod<D, kHighCap, true>};
template <int D>
constexpr Launch kDecode[6] = {
    launch_decode_mod<D, kNoCap, false>,   launch_decode_mod<D, kNoCap, true>,
    launch_decode_mod<D, kCap, false>,     launch_decode_mod<D, kCap, true>,
    launch_decode_mod<D, kHighCap, false>, launch_decode_mod<D, kHighCap, true>};

rx_status pick(int D, const rx_score_mod& m, const Launch (&f128)[6], const Launch (&f256)[6],
               const TcArgs& a, const rx_pool_desc* pool, unsigned ctas, cudaStream_t s) {
  const int cap = !(m.softcap > 0.f) ? kNoCap : a.cap_out <= kLowCap ? kCap : kHighCap;
  const int which = 2 * cap + (m.d_slopes ? 1 : 0);
  return (D == 128 ? f128[which] : f256[which])(a, pool, ctas, s);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

namespace rx_internal {

int32_t mod_error_flags(bool clear) {
  int32_t v = 0;
  cudaMemcpyFromSymbol(&v, g_tc_error, sizeof(v));
  if (clear && v) {
    int32_t z = 0;
    cudaMemcpyToSymbol(g_tc_error, &z, sizeof(z));
  }
  return v;
}

}  // namespace rx_internal

// What both attention calls with modified scores check of them.
static rx_status check_mod(const rx_score_mod* mod, float scale, int32_t out_type) {
  constexpr float kLeast = 9.094947e-13f, kMost = 1.0995116e12f;  // 2^-40, 2^40
  if (!(scale >= kLeast && scale <= kMost))
    return rx_internal::set_error(RX_ERR_INVALID, "attention: scale not within 2^-40 and 2^40");
  if (out_type != RX_OUT_F32 && out_type != RX_OUT_BF16)
    return rx_internal::set_error(RX_ERR_INVALID, "attention: unknown out_type");
  if (mod && mod->softcap != 0.f && !(mod->softcap >= kLeast && mod->softcap <= kMost))
    return rx_internal::set_error(RX_ERR_INVALID,
                                  "score mod: softcap neither 0 nor within 2^-40 and 2^40");
  if (mod && mod->window < 0)
    return rx_internal::set_error(RX_ERR_INVALID, "score mod: window < 0");
  return RX_OK;
}

extern "C" rx_status rx_extend_attention_mod(
    const rx_pool_desc* pool, int32_t layer, const void* d_q, int32_t num_q_heads,
    const int32_t* d_req_to_token, int64_t row_stride, const int32_t* d_req_rows,
    const int32_t* d_prefix_len, const int32_t* d_qo_indptr, const int32_t* d_tile_indptr,
    int32_t R, int64_t num_tiles, float scale, const rx_score_mod* mod, void* d_out,
    int32_t out_type, float* d_lse, rx_stream_t stream) {
  rx_status st = rx_internal::check_pool(pool, layer);
  if (st == RX_OK) st = check_mod(mod, scale, out_type);
  if (st != RX_OK) return st;
  if (num_q_heads <= 0 || num_q_heads % pool->num_kv_heads != 0)
    return rx_internal::set_error(RX_ERR_INVALID, "rx_extend_attention_mod: Hq % Hkv != 0");
  if (R < 0 || num_tiles < 0 || num_tiles * pool->num_kv_heads > INT32_MAX)
    return rx_internal::set_error(RX_ERR_INVALID, "rx_extend_attention_mod: bad R or num_tiles");
  if (R == 0 || num_tiles == 0) return RX_OK;
  if (!d_q || !d_req_to_token || !d_req_rows || !d_prefix_len || !d_qo_indptr ||
      !d_tile_indptr || !d_out || !d_lse || !aligned16(d_q) || !aligned16(d_out))
    return rx_internal::set_error(RX_ERR_INVALID, "rx_extend_attention_mod: NULL or misaligned");
  const int D = pool->head_dim;
  const rx_score_mod none{};
  TcArgs a{};
  set_common(&a, pool, layer, d_q, num_q_heads, d_req_to_token, row_stride, scale,
             mod ? *mod : none);
  a.req_rows = d_req_rows;
  a.prefix_len = d_prefix_len;
  a.qo_indptr = d_qo_indptr;
  a.tile_indptr = d_tile_indptr;
  a.num_req = R;
  a.num_tiles = int(num_tiles);
  // heads interleaved as in rx_extend_attention; a window bounds a tile's keys
  const int64_t keys = a.window > 0 ? std::min<int64_t>(row_stride, a.window) : row_stride;
  const int64_t ctas = num_tiles * pool->num_kv_heads;
  a.heads_interleaved =
      ctas <= int64_t(kExtendInterleaveWaves) * rx_internal::sm_count() ||
      keys * pool->num_kv_heads * int64_t(D) * 4 <= kExtendInterleaveKvBytes;
  a.out = static_cast<float*>(d_out);
  a.lse = d_lse;
  a.out_bf16 = out_type == RX_OUT_BF16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return pick(D, mod ? *mod : none, kExtend<128>, kExtend<256>, a, pool, unsigned(ctas), s);
}

extern "C" rx_status rx_decode_attention_mod(
    const rx_pool_desc* pool, int32_t layer, const void* d_q, int32_t num_q_heads,
    const int32_t* d_req_to_token, int64_t row_stride, const int32_t* d_plan,
    const rx_decode_plan_info* info, int32_t B, int32_t step, float scale,
    const rx_score_mod* mod, void* d_out, int32_t out_type, float* d_lse, void* d_workspace,
    size_t workspace_bytes, rx_stream_t stream) {
  rx_status st = rx_internal::check_pool(pool, layer);
  if (st == RX_OK) st = check_mod(mod, scale, out_type);
  if (st != RX_OK) return st;
  auto bad = [](const char* why) { return rx_internal::set_error(RX_ERR_INVALID, why); };
  if (!info || num_q_heads <= 0 || num_q_heads % pool->num_kv_heads != 0 || B < 0 || step < 0)
    return bad("rx_decode_attention_mod: bad argument");
  if (B == 0) return RX_OK;
  if (int64_t(workspace_bytes) < info->workspace_bytes || !d_workspace || !aligned16(d_workspace))
    return bad("rx_decode_attention_mod: workspace missing, small or misaligned");
  if (!d_q || !d_req_to_token || !d_plan || !d_out || !d_lse || !aligned16(d_q) ||
      !aligned16(d_out))
    return bad("rx_decode_attention_mod: NULL or misaligned");
  if (mod && (mod->window > 0 || mod->d_slopes) && !mod->d_ctx_len)
    return bad("rx_decode_attention_mod: a window or slopes need d_ctx_len");
  if (info->window > 0 && (!mod || mod->window == 0 || mod->window > info->window))
    return bad("rx_decode_attention_mod: the plan was made for a smaller window");
  const int64_t n_small = info->n_work - info->n_work_tc;
  if (info->n_work < 0 || n_small < 0 || info->n_work_tc < 0 || info->n_parts < 0 ||
      info->n_work > INT32_MAX / pool->num_kv_heads)
    return bad("rx_decode_attention_mod: bad plan info");
  const int D = pool->head_dim;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t o_bytes = (info->n_parts * num_q_heads * int64_t(D) * 4 + 255) / 256 * 256;
  const int64_t l_bytes = (info->n_parts * num_q_heads * 4 + 255) / 256 * 256;
  char* ws = static_cast<char*>(d_workspace);
  float* ws_o = reinterpret_cast<float*>(ws);
  float* ws_lse = reinterpret_cast<float*>(ws + o_bytes);
  int32_t* counter = reinterpret_cast<int32_t*>(ws + o_bytes + l_bytes);
  const rx_score_mod none{};
  if (info->n_work > 0) {
    TcArgs a{};
    set_common(&a, pool, layer, d_q, num_q_heads, d_req_to_token, row_stride, scale,
               mod ? *mod : none);
    const int64_t hkv = pool->num_kv_heads;
    const int64_t small_units = n_small * hkv, tc_ctas = info->n_work_tc * hkv;
    // as many stream CTAs as SMs, or as units: with no more units than warps every
    // unit has its own, on as many SMs as there are; more are taken from a counter
    const int64_t sms = rx_internal::sm_count();
    const int64_t ctas = std::min(small_units, sms);
    const bool counted = small_units > sms * kPipeWarps || (tc_ctas > 0 && small_units > 0);
    a.work_small = d_plan + info->off_work;
    a.work = a.work_small + n_small * RX_WORK_WORDS;
    a.members = d_plan + info->off_members;
    a.ws_o = ws_o;
    a.ws_lse = ws_lse;
    a.n_small_units = int(small_units);
    a.n_tc_ctas = int(tc_ctas);
    a.step = step;
    if (counted) {
      a.unit_counter = counter;
      if (cudaMemsetAsync(counter, 0, sizeof(int32_t), s) != cudaSuccess)
        return rx_internal::launch_status("rx_decode_attention_mod: counter reset");
    }
    st = pick(D, mod ? *mod : none, kDecode<128>, kDecode<256>, a, pool, unsigned(ctas), s);
    if (st != RX_OK) return st;
  }
  return rx_internal::merge_parts(D, d_plan + info->off_req_part_indptr,
                                  d_plan + info->off_req_parts, ws_o, ws_lse, num_q_heads, B,
                                  d_out, out_type == RX_OUT_BF16, d_lse, info->n_work > 0, s,
                                  "rx_decode_attention_mod: merge");
}

