// Tensor-core tile of attention over the 8-bit KV pool: 128 query rows that
// read one KV head over one key range (tcgen05, TMEM; sm_103a).  Included by
// kv8_attention.cu.
//
// Per key tile of BN keys (128 at head_dim 128, 64 at 256):
//   S = Q K^T      kind::f8f6f4, K's codes as they lie in the pool and Q as a
//                  sum of two e4m3 operands;
//   softmax        x = S ks rs, P = 2^(x - m) vs / vref in f16 into TMEM;
//   O += P V       kind::f16, V's codes converted to f16 in shared memory.
// Q split: a bf16 query has 8 significant bits, an e4m3 number 4.  With the
// row scaled by a power of two to at most 448, hi = e4m3(q) and lo =
// e4m3(q - hi) add up to q exactly down to 2^-10 of the row's largest
// magnitude, and are off by at most 2^-19 of that below.  The two products
// cost what one f16 product does (the e4m3 rate is twice f16's), and K needs
// no conversion and half the shared memory.  Splitting P the same way was
// not taken: a weight below 2^-18 of the row's largest would be lost, and
// long contexts with one dominant key have most of their sum there.  P stays
// f16, so V is converted.
//
// 512 threads:
//   warps 0-7    softmax in two warpgroups that split every key tile's keys;
//                thread (w, i) owns query row i = TMEM lane i;
//   warp 8       issues S; warp 10 issues P V;
//   warp 9       loads K's codes (one TMA box per 128 columns where the tile's
//                slots form a contiguous run, else a cp.async gather) and the
//                tile's scales;
//   warps 12-15  read V's codes into registers a tile ahead, convert them and
//                write them to swizzled shared memory.
// Every mbarrier wait is bounded; on a timeout the CTA sets an error bit,
// drains its tensor-core work and frees TMEM before returning.
#pragma once

#include <cuda.h>

#include "kv8.cuh"
#include "ptx_util.cuh"
#include "tc_util.cuh"

namespace {

constexpr int kTileThreads = 512;
constexpr int BM = 128;
constexpr long long kWaitLimit = 4000000000LL;  // clock cycles (~2 s)

template <int HEAD_DIM>
struct Tile8 {
  static constexpr int D = HEAD_DIM;
  static constexpr int BN = D == 128 ? 128 : 64;
  static constexpr int NB = 3;     // S buffers and K stages
  static constexpr int NV = 2;     // V stages
  static constexpr int SR = 8;     // scale ring
  static constexpr int Q_BYTES = BM * D;  // of each part
  static constexpr int K_BYTES = BN * D;
  static constexpr int V_BYTES = BN * D * 2;
  static constexpr int Q = 0;
  static constexpr int K0 = Q + 2 * Q_BYTES;
  static constexpr int V0 = K0 + NB * K_BYTES;
  static constexpr int XCH = V0 + NV * V_BYTES;    // [2][2 warpgroups][128] floats
  static constexpr int KS = XCH + 2 * 2 * 128 * 4;  // [SR][BN] K scales
  static constexpr int VS = KS + SR * BN * 4;       // [SR][BN] 2^7 vs / vref
  static constexpr int VREF = VS + SR * BN * 4;     // [SR]
  static constexpr int BAR = VREF + SR * 4;
  // q, kfull[NB], vfull[NV], s[NB], p[NB], o[2], pf[NB], xch[2], sum, final, scales[SR]
  static constexpr int NBAR = 1 + NB + NV + NB + NB + 2 + NB + 2 + 1 + 1 + SR;
  static constexpr int MISC = BAR + NBAR * 8;
  static constexpr int BYTES = MISC + 16 + 1024;  // slack to align the swizzled tiles
  static constexpr int O_COL = D == 128 ? NB * BN : 256;
  static_assert(NB * BN <= O_COL && O_COL + D <= 512, "TMEM budget");
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
};

struct TileDesc8 {
  const int32_t* trow;
  int key_begin, key_end, nomask_end, n_rows;
  int gr0, q_base, prefix;
  int member_off, part_base;
};

template <bool DECODE>
__device__ __forceinline__ TileDesc8 describe8(const Args8& a, int tile) {
  TileDesc8 t;
  if constexpr (DECODE) {
    const int32_t* w = a.work + int64_t(a.n_small + tile) * RX_WORK_WORDS;
    t.trow = a.table + int64_t(w[0]) * a.row_stride;
    t.key_begin = w[1];
    t.key_end = w[7] > 0 ? min(w[2], w[7] + a.step) : w[2];
    t.member_off = w[3];
    t.part_base = w[5];
    t.n_rows = w[6];
    t.nomask_end = t.key_end;
    t.gr0 = t.q_base = t.prefix = 0;
  } else {
    // the last request with tile_indptr <= tile, 32 samples a round
    const int ln = int(threadIdx.x & 31);
    int lo = 0, hi = a.num_req;
    while (hi - lo > 32) {
      const int step = (hi - lo + 31) >> 5;
      const int p = lo + ln * step;
      const bool le = p < hi && __ldg(a.tile_indptr + p) <= tile;
      lo += (31 - __clz(__ballot_sync(0xffffffffu, le))) * step;
      hi = min(hi, lo + step);
    }
    const int p = lo + ln;
    const bool le = p < hi && __ldg(a.tile_indptr + p) <= tile;
    lo += 31 - __clz(__ballot_sync(0xffffffffu, le));
    const int G = a.group;
    t.q_base = a.qo_indptr[lo];
    const int s_r = a.qo_indptr[lo + 1] - t.q_base;
    t.prefix = a.prefix_len[lo];
    t.trow = a.table + int64_t(a.req_rows[lo]) * a.row_stride;
    t.gr0 = (tile - a.tile_indptr[lo]) * BM;
    t.n_rows = min(BM, s_r * G - t.gr0);
    t.key_begin = 0;
    t.key_end = t.prefix + (t.gr0 + t.n_rows - 1) / G + 1;
    t.nomask_end = t.prefix + t.gr0 / G + 1;
    t.member_off = t.part_base = 0;
  }
  return t;
}

// row -> query row of (query, head) order, its output entry and causal limit
template <bool DECODE>
__device__ __forceinline__ void row_info8(const Args8& a, const TileDesc8& t, int kvh, int row,
                                          int64_t& q_row, int64_t& out_row, int& lim) {
  const int G = a.group;
  if constexpr (DECODE) {
    const int unit = row / G;
    const int head = kvh * G + (row - unit * G);
    q_row = int64_t(a.members[t.member_off + unit]) * a.hq + head;
    out_row = (int64_t(t.part_base) + unit) * a.hq + head;
    lim = t.key_end;
  } else {
    const int gr = t.gr0 + row;
    const int tok = gr / G;
    q_row = (int64_t(t.q_base) + tok) * a.hq + kvh * G + (gr - tok * G);
    out_row = q_row;
    lim = t.prefix + tok + 1;
  }
}

// Byte address of 16-byte chunk `ch` of row r in a 128-byte-swizzled tile of
// `rows` rows, stored as blocks of 128-byte columns.
__device__ __forceinline__ uint32_t swz(uint32_t base, int rows, int r, int ch) {
  return base + uint32_t((ch >> 3) * rows * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ void st_shared_16(uint32_t at, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// D(tmem) (+)= A B, descriptors as 32-bit halves with a common high half.
__device__ __forceinline__ void mma8_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 ad, bd;\n setp.ne.b32 p, %5, 0;\n"
      " mov.b64 ad, {%1, %3};\n mov.b64 bd, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %4, p;\n}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                         uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 bd;\n setp.ne.b32 p, %5, 0;\n"
      " mov.b64 bd, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %4, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16x(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mul.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " add.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mov.b64 w, {%6, %7};\n fma.rn.f32x2 z, x, y, w;\n mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

template <int D, bool DECODE>
__device__ __forceinline__ void tile8(const Args8& a, const CUtensorMap* tmk, uint8_t* smem_raw,
                                      int tile, int kvh) {
  using Lo = Tile8<D>;
  constexpr int BN = Lo::BN, NB = Lo::NB, NV = Lo::NV, SR = Lo::SR;
  const uint32_t raw = rxk::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base + Lo::Q;
  const uint32_t bar = base + Lo::BAR;
  const uint32_t BAR_Q = bar;
  auto BAR_KF = [&](int s) { return bar + 8u * (1 + s); };
  auto BAR_VF = [&](int s) { return bar + 8u * (1 + NB + s); };
  auto BAR_S = [&](int b) { return bar + 8u * (1 + NB + NV + b); };
  auto BAR_P = [&](int b) { return bar + 8u * (1 + 2 * NB + NV + b); };
  constexpr uint32_t kAfterP = 1 + 3 * NB + NV;
  // PV_j completes phase j / 2 of BAR_O(j % 2) and phase j / NB of BAR_PF(j %
  // NB).  S_j is issued after PV_{j-NB} completed, so once S_j is complete,
  // PV_{j-3} is, and a wait for PV_{j-1} on BAR_O cannot see an older phase.
  auto BAR_O = [&](int p) { return bar + 8u * (kAfterP + p); };
  auto BAR_PF = [&](int b) { return bar + 8u * (kAfterP + 2 + b); };
  auto XB = [&](int p) { return bar + 8u * (kAfterP + 2 + NB + p); };
  const uint32_t XE = bar + 8u * (kAfterP + 4 + NB);
  const uint32_t BAR_FIN = bar + 8u * (kAfterP + 5 + NB);
  // the scales of tile j complete phase j / SR of BAR_SC(j % SR)
  auto BAR_SC = [&](int s) { return bar + 8u * (kAfterP + 6 + NB + s); };
  static_assert(kAfterP + 6 + NB + SR == Lo::NBAR, "barrier count");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Lo::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + Lo::MISC + 4);
  float* xch = reinterpret_cast<float*>(gbase + Lo::XCH);
  float* ks_ring = reinterpret_cast<float*>(gbase + Lo::KS);
  float* vs_ring = reinterpret_cast<float*>(gbase + Lo::VS);
  float* vref_ring = reinterpret_cast<float*>(gbase + Lo::VREF);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const TileDesc8 t = describe8<DECODE>(a, tile);
  const int n_tiles = (t.key_end - t.key_begin + BN - 1) / BN;
  // a tile of at most 64 rows runs M = 64 products; its row r then sits in
  // TMEM lane 32 (r / 16) + r % 16
  const bool m64 = t.n_rows <= 64;

  // ---- Q: thread (wg, i) reads half of query row i
  const int wg = warp >> 2;
  const int i = (warp & 3) * 32 + lane;
  constexpr int QC = D / 16;  // 16-byte chunks of bf16 in half a row
  uint4 qv[QC];
  if (warp < 8) {
    int64_t q_row = 0, out_row = 0;
    int lim = 0;
    const bool ok = i < t.n_rows;
    if (ok) row_info8<DECODE>(a, t, kvh, i, q_row, out_row, lim);
    const uint4* src = reinterpret_cast<const uint4*>(a.q + q_row * D) + wg * QC;
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < QC; ++c) {
      qv[c] = ok ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {qv[c].x, qv[c].y, qv[c].z, qv[c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)),
                                 fabsf(__uint_as_float(w[e] & 0xffff0000u))));
    }
    xch[wg * BM + i] = amax;
  }
  if (tid == 0) {
    tc::mbar_init(BAR_Q, 8 * 32);
    for (int s = 0; s < NV; ++s) tc::mbar_init(BAR_VF(s), 4);
    for (int b = 0; b < NB; ++b) {
      tc::mbar_init(BAR_KF(b), 1);
      tc::mbar_init(BAR_S(b), 1);
      tc::mbar_init(BAR_P(b), 8 * 32);
      tc::mbar_init(BAR_PF(b), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(BAR_O(b), 1);
      tc::mbar_init(XB(b), 8 * 32);
    }
    tc::mbar_init(XE, 8 * 32);
    tc::mbar_init(BAR_FIN, 2);  // one commit per issuing thread
    for (int s = 0; s < SR; ++s) tc::mbar_init(BAR_SC(s), 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 8) {
    tc::tmem_alloc(rxk::smem_addr(tmem_slot), 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Registers by warpgroup: 2 x 152 + 88 + 120 = 4 x 128, what the block was
  // launched with.
  if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
  if (warp == 9) {
    // ------------------------------------------------- K and scale loader
    constexpr int SPL = BN / 32;  // keys lane + 32 i of a tile
    constexpr int LPR = D / 16;   // 16-byte chunks per row
    const uint8_t* kb = a.kc + int64_t(kvh) * a.head_stride;
    const float2* sb = a.scales + int64_t(kvh) * a.scale_stride;
    const int64_t row0 = a.tma_row_base + int64_t(kvh) * a.num_slots;
    // slots of tile j + 2 and scales of tile j + 1 are in flight while tile
    // j is loaded
    auto load_slots = [&](int j, int32_t (&dst)[SPL]) {
      const int k0 = t.key_begin + j * BN;
#pragma unroll
      for (int e = 0; e < SPL; ++e) {
        const int key = k0 + lane + 32 * e;
        dst[e] = (j < n_tiles && key < t.key_end) ? __ldg(t.trow + key) : -1;
      }
    };
    auto check_slots = [&](int j, int32_t (&s)[SPL]) {
      const int k0 = t.key_begin + j * BN;
#pragma unroll
      for (int e = 0; e < SPL; ++e)
        if (j < n_tiles && k0 + lane + 32 * e < t.key_end && (s[e] < 0 || s[e] >= a.num_slots)) {
          atomicOr(&g_kv8_att_error, 1);
          s[e] = 0;
        }
    };
    auto load_scales = [&](const int32_t (&s)[SPL], float2 (&dst)[SPL]) {
#pragma unroll
      for (int e = 0; e < SPL; ++e)
        dst[e] = s[e] >= 0 ? __ldg(sb + (s[e] >> a.block_log2)) : make_float2(0.f, 0.f);
    };
    int32_t cur[SPL], nxt[SPL], nx2[SPL];
    float2 sc[SPL], sn[SPL];
    load_slots(0, cur);
    load_slots(1, nxt);
    check_slots(0, cur);
    load_scales(cur, sc);
    float vref = 0.f;
    int pend = -1;    // gathered tile whose arrival is still to be signalled
    int issued = 0;
    for (int j = 0; j < n_tiles; ++j) {
      load_slots(j + 2, nx2);
      check_slots(j + 1, nxt);
      load_scales(nxt, sn);
      // stage j % NB is free once S_{j-NB} completed, and the scales of tile
      // j - SR have been read then (softmax j - 2 NB is done)
      const int st = j % NB;
      if (j >= NB && !__all_sync(0xffffffffu, tc::mbar_wait(BAR_S(st), uint32_t(j / NB - 1) & 1u,
                                                             abort_flag, kWaitLimit)))
        break;
      float vm = 0.f;
#pragma unroll
      for (int e = 0; e < SPL; ++e) vm = fmaxf(vm, sc[e].y);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
      vref = fmaxf(vref, vm);
      const float inv = 1.f / vref;
#pragma unroll
      for (int e = 0; e < SPL; ++e) {
        ks_ring[(j % SR) * BN + lane + 32 * e] = sc[e].x;
        vs_ring[(j % SR) * BN + lane + 32 * e] = sc[e].y * inv * kWeightBias;
      }
      if (lane == 0) vref_ring[j % SR] = vref;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(BAR_SC(j % SR));

      const uint32_t dst = base + Lo::K0 + uint32_t(st * Lo::K_BYTES);
      const int32_t first = __shfl_sync(0xffffffffu, cur[0], 0);
      bool run = first >= 0 && int64_t(first) + BN <= a.num_slots;
#pragma unroll
      for (int e = 0; e < SPL; ++e) run = run && cur[e] == first + lane + 32 * e;
      run = __all_sync(0xffffffffu, run);
      if (run) {
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(BAR_KF(st), uint32_t(Lo::K_BYTES));
#pragma unroll
          for (int cb = 0; cb < D / 128; ++cb)
            tc::tma_load_2d(dst + uint32_t(cb * BN * 128), tmk, cb * 128, int(row0 + first),
                            BAR_KF(st));
        }
      } else {
#pragma unroll
        for (int e = 0; e < SPL; ++e)
#pragma unroll 4
          for (int k = 0; k < LPR; ++k) {
            const int row = 32 * e + k * (32 / LPR) + lane / LPR;
            const int32_t s = __shfl_sync(0xffffffffu, cur[e], row & 31);
            const int ch = lane % LPR;
            rxk::cp_async_16(swz(dst, BN, row, ch), kb + int64_t(s < 0 ? 0 : s) * D + ch * 16,
                             s >= 0);
          }
        rxk::cp_async_commit();
      }
      issued = j + 1;
      // a gathered tile is signalled once the next tile's loads are on their
      // way, so two tiles' round trips overlap
      if (pend >= 0) {
        if (run)
          rxk::cp_async_wait<0>();
        else
          rxk::cp_async_wait<1>();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(BAR_KF(pend % NB));
      }
      pend = run ? -1 : j;
      if (pend >= 0 && j + 1 == n_tiles) {
        rxk::cp_async_wait<0>();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(BAR_KF(pend % NB));
        pend = -1;
      }
#pragma unroll
      for (int e = 0; e < SPL; ++e) {
        cur[e] = nxt[e];
        nxt[e] = nx2[e];
        sc[e] = sn[e];
      }
    }
    // no copy is in flight when the CTA gives up its shared memory (after an
    // abort, a box load may still be)
    rxk::cp_async_wait<0>();
    if (lane == 0) {
      int drain_abort = 0;
      const int end = pend >= 0 ? pend : issued;  // a gather never signalled is not waited for
      for (int j = end > NB ? end - NB : 0; j < end; ++j)
        tc::mbar_wait(BAR_KF(j % NB), uint32_t(j / NB) & 1u, &drain_abort, kWaitLimit);
    }
    __syncwarp();
  } else if (warp == 8 || warp == 10) {
    // ------------------------------------------------------------ MMA issue
    if (lane == 0) {
      const uint32_t MN = m64 ? 64 : BM;
      // shared-memory descriptors: 128-byte swizzle, 1024 bytes between
      // 8-row groups, version 1
      constexpr uint32_t DHI = (1024u >> 4) | (1u << 14) | (2u << 29);
      static_assert(Lo::V0 + NV * Lo::V_BYTES < (1 << 18), "descriptor address field");
      if (warp == 8) {
        // e4m3 A and B (type 0), fp32 accumulator, both K-major
        const uint32_t idesc = (1u << 4) | (uint32_t(BN >> 3) << 17) | ((MN >> 4) << 24);
        const uint32_t q_lo = ((sQ & 0x3FFFFu) >> 4) | (1u << 16);
        const uint32_t k_lo0 = (((base + Lo::K0) & 0x3FFFFu) >> 4) | (1u << 16);
        const bool ok = tc::mbar_wait(BAR_Q, 0, abort_flag, kWaitLimit);
        int sb = 0;
        uint32_t k_phase = 0, pf_phase = 0;
        for (int j = 0; ok && j < n_tiles; ++j) {
          if (j >= NB && !tc::mbar_wait(BAR_PF(sb), pf_phase, abort_flag, kWaitLimit)) break;
          if (!tc::mbar_wait(BAR_KF(sb), k_phase, abort_flag, kWaitLimit)) break;
          tc::tc_fence_after();
          const uint32_t k_lo = k_lo0 + uint32_t(sb) * (uint32_t(Lo::K_BYTES) >> 4);
          const uint32_t d_s = tmem + uint32_t(sb * BN);
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
              const uint32_t a_off =
                  uint32_t((part * Lo::Q_BYTES + (ks >> 2) * (BM * 128) + (ks & 3) * 32) >> 4);
              const uint32_t b_off = uint32_t(((ks >> 2) * (BN * 128) + (ks & 3) * 32) >> 4);
              mma8_ss(d_s, q_lo + a_off, k_lo + b_off, DHI, idesc, (part | ks) ? 1u : 0u);
            }
          tc::mma_commit(BAR_S(sb));  // also frees K stage sb
          if (++sb == NB) {
            sb = 0;
            k_phase ^= 1u;
            if (j >= NB) pf_phase ^= 1u;
          }
        }
      } else {
        // f16 A (TMEM) and B (shared, MN-major), fp32 accumulator
        const uint32_t idesc =
            (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | ((MN >> 4) << 24);
        const uint32_t v_lo0 =
            (((base + Lo::V0) & 0x3FFFFu) >> 4) | (uint32_t(BN * 128 / 16) << 16);
        int sv = 0, pb = 0;
        uint32_t v_phase = 0, p_phase = 0;
        for (int j = 0; j < n_tiles; ++j) {
          if (!tc::mbar_wait(BAR_P(pb), p_phase, abort_flag, kWaitLimit)) break;
          if (!tc::mbar_wait(BAR_VF(sv), v_phase, abort_flag, kWaitLimit)) break;
          tc::tc_fence_after();
          const uint32_t v_lo = v_lo0 + uint32_t(sv) * (uint32_t(Lo::V_BYTES) >> 4);
          const uint32_t p_t = tmem + uint32_t(pb * BN);
#pragma unroll
          for (int ks = 0; ks < BN / 16; ++ks)
            mma16_ts(tmem + uint32_t(Lo::O_COL), p_t + uint32_t(ks * 8),
                     v_lo + uint32_t(ks * 2048 / 16), DHI, idesc, (j > 0 || ks > 0) ? 1u : 0u);
          tc::mma_commit(BAR_O(j & 1));  // also frees V stage sv (== j & 1)
          tc::mma_commit(BAR_PF(pb));    // S buffer pb may take S_{j+NB}
          if (++sv == NV) {
            sv = 0;
            v_phase ^= 1u;
          }
          if (++pb == NB) {
            pb = 0;
            p_phase ^= 1u;
          }
        }
      }
      // drained once both threads' products completed, whatever the abort flag
      tc::mma_commit(BAR_FIN);
      int drain_abort = 0;
      tc::mbar_wait(BAR_FIN, 0, &drain_abort, kWaitLimit);
    }
    __syncwarp();
  }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;\n");
    // ------------------------------------------------------ V converters
    // A warp instruction reads 32 chunks of 16 codes, whole rows; a thread
    // has one chunk of NP rows of a tile.  While tile j's codes are converted,
    // tile j + 1's are in flight and tile j + 2's slots are read.
    constexpr int LPR = D / 16;
    constexpr int RPI = 32 / LPR;
    constexpr int NP = BN / (4 * RPI);
    const int row_in = (warp - 12) * RPI + lane / LPR;
    const int c16 = lane % LPR;
    const uint8_t* vb = a.vc + int64_t(kvh) * a.head_stride + c16 * 16;
    auto load_slots = [&](int j, int32_t (&dst)[NP]) {
      const int k0 = t.key_begin + j * BN + row_in;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int key = k0 + p * 4 * RPI;
        dst[p] = (j < n_tiles && key < t.key_end) ? __ldg(t.trow + key) : -1;
      }
    };
    auto load_codes = [&](int32_t (&s)[NP], uint4 (&dst)[NP]) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        if (s[p] >= a.num_slots) s[p] = 0;  // (the K loader reports it)
        // keys past the range are zeros (their weights are 0)
        dst[p] = s[p] >= 0 ? __ldg(reinterpret_cast<const uint4*>(vb + int64_t(s[p]) * D))
                           : make_uint4(0, 0, 0, 0);
      }
    };
    int32_t slot[NP];
    uint4 va[NP], vc[NP];
    load_slots(0, slot);
    load_codes(slot, va);
    load_slots(1, slot);
    auto step = [&](int j, uint4 (&cur)[NP], uint4 (&nxt)[NP]) -> bool {
      load_codes(slot, nxt);
      load_slots(j + 2, slot);
      const int sv = j & 1;
      if (j >= NV && !__all_sync(0xffffffffu, tc::mbar_wait(BAR_O(sv), uint32_t(j / NV - 1) & 1u,
                                                             abort_flag, kWaitLimit)))
        return false;
      const uint32_t dst = base + Lo::V0 + uint32_t(sv * Lo::V_BYTES);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int row = p * 4 * RPI + row_in;
        const uint32_t w[4] = {cur[p].x, cur[p].y, cur[p].z, cur[p].w};
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = kv8::to_f16x2((e & 1) ? w[e >> 1] >> 16 : w[e >> 1]);
        // chunks 2 c16 and 2 c16 + 1 of the f16 row; lanes of the upper column
        // blocks write theirs in the other order, so that the lanes of a row
        // hit all banks
        const bool sw = (c16 >> 2) & 1;
        const uint32_t a0 = swz(dst, BN, row, 2 * c16 + (sw ? 1 : 0));
        const uint32_t a1 = swz(dst, BN, row, 2 * c16 + (sw ? 0 : 1));
        st_shared_16(a0, sw ? h[4] : h[0], sw ? h[5] : h[1], sw ? h[6] : h[2], sw ? h[7] : h[3]);
        st_shared_16(a1, sw ? h[0] : h[4], sw ? h[1] : h[5], sw ? h[2] : h[6], sw ? h[3] : h[7]);
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(BAR_VF(sv));
      return true;
    };
    for (int j = 0; j < n_tiles; j += 2) {
      if (!step(j, va, vc)) break;
      if (j + 1 < n_tiles && !step(j + 1, vc, va)) break;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;\n");
    // ------------------------------------------------------------ softmax
    constexpr int HALF = BN / 2;
    const uint32_t tl = tmem + (uint32_t((warp & 3) * 32) << 16);
    // the row this thread's Q half belongs to, and its scale: 2^e with q 2^-e
    // at most 448 (limited below, where the scores vanish anyway)
    const float qmax = fmaxf(xch[i], xch[BM + i]);
    const int qe = max(kv8::scale_exponent(qmax), -80);
    const float qinv = kv8::pow2(-qe);
#pragma unroll
    for (int c = 0; c < QC; c += 2) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t w[4] = {qv[c + u].x, qv[c + u].y, qv[c + u].z, qv[c + u].w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t h2[2], l2[2];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const uint32_t x = w[2 * e + f];
            const float x0 = __uint_as_float(x << 16) * qinv;
            const float x1 = __uint_as_float(x & 0xffff0000u) * qinv;
            h2[f] = kv8::to_e4m3x2(x0, x1);
            const float2 r = kv8::f16x2_to_float2(kv8::to_f16x2(h2[f]));
            l2[f] = kv8::to_e4m3x2(x0 - r.x, x1 - r.y);
          }
          hi[2 * u + e] = h2[0] | (h2[1] << 16);
          lo[2 * u + e] = l2[0] | (l2[1] << 16);
        }
      }
      const int ch = wg * (QC / 2) + c / 2;
      st_shared_16(swz(sQ, BM, i, ch), hi[0], hi[1], hi[2], hi[3]);
      st_shared_16(swz(sQ + Lo::Q_BYTES, BM, i, ch), lo[0], lo[1], lo[2], lo[3]);
    }
    tc::fence_proxy_async_smem();
    tc::mbar_arrive(BAR_Q);
    // the tile row in this thread's TMEM lane
    const int row = m64 ? (((i >> 5) << 4) | (i & 15)) : i;
    const bool valid = (!m64 || (i & 16) == 0) && row < t.n_rows;
    int64_t q_row = 0, out_row = 0;
    int lim = t.key_end;
    if (valid) row_info8<DECODE>(a, t, kvh, row, q_row, out_row, lim);
    const float rmax = m64 ? fmaxf(xch[row], xch[BM + row]) : qmax;
    const int re = max(kv8::scale_exponent(rmax), -80);
    // a query that is not finite has no defined scores: its row is NaN
    const float rs = rmax < INFINITY ? a.scale_log2 * kv8::pow2(re) : NAN;
    // every thread has read the Q maxima before the slots are used again
    // below: the first tile's exchange slot is the other parity's
    float m_ref = -INFINITY, vref = 0.f;
    float l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      const int s = j % NB;
      if (!__all_sync(0xffffffffu, tc::mbar_wait(BAR_SC(j % SR), uint32_t(j / SR) & 1u, abort_flag,
                                                  kWaitLimit) &&
                                       tc::mbar_wait(BAR_S(s), uint32_t(j / NB) & 1u, abort_flag,
                                                     kWaitLimit))) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const int k0 = t.key_begin + j * BN + wg * HALF;
      const bool need_mask = k0 + HALF > t.nomask_end;
      uint32_t sr[HALF];
      tc::tmem_ld_row<HALF>(tl + uint32_t(s * BN + wg * HALF), sr);
      tc::tmem_ld_wait();
      float x[HALF];
      const float4* ks4 = reinterpret_cast<const float4*>(ks_ring + (j % SR) * BN + wg * HALF);
#pragma unroll
      for (int e = 0; e < HALF; e += 4) {
        const float4 k4 = ks4[e >> 2];
        const float2 y0 = mul2(make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])),
                               make_float2(k4.x, k4.y));
        const float2 y1 = mul2(make_float2(__uint_as_float(sr[e + 2]), __uint_as_float(sr[e + 3])),
                               make_float2(k4.z, k4.w));
        x[e] = y0.x;
        x[e + 1] = y0.y;
        x[e + 2] = y1.x;
        x[e + 3] = y1.y;
      }
      if (need_mask) {
#pragma unroll
        for (int e = 0; e < HALF; ++e)
          if (k0 + e >= lim) x[e] = -INFINITY;
      }
      float mx4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int e = 4; e < HALF; e += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          mx4[u] = e + 4 + u < HALF ? fmaxf(fmaxf(mx4[u], x[e + u]), x[e + 4 + u])
                                    : fmaxf(mx4[u], x[e + u]);
      const float mx_half = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
      // the other half's max of this row (double-buffered by tile parity: a
      // thread writes tile j + 2's slot only after every thread has passed
      // tile j + 1's exchange, hence has read tile j's; tile 0 uses parity 1,
      // the Q maxima lie in parity 0)
      const int xp = (j + 1) & 1;
      xch[(xp * 2 + wg) * BM + i] = mx_half;
      tc::mbar_arrive(XB(j & 1));
      if (!__all_sync(0xffffffffu,
                      tc::mbar_wait(XB(j & 1), (j >> 1) & 1, abort_flag, kWaitLimit))) {
        ok = false;
        break;
      }
      const float mx = rs * fmaxf(mx_half, xch[(xp * 2 + (1 - wg)) * BM + i]);
      const float m_new = fmaxf(m_ref, mx);
      const float v_new = vref_ring[j % SR];
      if (j == 0) {
        m_ref = m_new;
        vref = v_new;
      } else {
        const bool need = m_new > m_ref + kRescaleThreshold;
        const bool vneed = v_new > vref;  // the same for every thread of the CTA
        if (__any_sync(0xffffffffu, need || vneed)) {
          // O is rescaled once PV_{j-1} has written it; each warpgroup takes
          // half of its columns
          if (!__all_sync(0xffffffffu, tc::mbar_wait(BAR_O((j - 1) & 1), ((j - 1) >> 1) & 1,
                                                      abort_flag, kWaitLimit))) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const float alpha = need ? rxk::fast_exp2(m_ref - m_new) : 1.f;
          const float f = vneed ? alpha * (vref / v_new) : alpha;
#pragma unroll
          for (int cc = 0; cc < D / 64; ++cc) {
            uint32_t r[32];
            const uint32_t col = uint32_t(Lo::O_COL + wg * (D / 2) + cc * 32);
            tc::tmem_ld32(tl + col, r);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
            tc::tmem_st32(tl + col, r);
          }
          l *= alpha;
          if (need) m_ref = m_new;
          vref = v_new;
        }
      }
      const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
      const float2 rs2 = make_float2(rs, rs), nm2 = make_float2(neg_m, neg_m);
      float2 l2[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) l2[u] = make_float2(0.f, 0.f);
      const float4* vs4 = reinterpret_cast<const float4*>(vs_ring + (j % SR) * BN + wg * HALF);
#pragma unroll
      for (int cc = 0; cc < HALF / 32; ++cc) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 v4 = vs4[cc * 8 + (e >> 2)];
#pragma unroll
          for (int u = 0; u < 4; u += 2) {
            const int n = cc * 32 + e + u;
            const float2 y = fma2(make_float2(x[n], x[n + 1]), rs2, nm2);
            const float2 p = make_float2(rxk::fast_exp2(y.x), rxk::fast_exp2(y.y));
            l2[((e + u) >> 1) & 3] = add2(l2[((e + u) >> 1) & 3], p);
            const float2 w = mul2(p, u ? make_float2(v4.z, v4.w) : make_float2(v4.x, v4.y));
            pk[(e + u) >> 1] = pack_f16(w.x, w.y);
          }
        }
        // two keys per column over the first BN / 2 columns of S_j's buffer
        tmem_st16x(tl + uint32_t(s * BN + wg * (HALF / 2) + 16 * cc), pk);
      }
      const float2 ls = add2(add2(l2[0], l2[1]), add2(l2[2], l2[3]));
      l += ls.x + ls.y;
      tc::tmem_st_wait();
      tc::tc_fence_before();
      tc::mbar_arrive(BAR_P(s));
    }
    // ----------------------------------------------------------- epilogue
    const bool fin = ok && n_tiles > 0 &&
                     __all_sync(0xffffffffu, tc::mbar_wait(BAR_FIN, 0, abort_flag, kWaitLimit));
    // the row sums go through the parity that the last tile did not use
    const int xp = n_tiles & 1 ? 0 : 1;
    if (fin) xch[(xp * 2 + wg) * BM + i] = l;
    tc::mbar_arrive(XE);
    const bool xok = __all_sync(0xffffffffu, tc::mbar_wait(XE, 0, abort_flag, kWaitLimit));
    if (fin && xok) {
      tc::tc_fence_after();
      const float l_all = l + xch[(xp * 2 + (1 - wg)) * BM + i];
      const float inv = vref * (1.f / kWeightBias) / l_all;
      // warpgroup w writes output columns [w D/2, (w+1) D/2): through shared
      // memory (Q and the K and V stages are idle), so that a warp writes
      // whole contiguous row segments
      constexpr int HC = D / 2;
      constexpr int PITCH = HC * 4 + 16;
      static_assert(2 * BM * PITCH <= Lo::XCH, "staging fits before the exchange slots");
      uint8_t* stage = gbase + wg * (BM * PITCH);
#pragma unroll
      for (int cc = 0; cc < HC / 32; ++cc) {
        uint32_t r[32];
        tc::tmem_ld32(tl + uint32_t(Lo::O_COL + wg * HC + cc * 32), r);
        tc::tmem_ld_wait();
        float4* s4 = reinterpret_cast<float4*>(stage + i * PITCH + cc * 128);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          s4[e] = make_float4(__uint_as_float(r[4 * e]) * inv, __uint_as_float(r[4 * e + 1]) * inv,
                              __uint_as_float(r[4 * e + 2]) * inv,
                              __uint_as_float(r[4 * e + 3]) * inv);
      }
      __syncwarp();
      const int qrow = (warp & 3) * 32;
      const bool to_bf16 = !DECODE && a.out_bf16;
      uint8_t* obase = static_cast<uint8_t*>(DECODE ? static_cast<void*>(a.ws_o) : a.out);
      const long long my_row = valid ? (long long)out_row : -1ll;
      if (to_bf16) {
        constexpr int CPR = HC / 8;  // 16-byte pieces (8 columns) per row
#pragma unroll 4
        for (int k = 0; k < CPR; ++k) {
          const int idx = k * 32 + lane;
          const int rr = idx / CPR, c8 = idx - rr * CPR;
          const long long ro = __shfl_sync(0xffffffffu, my_row, rr);
          const float4* v =
              reinterpret_cast<const float4*>(stage + (qrow + rr) * PITCH + c8 * 32);
          const float4 v0 = v[0], v1 = v[1];
          if (ro >= 0)
            *reinterpret_cast<uint4*>(obase + (ro * D + wg * HC + c8 * 8) * 2) =
                make_uint4(rxk::pack_bf16(v0.x, v0.y), rxk::pack_bf16(v0.z, v0.w),
                           rxk::pack_bf16(v1.x, v1.y), rxk::pack_bf16(v1.z, v1.w));
        }
      } else {
        constexpr int CPR = HC / 4;
#pragma unroll 4
        for (int k = 0; k < CPR; ++k) {
          const int idx = k * 32 + lane;
          const int rr = idx / CPR, c4 = idx - rr * CPR;
          const long long ro = __shfl_sync(0xffffffffu, my_row, rr);
          const float4 v =
              *reinterpret_cast<const float4*>(stage + (qrow + rr) * PITCH + c4 * 16);
          if (ro >= 0)
            *reinterpret_cast<float4*>(obase + (ro * D + wg * HC + c4 * 4) * 4) = v;
        }
      }
      if (valid && wg == 0) (DECODE ? a.ws_lse : a.lse)[out_row] = m_ref * kLn2 + logf(l_all);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) atomicOr(&g_kv8_att_error, 2);
  if (warp == 8) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

}  // namespace
