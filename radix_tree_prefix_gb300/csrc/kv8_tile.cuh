// Tensor-core tile of attention over the 8-bit KV pool: 128 query rows that
// read one KV head over one key range (tcgen05, TMEM; sm_103a).  Included by
// kv8_attention.cu.
//
// Per key tile of BN keys (128 at head_dim 128, 64 at 256):
//   S = Q K^T      kind::f8f6f4, K's codes as they lie in the pool and Q as a
//                  sum of two e4m3 operands;
//   softmax        x = S ks rs, P = 2^(x - m + 6) in f16 into TMEM;
//   O += P V       kind::f16, V's codes converted to f16 times vs / vref.
// Q split: a bf16 query has 8 significant bits, an e4m3 number 4.  With the
// row scaled by a power of two to at most 448, hi = e4m3(q) and lo =
// e4m3(q - hi) add up to q exactly down to 2^-9.8 of the row's largest
// magnitude, and are off by at most 2^-17.8 of that below (lo's steps end at
// 2^-9, and the largest is above 224).  The two products
// cost what one f16 product does (the e4m3 rate is twice f16's), and K needs
// no conversion and half the shared memory.  Splitting P the same way was
// not taken: a weight below 2^-18 of the row's largest would be lost, and
// long contexts with one dominant key have most of their sum there.  P stays
// f16, so V is converted.
// vref is at least the largest V scale of the tile and the tiles before it (O
// is rescaled when it grows, which a factor of 4 of headroom makes rare).  A
// power-of-two scale, what rx_kv8_store writes, is exact in f16 over vref from
// 2^-24 of it, and its product with every code from 2^-15 of it (between them a
// product is off by 2^-25 vref at most); any other is rounded there, and again in
// its product with a code.
//
// 512 threads:
//   warps 0-7    softmax in two warpgroups that split every key tile's keys;
//                thread (w, i) owns query row i = TMEM lane i;
//   warps 8-11   convert V: codes into registers a tile ahead, by slot, then to
//                swizzled shared memory;
//   warp 12      issues S; warp 13 issues P V;
//   warp 14      loads K's codes, TMA boxes where the slots of the tile or of 16
//                keys of it are consecutive (runs and pages), and a cp.async
//                gather for other groups of 16; and the tile's scales.
// The roles run side by side, so the code of their loops together is the
// working set of the instruction cache (32 KB): what is rare is kept rolled.
// A tile takes about 1.3 us per key tile at both head dimensions (8,191 queries
// over themselves, 32 / 8 heads, d = 128: 674 us, 42 % of the bf16 peak on the
// causal products).  Issue and latency of the 15 warps' instructions set the
// pace (a softmax warp works 2,050 clocks a key tile, 670 if it is alone), not
// the tensor pipe (35 % busy) or shared memory (30 %).  At 128 registers a thread
// the d = 128 kernels spill a little (extend 12 bytes, with clusters 28; decode
// 28, with clusters 32).
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
// A score is S (at most 448^2 D < 2^26) times its K scale (up to 2^120) times the
// row's scale.  The K scale comes times 2^-20 and the mantissa of scale log2(e)
// (Args8::key_mul), so that the first product does not overflow, and the row's
// scale is a power of two, so that the second is exact: the largest score and the
// reference taken from it then differ by nothing, however large they are.
constexpr int kKeyShift = 20;

template <int HEAD_DIM>
struct Tile8 {
  static constexpr int D = HEAD_DIM;
  static constexpr int BN = D == 128 ? 128 : 64;
  static constexpr int NS = 3;             // S buffers (TMEM)
  static constexpr int NB = 3;             // K stages
  static constexpr int NV = 2;             // V stages
  static constexpr int SR = 8;             // ring of the tiles' scales
  static constexpr int Q_BYTES = BM * D;   // of each part
  static constexpr int K_BYTES = BN * D;
  static constexpr int V_BYTES = BN * D * 2;
  static constexpr int Q = 0;
  static constexpr int K0 = Q + 2 * Q_BYTES;
  static constexpr int V0 = K0 + NB * K_BYTES;
  static constexpr int XCH = V0 + NV * V_BYTES;      // [2][2 warpgroups][128] floats
  static constexpr int KS = XCH + 2 * 2 * 128 * 4;   // [SR][BN] K scales
  static constexpr int VREF = KS + SR * BN * 4;      // [SR]
  static constexpr int BAR = VREF + SR * 4;
  // q, kfull[NB], vfull[NV], s[NS], p[NS], o[2], pf[NS], xch[2], sum, final
  static constexpr int NBAR = 1 + NB + NV + 3 * NS + 2 + 2 + 1 + 1;
  static constexpr int MISC = BAR + NBAR * 8;
  static constexpr int BYTES = MISC + 16 + 1024;  // slack to align the swizzled tiles
  static constexpr int O_COL = D == 128 ? NS * BN : 256;
  static_assert(NS * BN <= O_COL && O_COL + D <= 512, "TMEM budget");
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
};

// Tensor maps of the pool's K codes: boxes of 128 columns by a tile's keys or 16.
struct Maps8 {
  CUtensorMap k, k16;
};

struct TileDesc8 {
  const int32_t* trow;
  int key_begin, key_end, nomask_end, n_rows;
  int gr0, q_base, prefix;
  int member_off, part_base;
  bool grows;  // steps of the plan store into its segment
};

template <bool DECODE>
__device__ __forceinline__ TileDesc8 describe8(const Args8& a, int tile) {
  TileDesc8 t;
  if constexpr (DECODE) {
    const int32_t* w = a.work + int64_t(a.n_small + tile) * RX_WORK_WORDS;
    t.trow = a.table + int64_t(w[0]) * a.row_stride;
    t.key_begin = w[1];
    t.grows = w[7] > 0;
    t.key_end = t.grows ? min(w[2], w[7] + a.step) : w[2];
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
    t.grows = false;
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

// D(tmem) (+)= A B, shared-memory descriptors as 32-bit halves with a common
// high half.
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

// Four e4m3 codes as two f16 pairs, exactly.
__device__ __forceinline__ void to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
      " cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Add `bytes` to the transaction count of the barrier's phase.
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
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

// A load from the pool.  A decode tile may be chained to a step's store, which
// then writes the pool while the kernel is alive: the non-coherent path is for
// memory that nothing writes so long (a scale's 32-byte sector holds its
// neighbours' too, which an item before on this SM may have fetched), so those
// loads go to L2.
template <bool DECODE, typename T>
__device__ __forceinline__ T ld_pool(const T* p) {
  if constexpr (DECODE)
    return __ldcg(p);
  else
    return __ldg(p);
}

// The CTA's place in its cluster, and an address in another CTA's shared memory.
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return int(r);
}
__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(r));
  return int(r);
}
// Every thread of the cluster meets; what was written to shared memory before
// is seen after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n"
               "barrier.cluster.wait.acquire.aligned;\n" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// SPLIT: the CTAs of a cluster share the tile's keys (a part has kMinPart key
// tiles at least, so short ranges use fewer CTAs) and join their normalised
// partial rows through each other's shared memory: no workspace, one launch.
constexpr int kMinPart = 3;
template <int D, bool DECODE, bool SPLIT = false>
__device__ __forceinline__ void tile8(const Args8& a, const Maps8& maps, uint8_t* smem_raw,
                                      int tile, int kvh) {
  using Lo = Tile8<D>;
  constexpr int BN = Lo::BN, NB = Lo::NB, NV = Lo::NV, NS = Lo::NS, SR = Lo::SR;
  const uint32_t raw = rxk::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base + Lo::Q;
  const uint32_t bar = base + Lo::BAR;
  // Rings of n barriers: entry j % n completes its phase j / n for tile j.
  constexpr uint32_t kKF = 1, kVF = kKF + NB, kS = kVF + NV, kP = kS + NS, kO = kP + NS,
                     kPF = kO + 2, kX = kPF + NS, kXE = kX + 2, kFin = kXE + 1;
  static_assert(kFin + 1 == Lo::NBAR, "barrier count");
  const uint32_t BAR_Q = bar;
  auto BAR_KF = [&](int j) { return bar + 8u * (kKF + j % NB); };  // K converted
  auto BAR_VF = [&](int j) { return bar + 8u * (kVF + j % NV); };  // V converted
  auto BAR_S = [&](int j) { return bar + 8u * (kS + j % NS); };    // S_j complete
  auto BAR_P = [&](int j) { return bar + 8u * (kP + j % NS); };    // P_j written
  // P V_j complete, in a ring of two and one of NS.  S_j is issued after PV_{j-NS}
  // completed, so once S_j is complete, PV_{j-3} is, and a wait for PV_{j-1} on
  // BAR_O cannot see an older phase.
  auto BAR_O = [&](int j) { return bar + 8u * (kO + (j & 1)); };
  auto BAR_PF = [&](int j) { return bar + 8u * (kPF + j % NS); };
  auto XB = [&](int j) { return bar + 8u * (kX + (j & 1)); };
  const uint32_t XE = bar + 8u * kXE;
  const uint32_t BAR_FIN = bar + 8u * kFin;
  auto wait = [&](uint32_t b, int phase, volatile int* abort) {
    return tc::mbar_wait(b, uint32_t(phase) & 1u, abort, kWaitLimit);
  };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Lo::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + Lo::MISC + 4);
  float* xch = reinterpret_cast<float*>(gbase + Lo::XCH);
  float* ks_ring = reinterpret_cast<float*>(gbase + Lo::KS);
  float* vref_ring = reinterpret_cast<float*>(gbase + Lo::VREF);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  TileDesc8 t = describe8<DECODE>(a, tile);
  int parts = 1, rank = 0;
  if constexpr (SPLIT) {
    const int all = (t.key_end - t.key_begin + BN - 1) / BN;
    rank = cluster_rank();
    parts = max(1, min(cluster_size(), all / kMinPart));
    // (every CTA of the cluster decides alike)
    if (parts == 1 && rank > 0) return;
    const int first = int(int64_t(all) * rank / parts);
    const int last = int(int64_t(all) * (rank + 1) / parts);
    if (rank < parts) t.key_end = min(t.key_end, t.key_begin + last * BN);
    t.key_begin = rank < parts ? t.key_begin + first * BN : t.key_end;  // (no part: no keys)
  }
  const int n_tiles = (t.key_end - t.key_begin + BN - 1) / BN;
  // Chained to a step's store: a segment that steps of the plan store into
  // waits for it, any other reads what no kernel of the run writes (a block of
  // slots holds no rows of a shared segment and of a tail), and waits before it
  // writes partial rows.
  if (DECODE && a.chained && t.grows) rxk::griddep_wait();
  if (DECODE && parts == 1 && n_tiles <= 0) {
    // keys that a later step of the plan brings: empty partial rows
    if (a.chained) rxk::griddep_wait();
    if (a.chained && a.counter && tid == 0) release_counter(a.counter);
    for (int idx = tid; idx < t.n_rows * (D / 4); idx += kTileThreads) {
      const int col = idx % (D / 4) * 4;
      int64_t q_row, out_row;
      int lim;
      row_info8<DECODE>(a, t, kvh, idx / (D / 4), q_row, out_row, lim);
      *reinterpret_cast<float4*>(a.ws_o + out_row * D + col) = make_float4(0.f, 0.f, 0.f, 0.f);
      if (col == 0) a.ws_lse[out_row] = -INFINITY;
    }
    return;
  }
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
    tc::mbar_init(BAR_Q, 8);
    for (int j = 0; j < NB; ++j) tc::mbar_init(BAR_KF(j), 2);  // the codes, and the scales
    for (int j = 0; j < NV; ++j) tc::mbar_init(BAR_VF(j), 4);
    for (int j = 0; j < NS; ++j) {
      tc::mbar_init(BAR_S(j), 2);  // the commit, and the issuer
      tc::mbar_init(BAR_P(j), 8);
      tc::mbar_init(BAR_PF(j), 1);
    }
    for (int j = 0; j < 2; ++j) {
      tc::mbar_init(BAR_O(j), 1);
      tc::mbar_init(XB(j), 8 * 32);
    }
    tc::mbar_init(XE, 8 * 32);
    tc::mbar_init(BAR_FIN, 2);  // one commit per issuing thread
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 12) {
    tc::tmem_alloc(rxk::smem_addr(tmem_slot), 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Registers by warpgroup: 2 x 152 + 120 + 88 = 4 x 128, what the block was
  // launched with.
  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
    if (warp == 14) {
      // ------------------------------------------------------------ K loader
      constexpr int LPR = D / 16;   // 16-byte pieces per row
      constexpr int RPI = 32 / LPR;  // rows a gather instruction copies
      constexpr int rows = BN;
      constexpr int SPL = BN / 32;
      const uint8_t* src0 = a.kc + int64_t(kvh) * a.head_stride + (lane % LPR) * 16;
      const int64_t row0 = a.tma_row_base + int64_t(kvh) * a.num_slots;
      // lane l holds the slots of keys l, l + 32, .. of a tile; the next tile's
      // are on their way while one is loaded
      int32_t cur[SPL], nxt[SPL];
      auto load_slots = [&](int k0, int32_t (&dst)[SPL]) {
  #pragma unroll
        for (int e = 0; e < SPL; ++e)
          dst[e] = k0 + lane + 32 * e < t.key_end ? __ldg(t.trow + k0 + lane + 32 * e) : -1;
      };
      load_slots(t.key_begin, nxt);
      // It passes on the scales too: K's, and vref.  The next tile's are read a
      // tile ahead.
      const float2* sb = a.scales + int64_t(kvh) * a.scale_stride;
      float2 sc[SPL], sn[SPL];
      auto load_scales = [&](int k0, const int32_t (&s)[SPL], float2 (&dst)[SPL]) {
  #pragma unroll
        for (int e = 0; e < SPL; ++e) {
          // (a bad slot is reported and read as slot 0 when its tile is loaded)
          const uint32_t at = uint32_t(s[e]) < uint32_t(a.num_slots) ? uint32_t(s[e]) : 0u;
          dst[e] = k0 + lane + 32 * e < t.key_end ? ld_pool<DECODE>(sb + (at >> a.block_log2))
                                                  : make_float2(0.f, 0.f);
        }
      };
      float vref = 0.f;
      load_scales(t.key_begin, nxt, sn);
      uint32_t pend = 0;  // barrier of gathered rows whose arrival is still to be signalled
      int j = 0;
  #pragma unroll 1
      for (; j < n_tiles; ++j) {
        const int k0 = t.key_begin + j * rows;
        bool bad = false, whole = true;
  #pragma unroll
        for (int e = 0; e < SPL; ++e) {
          cur[e] = nxt[e];
          if (k0 + lane + 32 * e < t.key_end && (cur[e] < 0 || cur[e] >= a.num_slots)) {
            bad = true;
            cur[e] = 0;
          }
        }
        load_slots(k0 + rows, nxt);
        if (bad) atomicOr(&g_kv8_att_error, 1);
        const int32_t first = __shfl_sync(0xffffffffu, cur[0], 0);
  #pragma unroll
        for (int e = 0; e < SPL; ++e) whole = whole && cur[e] == first + lane + 32 * e;
        whole = __all_sync(0xffffffffu, whole && first >= 0);
        // stage j % NB is free once S_{j-NB} completed
        static_assert(NB == NS, "a K stage is freed by the S of its index");
        if (j >= NB && !__all_sync(0xffffffffu, wait(BAR_S(j), j / NB - 1, abort_flag))) break;
        const uint32_t full = BAR_KF(j), dst = base + Lo::K0 + uint32_t((j % NB) * Lo::K_BYTES);
        uint32_t done = 0;  // barrier of this stage, if it needs a signal later
        if (whole) {
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(full, uint32_t(rows * D));
  #pragma unroll
            for (int cb = 0; cb < D / 128; ++cb)
              tc::tma_load_2d(dst + uint32_t(cb * rows * 128), &maps.k, cb * 128,
                              int(row0 + first), full);
          }
        } else {
          // groups of 16 keys: a box load where their slots are consecutive;
          // the rest is gathered (past the key range a slot is -1, its row zeros)
          uint32_t run = 0;
          int32_t gfirst = 0;  // lane g: first slot of group g
  #pragma unroll
          for (int e = 0; e < SPL; ++e) {
            const int32_t f = __shfl_sync(0xffffffffu, cur[e], lane & 16);
            const uint32_t m = __ballot_sync(0xffffffffu, f >= 0 && cur[e] == f + (lane & 15));
            if ((m & 0xffffu) == 0xffffu) run |= 1u << (2 * e);
            if (m >> 16 == 0xffffu) run |= 2u << (2 * e);
            const int32_t g = __shfl_sync(0xffffffffu, cur[e], (lane & 1) << 4);
            if ((lane >> 1) == e) gfirst = g;
          }
          const bool all = __popc(run) * 16 == rows;
          if (lane == 0 && run) {
            const uint32_t bytes = uint32_t(__popc(run)) * 16u * D;
            if (all)
              tc::mbar_arrive_expect_tx(full, bytes);
            else
              mbar_expect_tx(full, bytes);
          }
          __syncwarp();
          if (lane < 8 && ((run >> lane) & 1u)) {
  #pragma unroll 1
            for (int cb = 0; cb < D / 128; ++cb)
              tc::tma_load_2d(dst + uint32_t(cb * rows * 128 + lane * 16 * 128), &maps.k16,
                              cb * 128, int(row0 + gfirst), full);
          }
          if (!all) {
  #pragma unroll 1
            for (int e = 0; e < rows / 32; ++e) {
              int32_t ce = cur[0];
  #pragma unroll
              for (int u = 1; u < SPL; ++u)
                if (e == u) ce = cur[u];
  #pragma unroll 4
              for (int k = 0; k < 32; k += RPI) {
                const int row = k + lane / LPR;
                const int32_t sl = __shfl_sync(0xffffffffu, ce, row);
                if (!((run >> (2 * e + (row >> 4))) & 1u))
                  rxk::cp_async_16(swz(dst, rows, 32 * e + row, lane % LPR),
                                   src0 + int64_t(sl < 0 ? 0 : sl) * D, sl >= 0);
              }
            }
            rxk::cp_async_commit();
            done = full;
          }
        }
        // a gathered stage is signalled once the next one's loads are on their
        // way, so two stages' round trips overlap
        if (pend) {
          if (done)
            rxk::cp_async_wait<1>();
          else
            rxk::cp_async_wait<0>();
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(pend);
        }
        pend = done;
        // S_{j-NB} has completed, so the softmax of tile j - NB - NS is done, and
        // with it every read of the ring's entry
        static_assert(SR > NB + NS, "scale ring");
  #pragma unroll
        for (int e = 0; e < SPL; ++e) sc[e] = sn[e];
        load_scales(k0 + rows, nxt, sn);
        float vm = 0.f;
  #pragma unroll
        for (int e = 0; e < SPL; ++e) {
          vm = fmaxf(vm, sc[e].y);
          ks_ring[(j % SR) * BN + lane + 32 * e] = sc[e].x * a.key_mul;
        }
        // (positive floats compare as integers)
        vm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vm)));
        if (vm > vref) vref = 4.f * vm;
        if (lane == 0) vref_ring[j % SR] = vref;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(BAR_KF(j));
      }
      rxk::cp_async_wait<0>();
      if (pend) {
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(pend);
      }
      // No copy is in flight when the CTA gives up its shared memory: every box
      // load has been consumed, unless a wait gave up, and then the stages' last
      // phases get one more bounded wait.
      if (lane == 0 && *abort_flag) {
        int drain_abort = 0;
        for (int e = j > NB ? j - NB : 0; e < j; ++e) wait(BAR_KF(e), e / NB, &drain_abort);
      }
      __syncwarp();
    } else if (warp < 14) {
      // ------------------------------------------------------------ MMA issue
      if (lane == 0) {
        // shared-memory descriptors: 128-byte swizzle, 1024 bytes between
        // 8-row groups, version 1
        constexpr uint32_t DHI = (1024u >> 4) | (1u << 14) | (2u << 29);
        static_assert(Lo::XCH < (1 << 18), "descriptor address field");
        if (warp == 12) {
          // e4m3 A and B (type 0), fp32 accumulator, both K-major
          constexpr uint32_t idesc =
              (1u << 4) | (uint32_t(BN >> 3) << 17) | (uint32_t(BM >> 4) << 24);
          const uint32_t q_lo = ((sQ & 0x3FFFFu) >> 4) | (1u << 16);
          const uint32_t k_lo0 = (((base + Lo::K0) & 0x3FFFFu) >> 4) | (1u << 16);
          const bool ok = wait(BAR_Q, 0, abort_flag);
  #pragma unroll 1
          for (int j = 0; ok && j < n_tiles; ++j) {
            // buffer j % NS is free once P V_{j-NS} has read its P
            if (j >= NS && !wait(BAR_PF(j), j / NS - 1, abort_flag)) break;
            if (!wait(BAR_KF(j), j / NB, abort_flag)) break;
            tc::tc_fence_after();
            const uint32_t k_lo = k_lo0 + uint32_t(j % NB) * (uint32_t(Lo::K_BYTES) >> 4);
            const uint32_t d_s = tmem + uint32_t((j % NS) * BN);
            // Q's two parts by D / 128 blocks of 128 columns, 4 steps each
  #pragma unroll 1
            for (int blk = 0; blk < 2 * (D / 128); ++blk) {
              const uint32_t q_at = q_lo + uint32_t(blk) * uint32_t(BM * 128 / 16);
              const uint32_t k_at = k_lo + uint32_t(blk % (D / 128)) * uint32_t(BN * 128 / 16);
  #pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma8_ss(d_s, q_at + uint32_t(ks * 2), k_at + uint32_t(ks * 2), DHI, idesc,
                        (blk | ks) ? 1u : 0u);
            }
            tc::mma_commit(BAR_S(j));   // also frees the K stage
            tc::mbar_arrive(BAR_S(j));  // (passes the scales on, seen through KF)
          }
        } else {
          // f16 A (TMEM) and B (shared, MN-major), fp32 accumulator
          constexpr uint32_t idesc =
              (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | (uint32_t(BM >> 4) << 24);
          const uint32_t v_lo0 =
              (((base + Lo::V0) & 0x3FFFFu) >> 4) | (uint32_t(BN * 128 / 16) << 16);
  #pragma unroll 1
          for (int j = 0; j < n_tiles; ++j) {
            if (!wait(BAR_VF(j), j / NV, abort_flag)) break;
            if (!wait(BAR_P(j), j / NS, abort_flag)) break;
            tc::tc_fence_after();
            const uint32_t v_lo = v_lo0 + uint32_t(j % NV) * (uint32_t(Lo::V_BYTES) >> 4);
            const uint32_t p_t = tmem + uint32_t((j % NS) * BN);
  #pragma unroll
            for (int ks = 0; ks < BN / 16; ++ks)
              mma16_ts(tmem + uint32_t(Lo::O_COL), p_t + uint32_t(ks * 8),
                       v_lo + uint32_t(ks * 2048 / 16), DHI, idesc, (j > 0 || ks > 0) ? 1u : 0u);
            tc::mma_commit(BAR_O(j));   // also frees the V stage
            tc::mma_commit(BAR_PF(j));  // S buffer j % NS may take S_{j+NS}
          }
        }
        // drained once both threads' products completed, whatever the abort flag
        tc::mma_commit(BAR_FIN);
        int drain_abort = 0;
        wait(BAR_FIN, 0, &drain_abort);
      }
      __syncwarp();
    } else if (DECODE && a.chained) {
      // (warp 15, idle otherwise) the streams beside the tiles start once the
      // store has completed
      rxk::griddep_wait();
      if (a.counter && lane == 0) release_counter(a.counter);
      __syncwarp();
      rxk::griddep_launch_dependents();
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;\n");
    // ------------------------------------------------------ V converters
    // A warp instruction reads 32 pieces of 16 codes, whole rows; a thread has
    // a piece of NP rows of a tile, row p * RPP + row_in for p < NP.  A piece's
    // registers are refilled with the next tile's as soon as it is converted.
    constexpr int LPR = D / 16;
    constexpr int RPP = 4 * (32 / LPR);
    constexpr int NP = BN / RPP;
    constexpr int SPL = BN / 32;  // keys lane + 32 e of a tile
    // Lane bits: piece within a column block (2), row (1), column block, row.
    // A store's phase of 8 lanes is then two rows by four pieces of one column
    // block, which hit all banks.
    const int c16 = (lane & 3) | ((lane >> 3) % (LPR / 4)) << 2;
    const int row_in = (warp & 3) * (32 / LPR) + ((lane >> 2) & 1) + 2 * ((lane >> 3) / (LPR / 4));
    const uint8_t* src = a.vc + int64_t(kvh) * a.head_stride + c16 * 16;
    const float2* sb = a.scales + int64_t(kvh) * a.scale_stride;
    // pieces 2 c16 and 2 c16 + 1 of the f16 row (RPP is a multiple of 8: the
    // swizzle of all its rows is the same)
    uint8_t* at0 = gbase + swz(Lo::V0, BN, row_in, 2 * c16);
    uint8_t* at1 = gbase + swz(Lo::V0, BN, row_in, 2 * c16 + 1);
    // lane l holds the slots and scales of keys l, l + 32, .. of a tile
    int32_t slot[SPL];
    float sc[SPL];
    uint4 v[NP];
    auto load_slots = [&](int j) {
      const int k0 = t.key_begin + j * BN + lane;
#pragma unroll
      for (int e = 0; e < SPL; ++e)
        slot[e] = __ldg(t.trow + min(k0 + 32 * e, t.key_end - 1));
    };
    // keys past the range take the last key's slot and scales of 0: their weights
    // are 0, and 0 V is 0 for codes that count anyway
    auto load_scales = [&](int j) {
      const int k0 = t.key_begin + j * BN + lane;
#pragma unroll
      for (int e = 0; e < SPL; ++e) {
        // (the K loader reports a bad slot)
        if (slot[e] < 0 || slot[e] >= a.num_slots) slot[e] = 0;
        sc[e] = k0 + 32 * e < t.key_end ? ld_pool<DECODE>(&sb[slot[e] >> a.block_log2].y) : 0.f;
      }
    };
    // piece p is of row p * RPP + row_in, i.e. of the key that lane row % 32 holds
    // in its entry row / 32 (row_in < RPP <= 16)
    int32_t s[NP];
    auto spread_slots = [&]() {
#pragma unroll
      for (int p = 0; p < NP; ++p)
        s[p] = __shfl_sync(0xffffffffu, slot[(p * RPP) >> 5], ((p * RPP) & 31) + row_in);
    };
    auto load_pieces = [&]() {
#pragma unroll
      for (int p = 0; p < NP; ++p)
        v[p] = ld_pool<DECODE>(
            reinterpret_cast<const uint4*>(src + uint64_t(uint32_t(s[p])) * D));
    };
    load_slots(0);
    load_scales(0);
    spread_slots();
    load_pieces();
    load_slots(1);
    float vref = 0.f;
#pragma unroll 1
    for (int j = 0; j < n_tiles; ++j) {
      // vref as the K loader has it, and this tile's quotients
      float vm = 0.f;
#pragma unroll
      for (int e = 0; e < SPL; ++e) vm = fmaxf(vm, sc[e]);
      vm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vm)));
      if (vm > vref) vref = 4.f * vm;
      const float inv = 1.f / vref;
      uint32_t f[NP];
      {
        uint32_t fl[SPL];
#pragma unroll
        for (int e = 0; e < SPL; ++e) {
          fl[e] = pack_f16(sc[e] * inv, sc[e] * inv);
        }
#pragma unroll
        for (int p = 0; p < NP; ++p)
          f[p] = __shfl_sync(0xffffffffu, fl[(p * RPP) >> 5], ((p * RPP) & 31) + row_in);
      }
      load_scales(j + 1);
      // the stage is free once P V_{j-NV} completed
      if (!__all_sync(0xffffffffu, j < NV || wait(BAR_O(j), j / 2 - 1, abort_flag))) break;
      const uint32_t stage = uint32_t((j % NV) * Lo::V_BYTES);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          to_f16x4(w[e], h[2 * e], h[2 * e + 1]);
          h[2 * e] = mul_f16x2(h[2 * e], f[p]);
          h[2 * e + 1] = mul_f16x2(h[2 * e + 1], f[p]);
        }
        *reinterpret_cast<uint4*>(at0 + stage + p * RPP * 128) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(at1 + stage + p * RPP * 128) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      // the next tile's codes, and the slots of the one after it
      spread_slots();
      load_pieces();
      load_slots(j + 2);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(BAR_VF(j));
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;\n");
    // ------------------------------------------------------------ softmax
    constexpr int HALF = BN / 2;
    const bool valid = i < t.n_rows;
    int lim = t.key_end;
    if (valid && !DECODE) lim = t.prefix + (t.gr0 + i) / a.group + 1;
    const uint32_t tl = tmem + (uint32_t((warp & 3) * 32) << 16);
    // The row's scale: 2^e with q 2^-e at most 448 (limited below, where the
    // scores vanish anyway).  A query that is not finite has no defined
    // scores: its row is NaN.
    const float qmax = fmaxf(xch[i], xch[BM + i]);
    const int qe = max(kv8::scale_exponent(qmax), -80);
    const float rs =
        qmax < INFINITY ? kv8::pow2(min(qe + a.scale_exp + kKeyShift, 127)) : NAN;
    {
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
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(BAR_Q);
    }
    // a warp without query rows only keeps the barriers going
    const bool busy = (warp & 3) * 32 < t.n_rows;
    // the first tile's exchange slot is parity 1: the Q maxima lie in parity 0
    float nm = INFINITY, vref = 0.f;  // 6 - the row's reference
    float l = 0.f;                    // times 2^6
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < n_tiles; ++j) {
      if (!__all_sync(0xffffffffu, wait(BAR_S(j), j / NS, abort_flag))) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const uint32_t s_col = tl + uint32_t((j % NS) * BN);
      const int k0 = t.key_begin + j * BN + wg * HALF;
      float x[HALF];
      float mx_half = -INFINITY;
      const float v_new = vref_ring[j % SR];
      if (busy) {
        uint32_t sr[HALF];
        tc::tmem_ld_row<HALF>(s_col + uint32_t(wg * HALF), sr);
        const float4* ks4 = reinterpret_cast<const float4*>(ks_ring + (j % SR) * BN + wg * HALF);
        float4 kp[4];  // the first scales, read while S is on its way
#pragma unroll
        for (int e = 0; e < 4; ++e) kp[e] = ks4[e];
        tc::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < HALF; e += 4) {
          const float4 k4 = e < 16 ? kp[(e >> 2) & 3] : ks4[e >> 2];
          const float2 y0 = mul2(make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])),
                                 make_float2(k4.x, k4.y));
          const float2 y1 =
              mul2(make_float2(__uint_as_float(sr[e + 2]), __uint_as_float(sr[e + 3])),
                   make_float2(k4.z, k4.w));
          x[e] = y0.x;
          x[e + 1] = y0.y;
          x[e + 2] = y1.x;
          x[e + 3] = y1.y;
        }
        if (k0 + HALF > t.nomask_end) {
          const int n = lim - k0;  // visible keys of this half
#pragma unroll
          for (int e = 0; e < HALF; ++e)
            if (e >= n) x[e] = -INFINITY;
        }
        float mx4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) mx4[u] = max3(x[3 * u], x[3 * u + 1], x[3 * u + 2]);
#pragma unroll
        for (int e = 12; e < HALF; e += 2)
          mx4[(e >> 1) & 3] = max3(mx4[(e >> 1) & 3], x[e], x[e + 1]);
        mx_half = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
      }
      // the other half's max of this row (double-buffered by tile parity: a
      // thread writes tile j + 2's slot only after every thread has passed
      // tile j + 1's exchange, hence has read tile j's)
      const int xp = (j + 1) & 1;
      xch[(xp * 2 + wg) * BM + i] = mx_half;
      tc::mbar_arrive(XB(j));
      if (!__all_sync(0xffffffffu, wait(XB(j), j >> 1, abort_flag))) {
        ok = false;
        break;
      }
      const float mx = rs * fmaxf(mx_half, xch[(xp * 2 + (1 - wg)) * BM + i]);
      // the reference moves when a weight would exceed 2^15
      const float nm_new = mx + nm > kMaxWeight ? kWeightBias - mx : nm;
      if (j > 0 && __any_sync(0xffffffffu, nm_new != nm || v_new != vref)) {
        // O is rescaled once P V_{j-1} has written it; each warpgroup takes
        // half of its columns
        if (!__all_sync(0xffffffffu, wait(BAR_O(j - 1), (j - 1) >> 1, abort_flag))) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const float alpha = nm_new != nm ? rxk::fast_exp2(nm_new - nm) : 1.f;  // 0 from inf
        const float f = alpha * (vref / v_new);
#pragma unroll 1
        for (int cc = 0; cc < D / 64; ++cc) {
          uint32_t r[32];
          const uint32_t col = tl + uint32_t(Lo::O_COL + wg * (D / 2) + cc * 32);
          tc::tmem_ld32(col, r);
          tc::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
          tc::tmem_st32(col, r);
        }
        l *= alpha;
      }
      nm = nm_new;
      vref = v_new;
      if (busy) {
        const float add = nm == INFINITY ? 0.f : nm;
        const float2 rs2 = make_float2(rs, rs), nm2 = make_float2(add, add);
        float2 l2[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) l2[u] = make_float2(u ? 0.f : l, 0.f);
#pragma unroll
        for (int cc = 0; cc < HALF / 32; ++cc) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const int n = cc * 32 + e;
            const float2 y = fma2(make_float2(x[n], x[n + 1]), rs2, nm2);
            const float2 p = make_float2(rxk::fast_exp2(y.x), rxk::fast_exp2(y.y));
            l2[(e >> 1) & 3] = add2(l2[(e >> 1) & 3], p);
            pk[e >> 1] = pack_f16(p.x, p.y);
          }
          // two keys per column over the first BN / 2 columns of S_j's buffer
          tmem_st16x(s_col + uint32_t(wg * (HALF / 2) + 16 * cc), pk);
        }
        const float2 ls = add2(add2(l2[0], l2[1]), add2(l2[2], l2[3]));
        l = ls.x + ls.y;
      }
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(BAR_P(j));
    }
    // ----------------------------------------------------------- epilogue
    if (DECODE && a.chained) rxk::griddep_wait();
    const bool fin = ok && n_tiles > 0 && __all_sync(0xffffffffu, wait(BAR_FIN, 0, abort_flag));
    // the row sums go through the parity that the last tile did not use
    const int xp = n_tiles & 1 ? 0 : 1;
    if (fin) xch[(xp * 2 + wg) * BM + i] = l;
    tc::mbar_arrive(XE);
    const bool xok = __all_sync(0xffffffffu, wait(XE, 0, abort_flag));
    if (fin && xok) {
      tc::tc_fence_after();
      const float l_all = l + xch[(xp * 2 + (1 - wg)) * BM + i];
      // (2^6 in both O and l; a part whose keys a row does not see leaves zeros)
      const float inv = SPLIT && l_all == 0.f ? 0.f : vref / l_all;
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
      int64_t q_row, out_row = -1;
      if (valid && parts == 1) row_info8<DECODE>(a, t, kvh, i, q_row, out_row, lim);
      const long long my_row = out_row;  // (-1: stays in shared memory)
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
      const float lse = SPLIT && l_all == 0.f ? -INFINITY : logf(l_all) - nm * kLn2;
      if (SPLIT && parts > 1) {
        if (wg == 0) ks_ring[i] = lse;  // (the scales are done with)
      } else if (valid && wg == 0) {
        (DECODE ? a.ws_lse : a.lse)[out_row] = lse;
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) atomicOr(&g_kv8_att_error, 2);
  if constexpr (SPLIT) {
    if (parts > 1) {
      // each CTA of the cluster joins 128 / C rows of all parts
      if (DECODE && a.chained) rxk::griddep_wait();
      cluster_sync();
      constexpr int HC = D / 2, PITCH = HC * 4 + 16;
      const int per = BM / cluster_size();
      for (int idx = tid; idx < per * (D / 4); idx += kTileThreads) {
        const int row = rank * per + idx / (D / 4), col = idx % (D / 4) * 4;
        if (row >= t.n_rows) break;
        const uint32_t at = base + uint32_t(col / HC * (BM * PITCH) + row * PITCH + col % HC * 4);
        const uint32_t lse_at = base + uint32_t(Lo::KS + row * 4);
        float m = -INFINITY;
        for (int p = 0; p < parts; ++p) m = fmaxf(m, ld_peer(peer_addr(lse_at, p)));
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 4
        for (int p = 0; p < parts; ++p) {
          const float li = ld_peer(peer_addr(lse_at, p));
          const float4 v = ld_peer4(peer_addr(at, p));
          const float w = li == -INFINITY ? 0.f : rxk::fast_exp2((li - m) * kLog2e);
          sum += w;
          y.x += w * v.x;
          y.y += w * v.y;
          y.z += w * v.z;
          y.w += w * v.w;
        }
        const float inv = 1.f / sum;
        y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
        int64_t q_row, out_row;
        int lim;
        row_info8<DECODE>(a, t, kvh, row, q_row, out_row, lim);
        if (!DECODE && a.out_bf16)
          *reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + out_row * D + col) =
              make_uint2(rxk::pack_bf16(y.x, y.y), rxk::pack_bf16(y.z, y.w));
        else
          *reinterpret_cast<float4*>((DECODE ? a.ws_o : static_cast<float*>(a.out)) +
                                     out_row * D + col) = y;
        if (col == 0) (DECODE ? a.ws_lse : a.lse)[out_row] = m + logf(sum);
      }
      __syncwarp();
      cluster_sync();  // no CTA leaves while another reads its rows
    }
  }
  if (warp == 12) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

}  // namespace
