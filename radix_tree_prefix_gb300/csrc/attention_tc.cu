// S6-S8: extend and decode attention on the 5th-generation tensor cores
// (tcgen05, TMEM), plus the warp role that decode adds for work items of few
// query rows; decode runs both in one launch per step (decode_fused_kernel).
//
// What is computed ("SGLang: Structured LLM Programs for Efficient
// Inference", sections "A quick recap of how an LLM generates text" and "How
// RadixAttention reuses past work"): every suffix query attends with softmax
// over its request's keys up to and including itself; reused prefix keys are
// read from the slots the radix cache handed out, as if just computed.
//
// One tile = 128 query rows that read one KV head over one key range:
//   extend: rows = (suffix token, head in group) of one request, token-major,
//           causal limit per row = prefix + token + 1;
//   decode: rows = (member request, head in group) of a tree segment chunk
//           shared by the members; writes partial (o, lse) per row.
// The tile (tc_tile3, 384 threads) streams K and V tiles of 32 KB (128 keys
// at head_dim 128, 64 at head_dim 256):
//   warps 0-7  softmax in two warpgroups that split every key tile's keys;
//              thread (w, i) owns query row i = TMEM lane i; the two halves
//              of a row agree on its max through shared memory; P (bf16)
//              goes into TMEM over the S tile it came from; O is rescaled in
//              TMEM when the max grows by more than 2^8 (rare after the
//              first tile); then the output is written;
//   warp 8     allocates TMEM and issues S_j = Q K_j^T (tcgen05.mma from
//              one thread) into a ring of three TMEM buffers, ahead of the
//              softmax;
//   warp 11    issues O += P_j V_j with P_j read from TMEM (O stays in TMEM
//              for the whole key loop);
//   warps 9-10 load K and V into 128-byte swizzled shared memory (three and
//              two stages): a tile whose slots form one contiguous run (the
//              allocator hands out runs, so this is the common case) is one
//              TMA box load per 64 columns; any other tile, and the ragged
//              last tile, is gathered slot by slot with 16-byte cp.async
//              (rows past the key range are zero-filled).
// Every mbarrier wait is bounded (about 2 s); on a timeout the CTA sets an
// error bit, drains its tensor-core work and frees TMEM before returning.

#include "attention_tile.cuh"

namespace {

// Tensor-core tile: 128 query rows, key tiles of BN = 128 keys at head_dim
// 128 and 64 at head_dim 256 (a K or V tile is 32 KB either way), 384
// threads.  The MMA warps keep S tiles ahead of the softmax: S_{j+2} =
// Q K_{j+2}^T is issued before PV_j, into a ring of three S buffers in TMEM,
// so the softmax of tile j+1 never waits for an MMA.  P_j (bf16, two keys per
// column) overwrites the first BN/2 columns of S_j's buffer once the softmax
// has read S_j, and PV_j reads it from TMEM as its A operand; the S issuer
// waits for PV_j's completion (barrier pf) before S_{j+3} reuses that
// buffer.
// TMEM: S ring [0, 3 BN), O from column O_COL (D columns).  Shared memory: Q
// (128-byte swizzled, the A operand of S), K in three stages, V in two.
// Warps 0-7 softmax in two warpgroups that split each key tile's columns
// (thread (w, i) of warpgroup w: row i = TMEM lane i, keys [w BN/2, (w+1)
// BN/2); it also gathers half of Q row i first), warp 8 issues the S MMAs
// and warp 11 the PV MMAs (two instruction streams: one thread issuing all
// of a key tile's MMAs set the tile's period), warp 9 loads K and warp 10
// loads V (a V stage frees only when PV of its previous tile completes, and
// K loads must not queue behind that).
// 12 warps: 0-7 softmax (two warpgroups), 8 S = Q K^T issue, 9 K loader, 10 V
// loader, 11 O += P V issue
constexpr int kThreads3 = 384;

template <int HEAD_DIM>
struct Layout3 {
  static constexpr int D = HEAD_DIM;
  static constexpr int BN = D == 128 ? 128 : 64;
  static constexpr int KSTAGES = 3, VSTAGES = 2, SBUF = 3;
  static constexpr int KV_BYTES = BN * D * 2;
  static constexpr int Q = 0;
  static constexpr int K0 = Q + BM * D * 2;
  static constexpr int V0 = K0 + KSTAGES * KV_BYTES;
  // exchange slots: per-tile half-row maxima, two parities, [2][2
  // warpgroups][128 rows] floats; the final row sums reuse the parity that
  // follows the last tile
  static constexpr int XCH = V0 + VSTAGES * KV_BYTES;
  static constexpr int BAR = XCH + 2 * 2 * 128 * 4;
  // barriers: q, kfull, vfull (one per stage), s[3], p[3], o[2] (PV of even
  // / odd tiles), final, max exchange[2], sum exchange, pf[3] (PV of the P
  // in S buffer b done, so S may overwrite it).  A K stage is free
  // again when the S product that read it completes (s[] of the same index:
  // both rings have three entries) and a V stage when its PV product does
  // (o[] of the same parity: two V stages).
  static constexpr int NBAR = 1 + KSTAGES + VSTAGES + 2 * SBUF + 6 + SBUF;
  static_assert(KSTAGES == SBUF && VSTAGES == 2, "stage rings share the MMA barriers");
  static constexpr int MISC = BAR + NBAR * 8;  // tmem address, abort flag
  // At head_dim 128 the layout carries 1024 bytes of slack to align the
  // swizzled tiles.  At head_dim 256 it leaves under 1 KB of the 227 KB a CTA
  // may have, so the tile requires dynamic shared memory that starts on a
  // 1024-byte boundary: a CTA that finds otherwise sets an error bit and
  // returns without touching anything.
  static constexpr bool SLACK = D == 128;
  static constexpr int BYTES = MISC + 16 + (SLACK ? 1024 : 0);
  static constexpr int TMEM_COLS = 512;
  static constexpr int O_COL = D == 128 ? SBUF * BN : 256;
  static_assert(SBUF * BN <= O_COL && O_COL + D <= TMEM_COLS, "TMEM budget");
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
};

template <int D, bool DECODE>
__device__ __forceinline__ void tc_tile3(const TcArgs& a, const CUtensorMap* tmk,
                                         const CUtensorMap* tmv, uint8_t* smem_raw, int bx,
                                         int kvh) {
  using Lo = Layout3<D>;
  constexpr int BN = Lo::BN, NK = Lo::KSTAGES, NV = Lo::VSTAGES, NB = Lo::SBUF;
  const uint32_t raw = rxk::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // 1024-byte alignment of the swizzled tiles
  if constexpr (!Lo::SLACK) {
    if (base != raw) {  // uniform over the CTA: nothing initialised yet
      if (threadIdx.x == 0) atomicOr(&g_tc_error, 4);
      return;
    }
  }
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base + Lo::Q;
  const uint32_t bar = base + Lo::BAR;
  const uint32_t BAR_Q = bar;
  // barrier indices: q, kfull[NK], vfull[NV], s[NB], p[NB], o[2], final,
  // max exchange[2], sum exchange
  auto BAR_KF = [&](int s) { return bar + 8u * (1 + s); };
  auto BAR_VF = [&](int s) { return bar + 8u * (1 + NK + s); };
  auto BAR_S = [&](int b) { return bar + 8u * (1 + NK + NV + b); };
  auto BAR_P = [&](int b) { return bar + 8u * (1 + NK + NV + NB + b); };
  constexpr uint32_t kAfterP = 1 + NK + NV + 2 * NB;
  // PV_j completes phase j / 2 of BAR_O(j % 2).  One barrier per parity of
  // j: when the softmax of tile j waits for PV_{j-1}, PV_{j-3} has completed
  // (it was issued before S_j, whose completion the softmax waited for), so the
  // phase parity it waits on cannot be mistaken for an older phase; with a
  // single barrier PV_{j-2} may still be in flight and the parity would be
  // ambiguous.
  auto BAR_O = [&](int p) { return bar + 8u * (kAfterP + p); };
  const uint32_t BAR_FIN = bar + 8u * (kAfterP + 2);
  auto XB = [&](int p) { return bar + 8u * (kAfterP + 3 + p); };
  const uint32_t XE = bar + 8u * (kAfterP + 5);
  // PV_j completes phase j / NB of BAR_PF(j % NB): S buffer j % NB is free
  // for S_{j+NB}
  auto BAR_PF = [&](int b) { return bar + 8u * (kAfterP + 6 + b); };
  static_assert(kAfterP + 6 + NB == Lo::NBAR, "barrier count");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Lo::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + Lo::MISC + 4);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const TileDesc t = describe<DECODE, false>(a, bx);
  const int n_tiles = (t.key_end - t.key_begin + BN - 1) / BN;
  // Softmax threads: the query row of their TMEM lane, and the gather of
  // half of Q row i, issued before the barriers and TMEM are set up so the
  // copies overlap that start-up (nothing else uses the Q buffer yet; the
  // arrival on the Q barrier follows the CTA-wide sync below).
  const int wg = warp >> 2;
  const int i = (warp & 3) * 32 + lane;  // TMEM lane
  // the tile row in lane i: row i, or with M = 64 products (at most 64
  // rows) row 16 (i / 32) + i % 16 in the first 16 lanes of each quadrant
  const bool m64 = t.n_rows <= 64;
  const int row = m64 ? (((i >> 5) << 4) | (i & 15)) : i;
  int64_t qi = 0, part = 0;
  int head = 0, lim = t.key_end;
  bool valid = false;
  if (warp < 8) {
    valid = (!m64 || (i & 16) == 0) && row < t.n_rows;
    if (valid) row_info<DECODE>(a, t, kvh, row, qi, head, part, lim);
    // the Q row this thread gathers: tile row i into shared-memory row i
    // (the A operand's rows, whatever the TMEM layout of the products)
    int64_t gqi = qi;
    int ghead = head;
    bool gvalid = valid;
    if (m64) {
      int64_t gpart = 0;
      int glim = 0;
      gqi = 0;
      ghead = 0;
      gvalid = i < t.n_rows;
      if (gvalid) row_info<DECODE>(a, t, kvh, i, gqi, ghead, gpart, glim);
    }
    // the queries (and, below, the outputs: decode's partial buffers the
    // previous merge read) are touched only once earlier kernels on the
    // stream are done; with early inputs the queries are complete already
    // and only the partial writes wait
    if (!DECODE || !a.early_inputs) rxk::griddep_wait();
    // chunks [8 w, 8 w + 8) of Q row i (zeros past the tile's rows) while
    // the loader warps already stream the first K/V tiles
    const bf16* src = a.q + (gqi * a.hq + ghead) * D;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const int ch = wg * (D / 16) + c;
      rxk::cp_async_16(sw128(sQ, BM, i, ch), src + ch * 8, gvalid);
    }
    rxk::cp_async_commit();
  }

  if (tid == 0) {
    tc::mbar_init(BAR_Q, 8 * 32);  // every softmax thread lands half a Q row
    for (int s = 0; s < NK; ++s) tc::mbar_init(BAR_KF(s), 1);
    for (int s = 0; s < NV; ++s) tc::mbar_init(BAR_VF(s), 1);
    for (int b = 0; b < NB; ++b) {
      tc::mbar_init(BAR_S(b), 1);
      tc::mbar_init(BAR_P(b), 8 * 32);
    }
    tc::mbar_init(XB(0), 8 * 32);
    tc::mbar_init(XB(1), 8 * 32);
    tc::mbar_init(XE, 8 * 32);
    tc::mbar_init(BAR_O(0), 1);
    tc::mbar_init(BAR_O(1), 1);
    tc::mbar_init(BAR_FIN, 2);  // one commit per issuing thread
    for (int b = 0; b < NB; ++b) tc::mbar_init(BAR_PF(b), 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 8) {
    tc::tmem_alloc(rxk::smem_addr(tmem_slot), Lo::TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 9 || warp == 10) {
    // ------------------------------------------------------------- loaders
    const bool load_v = warp == 10;
    // keys written by earlier kernels on the stream are read from here on
    // (a decode step after the first of a run reads shared segments that no
    // kernel of the run writes: it need not wait)
    if (!DECODE || !a.early_inputs) rxk::griddep_wait();
    constexpr int CPR = D / 8;
    constexpr int SPL = BN / 32;  // slots per lane: rows lane + 32 i
    const bf16* kb = a.kpool + int64_t(kvh) * a.head_stride;
    const bf16* vb = a.vpool + int64_t(kvh) * a.head_stride;
    const int64_t row0 = a.tma_row_base + int64_t(kvh) * a.tma_head_rows;
    // slots of four consecutive tiles (tile j in ring j % 4): a tile's table
    // reads are issued four tiles ahead into registers that nothing touches
    // until then, so their round trips to L2 overlap the loads before them
    int32_t sa[SPL], sb[SPL], sc[SPL], sd[SPL];
    auto load_slots = [&](int j, int32_t (&dst)[SPL]) {
      const int k0 = t.key_begin + j * BN;
#pragma unroll
      for (int i = 0; i < SPL; ++i) {
        const int key = k0 + lane + 32 * i;
        dst[i] = (j < n_tiles && key < t.key_end) ? __ldg(t.trow + key) : -1;
      }
    };
    auto check_slots = [&](int32_t (&slot)[SPL]) {
#pragma unroll
      for (int i = 0; i < SPL; ++i) {
        if (slot[i] >= a.num_slots || slot[i] < -1) {
          atomicOr(&g_tc_error, 1);
          slot[i] = 0;
        }
      }
    };
    // one K or V tile: TMA box loads if the slots are one contiguous run of
    // BN valid slots, else a zero-filling cp.async gather
    auto load_tile = [&](int32_t (&slot)[SPL], const CUtensorMap* tm, const bf16* src_base,
                         uint32_t dst, uint32_t full_bar) {
      const int32_t first = __shfl_sync(0xffffffffu, slot[0], 0);
      bool run = first >= 0 && int64_t(first) + BN <= a.num_slots;
#pragma unroll
      for (int i = 0; i < SPL; ++i) run = run && (slot[i] == first + lane + 32 * i);
      run = __all_sync(0xffffffffu, run);
      if (run) {
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(full_bar, uint32_t(BN * D * 2));
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb)
            tc::tma_load_2d(dst + uint32_t(cb * BN * 128), tm, cb * 64, int(row0 + first),
                            full_bar);
        }
      } else {
        // lanes 0-15 and 16-31 copy chunks (lane % 16) + 16 h of rows 2k, 2k+1
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
#pragma unroll 4
          for (int k = 0; k < 16; ++k) {
            const int row = 32 * i + 2 * k + (lane >> 4);
            const int32_t sl = __shfl_sync(0xffffffffu, slot[i], row & 31);
            const bool ok = sl >= 0;
            const int64_t s64 = ok ? int64_t(sl) : 0;
#pragma unroll
            for (int h = 0; h < CPR / 16; ++h) {
              const int ch = (lane & 15) + 16 * h;
              rxk::cp_async_16(sw128(dst, BN, row, ch), src_base + s64 * D + ch * 8, ok);
            }
          }
        }
        rxk::cp_async_commit();
        rxk::cp_async_wait<0>();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(full_bar);
      }
    };
    load_slots(0, sa);
    load_slots(1, sb);
    load_slots(2, sc);
    load_slots(3, sd);
    // tile j (K stage j % NK, V stage j % NV): K and V with the slots in
    // `slot`, then tile j + 4's table reads into the same registers; a stage
    // is refilled once the MMA that read its previous tile has completed:
    // S_{j-NK} (barrier s[j % NK]) for K, PV_{j-2} (barrier o[j % 2]) for V
    int issued = 0;  // tiles whose K (or V) load has been issued
    auto step = [&](int j, int32_t (&slot)[SPL]) -> bool {
      const int sk = j % NK, sv = j % NV;
      check_slots(slot);
      if (!load_v) {
        if (j >= NK &&
            !__all_sync(0xffffffffu, tc::mbar_wait(BAR_S(sk), uint32_t(j / NK - 1) & 1u,
                                                    abort_flag, kWaitLimit, kSleepNs)))
          return false;
        load_tile(slot, tmk, kb, base + Lo::K0 + sk * Lo::KV_BYTES, BAR_KF(sk));
      } else {
        if (j >= NV &&
            !__all_sync(0xffffffffu, tc::mbar_wait(BAR_O(sv), uint32_t(j / NV - 1) & 1u,
                                                    abort_flag, kWaitLimit, kSleepNs)))
          return false;
        load_tile(slot, tmv, vb, base + Lo::V0 + sv * Lo::KV_BYTES, BAR_VF(sv));
      }
      issued = j + 1;
      load_slots(j + 4, slot);
      return true;
    };
    for (int j = 0; j < n_tiles; j += 4) {
      if (!step(j, sa)) break;
      if (j + 1 < n_tiles && !step(j + 1, sb)) break;
      if (j + 2 < n_tiles && !step(j + 2, sc)) break;
      if (j + 3 < n_tiles && !step(j + 3, sd)) break;
    }
    // Before the CTA gives up its shared memory, the last load of every
    // stage has landed.  On the normal path the MMAs consumed them all and
    // these waits return at once; after a wait of another warp timed out
    // (abort), TMA box loads may still be in flight, so they get one more
    // bounded wait that does not look at the abort flag.
    if (lane == 0) {
      const int NS = load_v ? NV : NK;
      int drain_abort = 0;
      for (int j = issued > NS ? issued - NS : 0; j < issued; ++j) {
        const uint32_t fb = load_v ? BAR_VF(j % NV) : BAR_KF(j % NK);
        tc::mbar_wait(fb, uint32_t(j / NS) & 1u, &drain_abort, kWaitLimit);
      }
    }
    __syncwarp();
  } else if (warp == 8 || warp == 11) {
    // ------------------------------------------------------------ MMA issue
    // Two issuing threads, so neither instruction stream alone sets the key
    // tile's period: warp 8 issues S_j = Q K_j^T into S buffer j % 3, warp 11
    // issues O += P_j V_j with P_j from TMEM.  The two streams no longer
    // complete in one order, so the S issuer waits, before S_j, until PV_{j-3}
    // (which read P_{j-3} from the same buffer) has completed (barrier pf[j %
    // 3]); hence S_j completing still implies PV_{j-3} completed, which the
    // softmax's wait on o[] relies on.
    if (lane == 0) {
      // a tile of at most 64 rows runs M = 64 products (half the MMA work;
      // its row r then sits in TMEM lane 32 (r / 16) + r % 16)
      const bool m64 = t.n_rows <= 64;
      const uint32_t IDESC_S = m64 ? tc::idesc_bf16(64, BN, 0) : tc::idesc_bf16(BM, BN, 0);
      const uint32_t IDESC_PV = m64 ? tc::idesc_bf16(64, D, 1) : tc::idesc_bf16(BM, D, 1);
      // shared-memory descriptors (128-byte swizzle, 1024 bytes between
      // 8-row groups): common high half; low halves of Q, K stage 0 (K-major,
      // leading offset 16 B) and V stage 0 (MN-major, leading offset = one
      // 64-column block of BN rows).  Fields of the 64-bit descriptor: start
      // address >> 4 in bits 0-13, leading byte offset >> 4 in bits 16-29,
      // stride byte offset >> 4 in bits 32-45, version 1 at bit 46, layout
      // (2 = 128-byte swizzle) in bits 61-63; swizzle atoms (8 rows x 128 B)
      // start on 1024-byte boundaries
      constexpr uint32_t DHI = (1024u >> 4) | (1u << 14) | (2u << 29);
      constexpr uint32_t KV_STEP = uint32_t(Lo::KV_BYTES) >> 4;
      static_assert(Lo::V0 + NV * Lo::KV_BYTES < (1 << 18), "descriptor address field");
      if (warp == 8) {
        const uint32_t q_lo = ((sQ & 0x3FFFFu) >> 4) | (1u << 16);
        const uint32_t k_lo0 = (((base + Lo::K0) & 0x3FFFFu) >> 4) | (1u << 16);
        const bool ok = tc::mbar_wait(BAR_Q, 0, abort_flag, kWaitLimit, kSleepNs);
        // S_j's K stage and S buffer (the same index: both rings have NB
        // entries) and the phases of its waits
        int sb = 0;
        uint32_t k_phase = 0, pf_phase = 0;
        for (int j = 0; ok && j < n_tiles; ++j) {
          if (j >= NB && !tc::mbar_wait(BAR_PF(sb), pf_phase, abort_flag, kWaitLimit, kSleepNs))
            break;
          if (!tc::mbar_wait(BAR_KF(sb), k_phase, abort_flag, kWaitLimit, kSleepNs)) break;
          tc::tc_fence_after();
          const uint32_t k_lo = k_lo0 + uint32_t(sb) * KV_STEP;
          const uint32_t d_s = tmem + uint32_t(sb * BN);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t a_off = uint32_t(((ks >> 2) * (BM * 128) + (ks & 3) * 32) >> 4);
            const uint32_t b_off = uint32_t(((ks >> 2) * (BN * 128) + (ks & 3) * 32) >> 4);
            mma_ss_split(d_s, q_lo + a_off, k_lo + b_off, DHI, IDESC_S, ks > 0 ? 1u : 0u);
          }
          tc::mma_commit(BAR_S(sb));  // also frees K stage sb
          if (++sb == NB) {
            sb = 0;
            k_phase ^= 1u;
            if (j >= NB) pf_phase ^= 1u;
          }
        }
      } else {
        const uint32_t v_lo0 =
            (((base + Lo::V0) & 0x3FFFFu) >> 4) | (uint32_t(BN * 128 / 16) << 16);
        int sv = 0, pb = 0;
        uint32_t v_phase = 0, p_phase = 0;
        for (int j = 0; j < n_tiles; ++j) {
          if (!tc::mbar_wait(BAR_P(pb), p_phase, abort_flag, kWaitLimit, kSleepNs)) break;
          if (!tc::mbar_wait(BAR_VF(sv), v_phase, abort_flag, kWaitLimit, kSleepNs)) break;
          tc::tc_fence_after();
          const uint32_t v_lo = v_lo0 + uint32_t(sv) * KV_STEP;
          const uint32_t p_t = tmem + uint32_t(pb * BN);
#pragma unroll
          for (int ks = 0; ks < BN / 16; ++ks)
            mma_ts_split(tmem + uint32_t(Lo::O_COL), p_t + uint32_t(ks * 8),
                         v_lo + uint32_t(ks * 2048 / 16), DHI, IDESC_PV,
                         (j > 0 || ks > 0) ? 1u : 0u);
          tc::mma_commit(BAR_O(j & 1));  // also frees V stage sv (== j & 1)
          tc::mma_commit(BAR_PF(pb));    // S buffer pb may take S_{j+3}
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
      // drain: every MMA this thread issued has completed once the final
      // barrier (one arrival per issuing thread) completes.  The wait ignores
      // the abort flag (bounded all the same): after another warp gave up,
      // MMAs already issued must finish writing TMEM and reading shared
      // memory before the CTA frees both.
      tc::mma_commit(BAR_FIN);
      int drain_abort = 0;
      tc::mbar_wait(BAR_FIN, 0, &drain_abort, kWaitLimit);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    // Two warpgroups: warpgroup w (warps 4w .. 4w+3) owns keys [64 w, 64 w +
    // 64) of every key tile for the same 128 rows (warp 4w + q reaches TMEM
    // lanes 32 q ..).  Per tile the two halves of a row agree on the row max
    // through shared memory (one bounded mbarrier round), so both write P
    // against the same reference and share one O accumulator.
    constexpr int HALF = BN / 2;
    const uint32_t tl = tmem + (uint32_t((warp & 3) * 32) << 16);
    float* xch = reinterpret_cast<float*>(gbase + Lo::XCH);  // [2][2 warpgroups][BM]
    // the Q gather issued at the start has landed
    rxk::cp_async_wait<0>();
    tc::fence_proxy_async_smem();
    tc::mbar_arrive(BAR_Q);
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      const int s = j % NB;  // S buffer
      // waits are made warp-uniform before any warp-collective tcgen05 op
      if (!__all_sync(0xffffffffu, tc::mbar_wait(BAR_S(s), uint32_t(j / NB) & 1u, abort_flag,
                                                  kWaitLimit))) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const int k0 = t.key_begin + j * BN + wg * HALF;  // first key of this half
      const bool need_mask = k0 + HALF > t.nomask_end;
      uint32_t sr[HALF];
      tc::tmem_ld_row<HALF>(tl + uint32_t(s * BN + wg * HALF), sr);
      tc::tmem_ld_wait();
      // row max of the raw scores over this half (masked keys get a large
      // negative finite score, so no exponent below is an infinity or a NaN,
      // even for a row whose keys are all masked); eight independent partial
      // maxima keep the chains short
      float mx8[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) mx8[u] = kMasked;
      if (need_mask) {
#pragma unroll
        for (int e = 0; e < HALF; ++e) {
          if (k0 + e >= lim) sr[e] = __float_as_uint(kMasked);
          mx8[e & 7] = fmaxf(mx8[e & 7], __uint_as_float(sr[e]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < HALF; ++e) mx8[e & 7] = fmaxf(mx8[e & 7], __uint_as_float(sr[e]));
      }
      const float mx_half = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                  fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
      // the other half's max of this row (parity-double-buffered slot: a thread
      // reaches tile j + 2's write only after every thread has passed tile
      // j + 1's exchange, hence has read tile j's)
      xch[((j & 1) * 2 + wg) * BM + i] = mx_half;
      tc::mbar_arrive(XB(j & 1));
      if (!__all_sync(0xffffffffu, tc::mbar_wait(XB(j & 1), (j >> 1) & 1, abort_flag, kWaitLimit))) {
        ok = false;
        break;
      }
      const float mx_other = xch[((j & 1) * 2 + (1 - wg)) * BM + i];
      const float mx = a.scale_log2 * fmaxf(mx_half, mx_other);
      const float m_new = fmaxf(m_ref, mx);
      if (j == 0) {
        m_ref = m_new;
      } else {
        const bool need = m_new > m_ref + kRescaleThreshold;
        // both warps of a row quadrant see the same rows, so they agree
        if (__any_sync(0xffffffffu, need)) {
          // O is rescaled once PV_{j-1} has written it; each warpgroup takes
          // half of its columns
          if (!__all_sync(0xffffffffu, tc::mbar_wait(BAR_O((j - 1) & 1), ((j - 1) >> 1) & 1,
                                                      abort_flag, kWaitLimit))) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const float alpha = need ? rxk::fast_exp2(m_ref - m_new) : 1.f;
#pragma unroll
          for (int cc = 0; cc < D / 64; ++cc) {
            uint32_t r[32];
            const uint32_t col = uint32_t(Lo::O_COL + wg * (D / 2) + cc * 32);
            tc::tmem_ld32(tl + col, r);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tc::tmem_st32(tl + col, r);
          }
          if (need) {
            l *= alpha;
            m_ref = m_new;
          }
        }
      }
      const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
      float l8[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) l8[u] = 0.f;
#pragma unroll
      for (int cc = 0; cc < HALF / 32; ++cc) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          // p = 2^(scale*s - m) for two keys: exp2 in fp32 on the SFU, then
          // both rounded to nearest into one bf16x2 word (the precision P has
          // in the PV product).  With the lazy max the dominant keys'
          // exponents reach +8, where a bf16 exponent or a bf16 exp2 result
          // would cost up to 1% per weight on peaked rows.  The row sum adds
          // exactly the rounded values in fp32, in eight independent partial
          // sums.
          const float x0 = fmaf(__uint_as_float(sr[cc * 32 + e]), a.scale_log2, -m_use);
          const float x1 = fmaf(__uint_as_float(sr[cc * 32 + e + 1]), a.scale_log2, -m_use);
          const uint32_t h = rxk::pack_bf16(rxk::fast_exp2(x0), rxk::fast_exp2(x1));
          l8[(e >> 1) & 7] += __uint_as_float(h << 16) + __uint_as_float(h & 0xffff0000u);
          pk[e >> 1] = h;
        }
        // keys of this half, two per column, over the first BN/2 columns
        // of S_j's buffer (half w at columns w BN/4 ..)
        tmem_st16(tl + uint32_t(s * BN + wg * (HALF / 2) + 16 * cc), pk);
      }
      l += ((l8[0] + l8[1]) + (l8[2] + l8[3])) + ((l8[4] + l8[5]) + (l8[6] + l8[7]));
      tc::tmem_st_wait();
      tc::tc_fence_before();
      tc::mbar_arrive(BAR_P(s));
    }
    // The epilogue waits on BAR_FIN, which completes exactly once, after every
    // MMA of the CTA, then the halves add
    // their row sums through shared memory and warpgroup w writes output
    // columns [64 w, 64 w + 64).  Every softmax thread arrives on the
    // exchange barrier, so no waiter is left behind when a wait gave up.
    const bool fin = ok && n_tiles > 0 &&
                     __all_sync(0xffffffffu, tc::mbar_wait(BAR_FIN, 0, abort_flag, kWaitLimit));
    if (DECODE && a.early_inputs) rxk::griddep_wait();  // the previous merge read ws
    // (a thread got here after every thread passed the exchange of tile
    // n_tiles - 1, hence had read the slot of tile n_tiles - 2)
    if (fin) xch[((n_tiles & 1) * 2 + wg) * BM + i] = l;
    tc::mbar_arrive(XE);
    const bool xok = __all_sync(0xffffffffu, tc::mbar_wait(XE, 0, abort_flag, kWaitLimit));
    if (fin && xok) {
      tc::tc_fence_after();
      const float l_all = l + xch[((n_tiles & 1) * 2 + (1 - wg)) * BM + i];
      const float inv = l_all > 0.f ? 1.f / l_all : 0.f;
      float* dst;
      float* lse_dst;
      if constexpr (DECODE) {
        dst = a.ws_o + (part * a.hq + head) * D;
        lse_dst = a.ws_lse + part * a.hq + head;
      } else {
        dst = a.out + (qi * a.hq + head) * D;
        lse_dst = a.lse + qi * a.hq + head;
      }
      // Warpgroup w owns output columns [w D/2, (w+1) D/2).  Its rows go
      // through shared memory (the K stages, idle once every MMA completed
      // and every load landed) so that each warp then writes the 32 rows of
      // its TMEM lane quadrant as whole contiguous row segments: one thread
      // per row would make every store instruction touch 32 rows.
      constexpr int HC = D / 2;           // columns per warpgroup
      constexpr int PITCH = HC * 4 + 16;  // staged row bytes (+16: conflict-free)
      constexpr int LPR = HC / 4;         // float4 per staged row
      static_assert(2 * BM * PITCH <= Lo::XCH - Lo::K0, "staging fits in the K/V stages");
      uint8_t* stage = gbase + Lo::K0 + wg * (BM * PITCH);
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
      const int qrow = (warp & 3) * 32;  // first row of this warp's quadrant
      const unsigned long long my_dst =
          valid ? reinterpret_cast<unsigned long long>(dst + wg * HC) : 0ull;
#pragma unroll 4
      for (int k = 0; k < LPR; ++k) {
        const int idx = k * 32 + lane;
        const int rr = idx / LPR, c4 = idx - rr * LPR;  // row within the quadrant, float4
        const unsigned long long rd = __shfl_sync(0xffffffffu, my_dst, rr);
        const float4 v = *reinterpret_cast<const float4*>(stage + (qrow + rr) * PITCH + c4 * 16);
        if (rd) reinterpret_cast<float4*>(rd)[c4] = v;
      }
      if (valid && wg == 0) *lse_dst = m_ref * kLn2 + logf(l_all);
    } else if (DECODE && n_tiles <= 0 && valid) {
      // keys that a later step of the plan brings: an empty partial row
      float4* dst = reinterpret_cast<float4*>(a.ws_o + (part * a.hq + head) * D + wg * (D / 2));
#pragma unroll 1
      for (int c = 0; c < D / 8; ++c) dst[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (wg == 0) a.ws_lse[part * a.hq + head] = -INFINITY;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) atomicOr(&g_tc_error, 2);
  if (warp == 8) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, Lo::TMEM_COLS);
  }
}

// Extend: one tile per CTA, heaviest row tile first.  With heads_interleaved
// (few waves of CTAs, or short contexts) CTA c takes row tile c / Hkv of KV
// head c % Hkv, so the heavy tiles of every head go out before the light
// ones and the last wave is short; otherwise CTA c takes head c / tiles, so
// the CTAs resident at one time read the keys of one head and those stay in
// L2.
template <int D>
__global__ void __launch_bounds__(kThreads3, 1)
    attn_tc3_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int c = int(blockIdx.x);
  if (a.heads_interleaved) {
    const int hkv = a.hq / a.group;
    tc_tile3<D, false>(a, &tmk, &tmv, smem_raw, c / hkv, c - (c / hkv) * hkv);
  } else {
    tc_tile3<D, false>(a, &tmk, &tmv, smem_raw, c % a.num_tiles, c / a.num_tiles);
  }
}

// One launch per decode step, at most one CTA per SM.  CTAs [w, w + n_tc_ctas)
// (w = n_warp_first) first run the tensor-core tile of one segment chunk with
// more than 16 query rows (CTA w + c: item c / Hkv, KV head c % Hkv).  Then
// the first six warps of every CTA take warp-role units (an item of <= 16
// rows and one KV head) from a shared counter, heaviest first, until none is
// left; so the SMs of finished tiles join the warp-role work.  When the tiles
// alone fill more than one wave, the w CTAs before them take warp-role units
// from the start, so the streaming of private tails (bound by HBM) runs
// beside the first wave of tiles (bound by the tensor core and the
// exponentials) instead of after it.  The counter starts at 0 and the merge
// after this kernel resets it.  Launched with programmatic stream
// serialization: the merge that follows may launch early, and this kernel waits
// (griddepcontrol.wait) for the previous kernels on the stream before it
// touches what they wrote or read.
template <int D>
struct Fused {
  static constexpr int THREADS = kThreads3;
  static constexpr int TILE_BYTES = Layout3<D>::BYTES;
  static constexpr int PIPE_BYTES = kPipeWarps * PipeCfg<D>::WARP_BYTES + 1024;
  static constexpr int SMEM = TILE_BYTES > PIPE_BYTES ? TILE_BYTES : PIPE_BYTES;
  static_assert(SMEM <= 227 * 1024, "fused decode CTA fits in shared memory");
};

template <int D>
__global__ void __launch_bounds__(Fused<D>::THREADS, 1)
    decode_fused_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv) {
  using Cfg = PipeCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  rxk::griddep_launch_dependents();
  const int cta = int(blockIdx.x) - a.n_warp_first;
  if (cta >= 0 && cta < a.n_tc_ctas) {
    const int hkv = a.hq / a.group;
    tc_tile3<D, true>(a, &tmk, &tmv, smem_raw, cta / hkv, cta - (cta / hkv) * hkv);
  }
  if (threadIdx.x >= kPipeWarps * 32) return;  // the warp role uses the first six warps
  // tiles_leave: in a run of steps a tile CTA leaves its SM to the next
  // step's tiles, which start there at once (early inputs) while this step's
  // warp-role units still stream on the other SMs
  if (a.tiles_leave && cta >= 0 && cta < a.n_tc_ctas) return;
  rxk::griddep_wait();
  // warp role: this warp's ring and slot buffer
  const uint32_t raw = rxk::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const int warp = int(threadIdx.x >> 5);
  const int lane = int(threadIdx.x & 31);
  const uint32_t ring = base + uint32_t(warp * Cfg::WARP_BYTES);
  int32_t* slot_buf = reinterpret_cast<int32_t*>(smem_raw + (base - raw) + warp * Cfg::WARP_BYTES +
                                                 Cfg::STAGES * Cfg::STAGE_BYTES);  // [2][kSlotBuf]
  uint32_t gstep = 0;
  NextUnit cur, nxt;
  cur.stage = 0;
  while (cur.stage < 3) next_unit_step(a, cur);
  while (cur.idx < a.n_small_units) {
    nxt.stage = 0;
    const int rows = cur.word(6);
    if (rows <= 8) {
      pipe_unit<1, D>(a, ring, slot_buf, gstep, cur, nxt);
    } else if constexpr (D == 128) {
      pipe_unit<2, D>(a, ring, slot_buf, gstep, cur, nxt);
    } else if (lane == 0) {
      atomicOr(&g_tc_error, 1);  // the plan gives head_dim 256 no such item
    }
    while (nxt.stage < 3) next_unit_step(a, nxt);  // short units: the rest now
    cur = nxt;
  }
}

template <int D>
rx_status launch_extend(TcArgs a, const rx_pool_desc* pool, int32_t layer, unsigned gx,
                        unsigned gy, cudaStream_t s) {
  using Lo = Layout3<D>;
  static std::atomic<bool> configured[kMaxDevices];
  const rx_status cs = ensure_smem(configured, attn_tc3_kernel<D>, Lo::BYTES);
  if (cs != RX_OK) return cs;
  const CUtensorMap *tmk, *tmv;
  if (!pool_maps(pool, Lo::BN, &tmk, &tmv))
    return rx_internal::set_error(RX_ERR_CUDA, "could not encode the pool's TMA tensor maps");
  a.tma_row_base = int64_t(layer) * pool->num_kv_heads * pool->num_slots;
  a.tma_head_rows = pool->num_slots;
  attn_tc3_kernel<D><<<dim3(gx * gy), kThreads3, Lo::BYTES, s>>>(a, *tmk, *tmv);
  return rx_internal::launch_status("extend attention (tcgen05)");
}

}  // namespace

namespace rx_internal {

// Looked up once per process (a function-local static is initialised exactly
// once, whichever thread gets there).
void* tensor_map_encoder() {
  static void* const fn = []() -> void* {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return p;
    return nullptr;
  }();
  return fn;
}

int32_t tc_error_flags(bool clear) {
  int32_t v = 0;
  cudaMemcpyFromSymbol(&v, g_tc_error, sizeof(v));
  if (clear && v) {
    int32_t z = 0;
    cudaMemcpyToSymbol(g_tc_error, &z, sizeof(z));
  }
  return v;
}

rx_status decode_fused(const rx_pool_desc* pool, int32_t layer, const void* d_q,
                       int32_t num_q_heads, const int32_t* d_req_to_token, int64_t row_stride,
                       const int32_t* d_work_small, int64_t n_small, const int32_t* d_work_tc,
                       int64_t n_tc, const int32_t* d_members, float scale, float* ws_o,
                       float* ws_lse, int32_t* unit_counter, int step, const void* k_new,
                       const void* v_new, const int32_t* slots_new, cudaStream_t stream,
                       bool early_inputs) {
  const int D = pool->head_dim;
  if (D != 128 && D != 256) return set_error(RX_ERR_INVALID, "decode needs head_dim 128 or 256");
  const int64_t hkv = pool->num_kv_heads;
  const int64_t small_units = n_small * hkv;
  const int64_t tc_ctas = n_tc * hkv;
  // the tiles plus CTAs for the warp-role units: when everything fits in one
  // wave, enough of them for every unit (after the tiles); otherwise up to a
  // quarter of the SMs, placed before the tiles so that they start at once
  const int64_t sms = rx_internal::sm_count();
  const int64_t unit_ctas = (small_units + kPipeWarps - 1) / kPipeWarps;
  int64_t warp_first = 0, ctas = tc_ctas;
  if (tc_ctas + unit_ctas <= sms)
    ctas = tc_ctas + unit_ctas;
  else if (tc_ctas >= sms)
    warp_first = std::min<int64_t>(unit_ctas, (sms + 3) / 4);
  else
    ctas = sms;
  ctas += warp_first;
  if (ctas == 0) return RX_OK;
  if (ctas > INT32_MAX) return set_error(RX_ERR_INVALID, "decode plan too large for one launch");
  TcArgs a{};
  a.q = static_cast<const bf16*>(d_q);
  const int64_t layer_off = int64_t(layer) * hkv * pool->num_slots * D;
  a.kpool = static_cast<const bf16*>(pool->k_pool) + layer_off;
  a.vpool = static_cast<const bf16*>(pool->v_pool) + layer_off;
  a.head_stride = pool->num_slots * D;
  a.num_slots = pool->num_slots;
  a.table = d_req_to_token;
  a.row_stride = row_stride;
  a.hq = num_q_heads;
  a.group = num_q_heads / int(hkv);
  a.scale_log2 = scale * kLog2e;
  a.work = d_work_tc;
  a.members = d_members;
  a.ws_o = ws_o;
  a.ws_lse = ws_lse;
  a.work_small = d_work_small;
  a.n_small_units = int(small_units);
  a.n_tc_ctas = int(tc_ctas);
  a.n_warp_first = int(warp_first);
  a.unit_counter = unit_counter;
  a.early_inputs = early_inputs ? 1 : 0;
  // with three times as many warp-role CTAs as tile CTAs (few, long tiles
  // beside many units), the tiles need not help with the units
  a.tiles_leave = early_inputs && ctas - tc_ctas >= 3 * tc_ctas ? 1 : 0;
  a.step = step;
  a.k_new = static_cast<const bf16*>(k_new);
  a.v_new = static_cast<const bf16*>(v_new);
  a.slots_new = slots_new;
  a.tma_row_base = int64_t(layer) * hkv * pool->num_slots;
  a.tma_head_rows = pool->num_slots;
  static std::atomic<bool> configured128[kMaxDevices], configured256[kMaxDevices];
  const rx_status cs =
      D == 128 ? ensure_smem(configured128, decode_fused_kernel<128>, Fused<128>::SMEM)
               : ensure_smem(configured256, decode_fused_kernel<256>, Fused<256>::SMEM);
  if (cs != RX_OK) return cs;
  const CUtensorMap *tmk, *tmv;
  if (!pool_maps(pool, D == 128 ? 128 : 64, &tmk, &tmv))
    return set_error(RX_ERR_CUDA, "could not encode the pool's TMA tensor maps");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(unsigned(D == 128 ? Fused<128>::THREADS : Fused<256>::THREADS));
  cfg.dynamicSmemBytes = D == 128 ? Fused<128>::SMEM : Fused<256>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (D == 128)
    cudaLaunchKernelEx(&cfg, decode_fused_kernel<128>, a, *tmk, *tmv);
  else
    cudaLaunchKernelEx(&cfg, decode_fused_kernel<256>, a, *tmk, *tmv);
  return launch_status("decode attention (fused)");
}

rx_status extend_attention_tc(const rx_pool_desc* pool, int32_t layer, const void* d_q,
                              int32_t num_q_heads, const int32_t* d_req_to_token,
                              int64_t row_stride, const int32_t* d_req_rows,
                              const int32_t* d_prefix_len, const int32_t* d_qo_indptr,
                              const int32_t* d_tile_indptr, int32_t R, int64_t num_tiles,
                              float scale, float* d_out, float* d_lse, cudaStream_t stream) {
  const int D = pool->head_dim;
  TcArgs a{};
  a.q = static_cast<const bf16*>(d_q);
  const int64_t layer_off = int64_t(layer) * pool->num_kv_heads * pool->num_slots * D;
  a.kpool = static_cast<const bf16*>(pool->k_pool) + layer_off;
  a.vpool = static_cast<const bf16*>(pool->v_pool) + layer_off;
  a.head_stride = pool->num_slots * D;
  a.num_slots = pool->num_slots;
  a.table = d_req_to_token;
  a.row_stride = row_stride;
  a.hq = num_q_heads;
  a.group = num_q_heads / pool->num_kv_heads;
  a.scale_log2 = scale * kLog2e;
  a.req_rows = d_req_rows;
  a.prefix_len = d_prefix_len;
  a.qo_indptr = d_qo_indptr;
  a.tile_indptr = d_tile_indptr;
  a.num_req = R;
  a.num_tiles = int(num_tiles);
  // heads interleaved (the heavy row tiles of every head first, a short
  // tail) for up to kExtendInterleaveWaves waves of CTAs, or when a
  // request's keys over all heads are small enough to stay in L2 while its
  // row tiles run (row_stride bounds a request's keys); otherwise
  // head-major, so the CTAs in flight read one head's long key ranges
  const int64_t kv_row_bytes = row_stride * pool->num_kv_heads * int64_t(D) * 4;
  a.heads_interleaved =
      num_tiles * pool->num_kv_heads <= int64_t(kExtendInterleaveWaves) * rx_internal::sm_count() ||
      kv_row_bytes <= kExtendInterleaveKvBytes;
  a.out = d_out;
  a.lse = d_lse;
  if (D == 128)
    return launch_extend<128>(a, pool, layer, unsigned(num_tiles), pool->num_kv_heads, stream);
  return launch_extend<256>(a, pool, layer, unsigned(num_tiles), pool->num_kv_heads, stream);
}

}  // namespace rx_internal
