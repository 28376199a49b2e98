// Extend and decode attention over the 8-bit KV pool (e4m3 codes, one scale
// for each KV head and block of slots), and the merge of decode partials.
//
// What is computed, for a query q and the keys j it sees, key j = ks_j kc_j
// and value j = vs_j vc_j (codes kc, vc; scales ks, vs of the block of key
// j's slot):
//   x_j = scale * ks_j * (q . kc_j),  p_j = exp(x_j - m),  l = sum_j p_j,
//   o = sum_j (p_j vs_j) vc_j / l,    lse = m + log l.
// ks_j multiplies a score.  vs_j joins the weight or the value, as a quotient
// by a reference vref that is at least the largest vs so far; the result is
// scaled back at the end.
//
// Extend, and decode items of more query rows than one warp takes, run on the
// tensor-core tile of kv8_tile.cuh; decode items of few rows (a request's own
// tail) on warps that stream the keys (stream_unit below).  Statistics, scores
// and accumulators are fp32.  What is rounded further:
//   q        tile, two e4m3 parts: exact from 2^-9.8 of its row's largest
//            magnitude, to 2^-17.8 of that below; streams, f16: exact from
//            2^-30 of it, to 2^-38 below;
//   weights  to f16, 11 bits, and to 2^-31 of the reference's below 2^-20 of it:
//            p_j in the tile, p_j vs_j / vref in the streams;
//   values   in the tile vs_j / vref and its product with a code are f16.  For
//            the power-of-two scales that rx_kv8_store writes that is exact
//            from 2^-13 of the largest scale so far, and off by at most 2^-23 of
//            that scale from 2^-22 of it; below, a value may count as 0.  Any
//            other scale costs two roundings of 2^-11;
//   output   once, if bf16.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>

#include "kv8.cuh"
#include "ptx_util.cuh"
#include "rx.h"
#include "rx_internal.h"

// Bit 0: a slot outside [0, num_slots) was read (slot 0 used instead); bit 1:
// a barrier wait timed out.  Read by rx_device_check().
static __device__ int32_t g_kv8_att_error;

namespace {

using bf16 = __nv_bfloat16;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
// A row's weights are 2^(x - m + 6), m its reference, which moves to the largest
// score when a weight would exceed 2^15: within f16, and full f16 precision down
// to 2^-20 of the reference's.
constexpr float kWeightBias = 6.f;
constexpr float kMaxWeight = 15.f;

struct Args8 {
  const bf16* q;
  const uint8_t* kc;  // layer base, [Hkv][num_slots][D]
  const uint8_t* vc;
  const float2* scales;  // layer base, [Hkv][num_slots >> block_log2]
  int64_t head_stride;   // bytes between KV heads (num_slots * D)
  int64_t scale_stride;  // scales between KV heads
  int64_t num_slots;
  int64_t tma_row_base;  // row of (layer, KV head 0, slot 0) in the tensor maps
  int block_log2;
  const int32_t* table;
  int64_t row_stride;
  int hq;
  int group;
  float scale_log2;  // scale * log2(e)
  float key_mul;     // its mantissa, times 2^-kKeyShift (tiles)
  int scale_exp;     // its exponent
  // extend
  const int32_t* req_rows;
  const int32_t* prefix_len;
  const int32_t* qo_indptr;
  const int32_t* tile_indptr;
  int num_req;
  int num_tiles;
  int heads_interleaved;  // CTA order: 1 = tile-major over heads, 0 = head-major
  void* out;
  int out_bf16;
  float* lse;
  // decode
  const int32_t* work;
  const int32_t* members;
  int n_small;  // items of up to decode_small_rows rows, then the tile items
  int step;
  float* ws_o;
  float* ws_lse;
  bool beside_tiles;  // the streams run beside tiles
  bool chained;       // the launch before is this step's store
  int32_t* counter;  // next unit of the small items, NULL: unit = warp index
};

__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// (lo, hi) rounded to nearest f16 and packed.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Transpose of an 8x8 matrix of 16-bit elements held one row per four lanes.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src, bool valid) {
  int n = valid ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

// The streams beside tiles are launched before the tiles end, so they cannot
// wait for the kernels before them.  What they read (the pool, as the step's
// store left it) is handed on through the unit counter: a tile CTA, once the store
// has completed, releases the counter and then lets the streams start; a warp
// acquires it with its first unit.
__device__ __forceinline__ void release_counter(int32_t* counter) {
  asm volatile("red.release.gpu.global.add.s32 [%0], 0;\n" ::"l"(counter) : "memory");
}
__device__ __forceinline__ int acquire_unit(int32_t* counter) {
  int u;
  asm volatile("atom.acquire.gpu.global.add.s32 %0, [%1], 1;\n"
               : "=r"(u)
               : "l"(counter)
               : "memory");
  return u;
}

}  // namespace

#include "kv8_tile.cuh"

namespace {

// ---------------------------------------------------------------------------
// One warp streams the keys of one KV head for up to 8 NR query rows, 32 keys
// a step (16 at d = 256), through a ring of shared-memory stages filled with cp.async.  As in
// the bf16 decode kernel the products are computed transposed, keys (then
// output columns) in the M dimension and query rows in N:
//   S^T (keys x 8 rows)   = K (codes -> f16) . Q^T
//   O^T (D x 8 rows)      += V^T (codes -> f16) . P^T
// The contraction index of a product may be permuted freely, and the M index
// of O^T too, so that codes go from ldmatrix to operand registers with one
// conversion each: a lane of an untransposed ldmatrix holds four adjacent
// codes of a key, taken as d = 4c .. 4c+3 of a k-step; a lane of a transposed
// one holds the codes (d, d+1) of two adjacent keys, taken as operand rows g
// and g + 8.
// Eight warps with three stages each beat six with four by 2 to 10 % over the
// batches tried (private contexts of 7,001 to 16,001 keys, d = 128: 155 us against 166
// at 32 requests, 278 against 288 at 64): a warp's step is a chain of latencies.
// Steps of 16 keys at d = 128 cost 16 % (180 us), at d = 256 they make room for
// the third stage.
constexpr int kWarps = 8;
template <int D>
struct Pipe8 {
  static constexpr int KEYS = D == 128 ? 32 : 16;  // per step
  static constexpr int STAGES = 3;
  static constexpr int PITCH = D + 16;  // ldmatrix reads all 32 banks
  static constexpr int SCALES = 2 * KEYS * PITCH;
  static constexpr int STAGE_BYTES = SCALES + KEYS * 8;
  static constexpr int WARP_BYTES = STAGES * STAGE_BYTES;
  static constexpr int BYTES = kWarps * WARP_BYTES + 128;
};

// What a warp works on: n_rows query rows over keys [kb, ke) of one table
// row; row r is query head kvh G + r % G of member r / G.
struct Unit8 {
  const int32_t* trow;
  int kb, ke, kvh, n_rows;
  const int32_t* members;
  int part_base;
};

template <int NR, int D>
__device__ __forceinline__ void stream_unit(const Args8& a, const Unit8& u, uint32_t ring,
                                            const uint8_t* ring_g) {
  using Cfg = Pipe8<D>;
  constexpr int S = Cfg::STAGES;
  constexpr int KEYS = Cfg::KEYS;
  constexpr int MT = KEYS / 16;    // m-tiles of keys per step
  constexpr int PITCH = Cfg::PITCH;
  constexpr int NK = D / 16;
  constexpr int LPR = D / 16;      // lanes (16 B chunks) per row
  constexpr int RPI = 32 / LPR;    // rows per load instruction
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint8_t* kbase = a.kc + int64_t(u.kvh) * a.head_stride;
  const uint8_t* vbase = a.vc + int64_t(u.kvh) * a.head_stride;
  const float2* sbase = a.scales + int64_t(u.kvh) * a.scale_stride;
  const int kb = u.kb, ke = u.ke;
  const int n_steps = ke > kb ? (ke - kb + KEYS - 1) / KEYS : 0;

  // the slot of key `lane` of a step (-1 past the range), read one step ahead
  // of its use
  auto read_slot = [&](int st) -> int32_t {
    const int key = kb + st * KEYS + lane;
    return (KEYS == 32 || lane < KEYS) && key < ke ? __ldg(u.trow + key) : -1;
  };
  int32_t next_slot = n_steps > 0 ? read_slot(0) : -1;
  auto issue = [&](int st) {
    int32_t sl = next_slot;
    if (st + 1 < n_steps) next_slot = read_slot(st + 1);
    if ((KEYS == 32 || lane < KEYS) && kb + st * KEYS + lane < ke &&
        (sl < 0 || sl >= a.num_slots)) {
      atomicOr(&g_kv8_att_error, 1);
      sl = 0;
    }
    const uint32_t dst = ring + uint32_t(st % S) * Cfg::STAGE_BYTES;
    if (KEYS == 32 || lane < KEYS)
      cp_async_8(dst + Cfg::SCALES + lane * 8, sbase + ((sl < 0 ? 0 : sl) >> a.block_log2),
                 sl >= 0);
#pragma unroll
    for (int i = 0; i < KEYS / RPI; ++i) {
      const int row = i * RPI + lane / LPR;
      const int32_t s = __shfl_sync(0xffffffffu, sl, row);
      const int64_t at = int64_t(s < 0 ? 0 : s) * D + (lane % LPR) * 16;
      const uint32_t to = dst + uint32_t(row * PITCH + (lane % LPR) * 16);
      // keys past the range are zeros (their weights are 0, and 0 * V must be 0)
      rxk::cp_async_16(to, kbase + at, s >= 0);
      rxk::cp_async_16(to + KEYS * PITCH, vbase + at, s >= 0);
    }
  };
  __syncwarp();  // the previous unit's last stage has been read
#pragma unroll 1
  for (int p = 0; p < S - 1; ++p) {
    if (p < n_steps) issue(p);
    rxk::cp_async_commit();
  }

  // Q^T operands: row nt * 8 + g, scaled by 2^sh (an exact product) so that
  // its largest magnitude lies in [2^13, 2^14) of f16's range; below 2^-40 a
  // row's scores are zero for every key in reach and sh stops there.
  uint32_t qb[NR][NK][2];
  float rs[NR][2];  // score to log2 units of rows 2c, 2c + 1 of each n-tile
#pragma unroll
  for (int nt = 0; nt < NR; ++nt) {
    const int r = nt * 8 + g;
    const bool ok = r < u.n_rows;
    const uint2* src = reinterpret_cast<const uint2*>(a.q);
    if (ok) {
      const int m = r / a.group;
      src = reinterpret_cast<const uint2*>(
          a.q + (int64_t(u.members[m]) * a.hq + u.kvh * a.group + (r - m * a.group)) * D);
    }
    float amax = 0.f;
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
      const uint2 x = ok ? __ldg(src + 4 * kk + c) : make_uint2(0, 0);
      qb[nt][kk][0] = x.x;
      qb[nt][kk][1] = x.y;
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(__uint_as_float(x.x << 16)),
                                     fabsf(__uint_as_float(x.x & 0xffff0000u))),
                               fmaxf(fabsf(__uint_as_float(x.y << 16)),
                                     fabsf(__uint_as_float(x.y & 0xffff0000u)))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int sh = min(13 - (int(__float_as_uint(amax) >> 23) - 127), 53);
    const float f = kv8::pow2(sh);
#pragma unroll
    for (int kk = 0; kk < NK; ++kk)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qb[nt][kk][e] = pack_f16(__uint_as_float(qb[nt][kk][e] << 16) * f,
                                 __uint_as_float(qb[nt][kk][e] & 0xffff0000u) * f);
    // a query that is not finite has no defined scores: its row is NaN
    const float mine = amax < INFINITY ? a.scale_log2 * kv8::pow2(-sh) : NAN;
#pragma unroll
    for (int e = 0; e < 2; ++e) rs[nt][e] = __shfl_sync(0xffffffffu, mine, 4 * (2 * c + e));
  }

  float o[NR][NK][4];
  float m_off[NR][2], l_run[NR][2];  // the reference less 6; the weights' sum
#pragma unroll
  for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
    for (int mt = 0; mt < NK; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
    m_off[nt][0] = m_off[nt][1] = -INFINITY;
    l_run[nt][0] = l_run[nt][1] = 0.f;
  }
  float vref = 0.f, inv_vref = 0.f;

  const uint32_t k_lane =
      uint32_t(((lane & 7) + ((lane >> 3) & 1) * 8) * PITCH + (lane >> 4) * 16);
  const uint32_t v_lane = uint32_t(KEYS * PITCH) + k_lane;

#pragma unroll 1
  for (int st = 0; st < n_steps; ++st) {
    rxk::cp_async_wait<S - 2>();
    __syncwarp();  // every lane has its part of this stage, and is done with the last one
    if (st + S - 1 < n_steps) issue(st + S - 1);
    rxk::cp_async_commit();
    const uint32_t stage = ring + uint32_t(st % S) * Cfg::STAGE_BYTES;
    const float2* sc = reinterpret_cast<const float2*>(
        ring_g + (st % S) * Cfg::STAGE_BYTES + Cfg::SCALES);
    // (K is converted too: mma.sync on e4m3 operands, with Q in two parts, is
    // slower than f16 with the conversions, 161 us against 155 at 32 private
    // contexts of 7,001 to 16,001 keys)
    float x[NR][MT][4];  // m-tile h: keys 16 h + g (+ 8)
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int h = 0; h < MT; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][h][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < NK; kk += 2) {
#pragma unroll
      for (int h = 0; h < MT; ++h) {
        uint32_t r0, r1, r2, r3;
        rxk::ldsm_x4(stage + k_lane + uint32_t(h * 16 * PITCH + kk * 16), r0, r1, r2, r3);
        const uint32_t a0 = kv8::to_f16x2(r0), a1 = kv8::to_f16x2(r1),
                       a2 = kv8::to_f16x2(r0 >> 16), a3 = kv8::to_f16x2(r1 >> 16);
        const uint32_t b0 = kv8::to_f16x2(r2), b1 = kv8::to_f16x2(r3),
                       b2 = kv8::to_f16x2(r2 >> 16), b3 = kv8::to_f16x2(r3 >> 16);
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
          mma_f16(x[nt][h], a0, a1, a2, a3, qb[nt][kk][0], qb[nt][kk][1]);
          mma_f16(x[nt][h], b0, b1, b2, b3, qb[nt][kk + 1][0], qb[nt][kk + 1][1]);
        }
      }
    }
    float2 s4[2 * MT];  // scales of keys g, g + 8, ..
    float vmax = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
      s4[i] = sc[g + 8 * i];
      vmax = fmaxf(vmax, s4[i].y);
    }
    const int key0 = kb + st * KEYS + g;
    bool grow = vmax > vref;
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // (rounded down: scores of 2^24 and more are whole steps apart)
        const float limit = __fadd_rd(m_off[nt][e], kMaxWeight);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
          float& y = x[nt][i >> 1][(i & 1) * 2 + e];
          y = key0 + 8 * i < ke ? y * (s4[i].x * rs[nt][e]) : -INFINITY;
          grow |= y > limit;
        }
      }
    if (__any_sync(0xffffffffu, grow)) {
      float vm = vmax;
      float mx[NR][2];
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[nt][e] = fmaxf(x[nt][0][e], x[nt][0][2 + e]);
          if (MT == 2)
            mx[nt][e] = fmaxf(mx[nt][e], fmaxf(x[nt][MT - 1][e], x[nt][MT - 1][2 + e]));
        }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, off));
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], off));
      }
      float vf = 1.f;
      if (vm > vref) {
        vf = vref / vm;
        vref = vm;
        inv_vref = 1.f / vm;
      }
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float alpha = 1.f;
          if (mx[nt][e] - kWeightBias > m_off[nt][e]) {
            alpha = rxk::fast_exp2(m_off[nt][e] - (mx[nt][e] - kWeightBias));  // 0 from -inf
            m_off[nt][e] = mx[nt][e] - kWeightBias;
            l_run[nt][e] *= alpha;
          }
          alpha *= vf;
#pragma unroll
          for (int mt = 0; mt < NK; ++mt) {
            o[nt][mt][e] *= alpha;
            o[nt][mt][2 + e] *= alpha;
          }
        }
    }
    // P^T operands: b0 (keys 2c, 2c+1 of row g) is the transpose of the
    // accumulators' (key g, rows 2c, 2c+1)
    float wv[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) wv[i] = s4[i].y * inv_vref;
    uint32_t pb[NR][2 * MT];
#pragma unroll
    for (int nt = 0; nt < NR; ++nt) {
      const float m0 = m_off[nt][0] == -INFINITY ? 0.f : m_off[nt][0];
      const float m1 = m_off[nt][1] == -INFINITY ? 0.f : m_off[nt][1];
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        const float p0 = rxk::fast_exp2(x[nt][i >> 1][(i & 1) * 2] - m0);
        const float p1 = rxk::fast_exp2(x[nt][i >> 1][(i & 1) * 2 + 1] - m1);
        l_run[nt][0] += p0;
        l_run[nt][1] += p1;
        pb[nt][i] = movmatrix_trans(pack_f16(p0 * wv[i], p1 * wv[i]));
      }
    }
#pragma unroll
    for (int h = 0; h < MT; ++h)
#pragma unroll
      for (int mt = 0; mt < NK; mt += 2) {
        uint32_t r0, r1, r2, r3;
        rxk::ldsm_x4_t(stage + v_lane + uint32_t(h * 16 * PITCH + mt * 16), r0, r1, r2, r3);
        // bytes (d of key 2c, d of key 2c+1, d+1 of both)
        r0 = __byte_perm(r0, 0, 0x3120);
        r1 = __byte_perm(r1, 0, 0x3120);
        r2 = __byte_perm(r2, 0, 0x3120);
        r3 = __byte_perm(r3, 0, 0x3120);
        const uint32_t a0 = kv8::to_f16x2(r0), a1 = kv8::to_f16x2(r0 >> 16),
                       a2 = kv8::to_f16x2(r1), a3 = kv8::to_f16x2(r1 >> 16);
        const uint32_t b0 = kv8::to_f16x2(r2), b1 = kv8::to_f16x2(r2 >> 16),
                       b2 = kv8::to_f16x2(r3), b3 = kv8::to_f16x2(r3 >> 16);
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
          mma_f16(o[nt][mt], a0, a1, a2, a3, pb[nt][2 * h], pb[nt][2 * h + 1]);
          mma_f16(o[nt][mt + 1], b0, b1, b2, b3, pb[nt][2 * h], pb[nt][2 * h + 1]);
        }
      }
  }
  rxk::cp_async_wait<0>();

  // rows nt * 8 + 2c + e: output columns 16 mt + 2g, + 1
#pragma unroll
  for (int nt = 0; nt < NR; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_run[nt][e];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const int r = nt * 8 + 2 * c + e;
      if (r >= u.n_rows) continue;
      // (2^6 in both O and l; no key: zeros, lse -inf)
      const float inv = l == 0.f ? 0.f : vref / l;
      const float lse = l == 0.f ? -INFINITY : m_off[nt][e] * kLn2 + logf(l);
      const int mem = r / a.group;
      const int64_t at =
          int64_t(u.part_base + mem) * a.hq + u.kvh * a.group + (r - mem * a.group);
      float2* dst = reinterpret_cast<float2*>(a.ws_o + at * D);
#pragma unroll
      for (int mt = 0; mt < NK; ++mt)
        dst[8 * mt + g] = make_float2(o[nt][mt][e] * inv, o[nt][mt][2 + e] * inv);
      if (g == 0) a.ws_lse[at] = lse;
    }
}

// Extend calls of few tiles: a cluster of CTAs per tile, which share its keys.
template <int D>
__global__ void __launch_bounds__(kTileThreads, 1)
    extend8_split_kernel(const __grid_constant__ Args8 a, const __grid_constant__ Maps8 maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int c = int(blockIdx.x) / cluster_size();
  const int hkv = a.hq / a.group;
  tile8<D, false, true>(a, maps, smem_raw, a.num_tiles - 1 - c / hkv, c % hkv);
}

// Decode, items of few rows: warps take units (item, KV head) until none is
// left.  With tile items in the plan the kernel is launched after theirs and
// starts beside it, on the SMs that the tiles leave free and as they finish;
// it reads nothing that the tiles write, sees what was stored before through the
// counter (release_counter), and ends only after the tiles did, so that the merge
// behind it sees both.  Without tiles it may be chained to a
// step's store, and waits for that first.  (The other order, streams first on half
// of the SMs or on those that the tiles leave, is slower: a chat step of 256
// 139 us against 129, 64 requests over a document of 32,768 keys 161 against 122.)
template <int D>
__global__ void __launch_bounds__(kWarps * 32, 1) stream8_kernel(const __grid_constant__ Args8 a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  rxk::griddep_launch_dependents();
  if (!a.beside_tiles) rxk::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = rxk::smem_addr(smem_raw);
  const uint32_t off = ((raw + 127u) & ~127u) - raw + uint32_t(warp * Pipe8<D>::WARP_BYTES);
  const int hkv = a.hq / a.group;
  const int n_units = a.n_small * hkv;
  int unit = int(blockIdx.x) * kWarps + warp;
  bool acquire = a.beside_tiles;  // (then there is a counter)
  while (true) {
    if (a.counter) {
      if (lane == 0) unit = acquire ? acquire_unit(a.counter) : atomicAdd(a.counter, 1);
      __syncwarp();
      unit = __shfl_sync(0xffffffffu, unit, 0);
      acquire = false;
    }
    if (unit >= n_units) break;
    const int item = unit / hkv;
    const int32_t* w = a.work + int64_t(item) * RX_WORK_WORDS;
    Unit8 u;
    u.trow = a.table + int64_t(w[0]) * a.row_stride;
    u.kb = w[1];
    u.ke = w[7] > 0 ? min(w[2], w[7] + a.step) : w[2];
    u.members = a.members + w[3];
    u.part_base = w[5];
    u.n_rows = w[6];
    u.kvh = unit - item * hkv;
    if (u.n_rows <= 8) {
      stream_unit<1, D>(a, u, raw + off, smem_raw + off);
    } else if constexpr (D == 128) {
      stream_unit<2, D>(a, u, raw + off, smem_raw + off);
    } else if (lane == 0) {
      atomicOr(&g_kv8_att_error, 1);  // the plan gives head_dim 256 no such item
    }
    if (!a.counter) break;
  }
  rxk::griddep_wait();
}

// The streams may start (with tiles chained to a store, a warp of the tile says
// so once that has completed).
__device__ __forceinline__ void start_streams(const Args8& a) {
  if (a.chained || threadIdx.x != 0) return;
  if (a.counter) release_counter(a.counter);
  rxk::griddep_launch_dependents();
}

// Decode, items of more rows: one CTA per (item, KV head).
template <int D>
__global__ void __launch_bounds__(kTileThreads, 1)
    decode8_tile_kernel(const __grid_constant__ Args8 a, const __grid_constant__ Maps8 maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  start_streams(a);
  const int hkv = a.hq / a.group;
  tile8<D, true>(a, maps, smem_raw, int(blockIdx.x) / hkv, int(blockIdx.x) % hkv);
}

// Few of those: a cluster of CTAs per (item, KV head), which share its keys.
template <int D>
__global__ void __launch_bounds__(kTileThreads, 1)
    decode8_split_kernel(const __grid_constant__ Args8 a, const __grid_constant__ Maps8 maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  start_streams(a);
  const int c = int(blockIdx.x) / cluster_size();
  const int hkv = a.hq / a.group;
  tile8<D, true, true>(a, maps, smem_raw, c / hkv, c % hkv);
}

// Extend: one tile per CTA, heaviest row tile first; heads interleaved or
// head-major, as in the bf16 kernel.
template <int D>
__global__ void __launch_bounds__(kTileThreads, 1)
    extend8_kernel(const __grid_constant__ Args8 a, const __grid_constant__ Maps8 maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int c = int(blockIdx.x);
  const int hkv = a.hq / a.group;
  const int tile = a.heads_interleaved ? c / hkv : c % a.num_tiles;
  const int kvh = a.heads_interleaved ? c % hkv : c / a.num_tiles;
  tile8<D, false>(a, maps, smem_raw, a.num_tiles - 1 - tile, kvh);
}

// lse = log sum_s exp(lse_s), o = sum_s exp(lse_s - lse) o_s over the parts of
// a request and query head, rounded once to the output type.  A request
// without parts, or with empty ones only, gets zeros and lse = -inf.
// W warps share a row: warp w takes the parts w, w + W, .. eight rows at a time
// in flight, and the warps' sums meet in shared memory.  One warp a row when
// there are rows for every SM several times over; few rows are bound by the
// latency of the chain part list, lse, rows, which W warps walk in fewer rounds
// (decode of one request of 3,201 keys, 26 parts: 18 us with a warp a row).
// The plan's lists are read before the wait for the kernels that write parts.
constexpr int kMergeWarps = 8;
template <int D, int W>
__global__ void __launch_bounds__(kMergeWarps * 32) merge8_kernel(
    const int32_t* __restrict__ indptr, const int32_t* __restrict__ parts,
    const float* __restrict__ ws_o, const float* __restrict__ ws_lse, int hq, int B, void* out,
    int out_bf16, float* __restrict__ lse_out) {
  constexpr int V = D / 128;               // float4 per lane
  constexpr int CH = 8 / V;                // rows loaded together
  constexpr int ROWS = kMergeWarps / W;    // per CTA
  __shared__ float4 part_o[kMergeWarps][V][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = warp % W;
  const int64_t row = int64_t(blockIdx.x) * ROWS + warp / W;
  const bool active = row < int64_t(B) * hq;
  const int b = active ? int(row / hq) : 0;
  const int h = active ? int(row - int64_t(b) * hq) : 0;
  const int p0 = active ? __ldg(indptr + b) : 0;
  const int n = active ? __ldg(indptr + b + 1) - p0 : 0;
  int64_t e = lane < n ? int64_t(__ldg(parts + p0 + lane)) * hq + h : 0;  // of part `lane`
  rxk::griddep_launch_dependents();
  rxk::griddep_wait();
  const float4* o4 = reinterpret_cast<const float4*>(ws_o);
  float m = lane < n ? __ldcg(ws_lse + e) : -INFINITY;
  float4 x[CH][V];
  // the first rows of this warp, on their way while the maxima are taken
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int i = w + k * W;
    const int64_t ek = __shfl_sync(0xffffffffu, e, i & 31);
#pragma unroll
    for (int v = 0; v < V; ++v)
      x[k][v] = i < min(n, 32) ? __ldcg(o4 + ek * (D / 4) + v * 32 + lane)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float li = m;
  for (int i = lane + 32; i < n; i += 32)
    m = fmaxf(m, __ldcg(ws_lse + int64_t(__ldg(parts + p0 + i)) * hq + h));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float4 acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;  // of all parts, in every warp of the row
  for (int base = 0; base < n; base += 32) {
    if (base > 0) {
      const int i = base + lane;
      e = i < n ? int64_t(__ldg(parts + p0 + i)) * hq + h : 0;
      li = i < n ? __ldcg(ws_lse + e) : -INFINITY;
    }
    const float wt = li == -INFINITY ? 0.f : rxk::fast_exp2((li - m) * kLog2e);
    sum += wt;
    const int cnt = min(32, n - base);
    for (int j = w; j < cnt; j += W * CH) {
      if (base > 0 || j > w) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int i = j + k * W;
          const int64_t ek = __shfl_sync(0xffffffffu, e, i & 31);
#pragma unroll
          for (int v = 0; v < V; ++v)
            x[k][v] = i < cnt ? __ldcg(o4 + ek * (D / 4) + v * 32 + lane)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int i = j + k * W;
        const float wk = __shfl_sync(0xffffffffu, wt, i & 31);
        if (i < cnt) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            acc[v].x += wk * x[k][v].x;
            acc[v].y += wk * x[k][v].y;
            acc[v].z += wk * x[k][v].z;
            acc[v].w += wk * x[k][v].w;
          }
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if constexpr (W > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) part_o[warp][v][lane] = acc[v];
    __syncthreads();
    if (w != 0 || !active) return;
    for (int k = 1; k < W; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float4 y = part_o[warp + k][v][lane];
        acc[v].x += y.x;
        acc[v].y += y.y;
        acc[v].z += y.z;
        acc[v].w += y.w;
      }
  } else if (!active) {
    return;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float4 y =
        make_float4(acc[v].x * inv, acc[v].y * inv, acc[v].z * inv, acc[v].w * inv);
    const int64_t at = row * (D / 4) + v * 32 + lane;
    if (out_bf16)
      reinterpret_cast<uint2*>(out)[at] =
          make_uint2(rxk::pack_bf16(y.x, y.y), rxk::pack_bf16(y.z, y.w));
    else
      reinterpret_cast<float4*>(out)[at] = y;
  }
  if (lane == 0) lse_out[row] = sum == 0.f ? -INFINITY : m + logf(sum);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// A kernel's dynamic shared-memory limit is raised once per device.
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

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Tensor maps over the pool's K codes [L * Hkv * num_slots rows][D] bytes, 128-
// byte swizzle.
rx_status make_maps(Maps8* m, const rx_kv8_pool_desc* p) {
  EncodeTiled fn = reinterpret_cast<EncodeTiled>(rx_internal::tensor_map_encoder());
  const cuuint64_t dims[2] = {cuuint64_t(p->head_dim),
                              cuuint64_t(p->num_layers) * p->num_kv_heads * p->num_slots};
  const cuuint64_t strides[1] = {cuuint64_t(p->head_dim)};
  const cuuint32_t estr[2] = {1, 1};
  auto encode = [&](CUtensorMap* map, cuuint32_t rows) {
    const cuuint32_t box[2] = {128, rows};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p->k_codes, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const int rows = p->head_dim == 128 ? Tile8<128>::BN : Tile8<256>::BN;
  if (!fn || !encode(&m->k, rows) || !encode(&m->k16, 16))
    return rx_internal::set_error(RX_ERR_CUDA, "could not encode the 8-bit pool's tensor maps");
  return RX_OK;
}

// The arguments both calls share, checked before any CUDA call.
rx_status common_args(const char* what, const rx_kv8_pool_desc* pool, int32_t layer,
                      const void* d_q, int32_t num_q_heads, const int32_t* d_table,
                      int64_t row_stride, float scale, int32_t out_type, Args8* a) {
  static thread_local char buf[160];
  rx_status st = rx_internal::check_kv8_pool(pool, layer);
  if (st != RX_OK) return st;
  const char* bad = nullptr;
  if (num_q_heads <= 0 || num_q_heads % pool->num_kv_heads != 0)
    bad = "Hq % Hkv != 0";
  else if (!(scale >= 0x1p-40f && scale <= 0x1p40f))
    bad = "scale outside [2^-40, 2^40]";
  else if (out_type != RX_OUT_F32 && out_type != RX_OUT_BF16)
    bad = "unknown out_type";
  else if (row_stride < 0)
    bad = "row_stride < 0";
  if (bad) {
    snprintf(buf, sizeof(buf), "%s: %s", what, bad);
    return rx_internal::set_error(RX_ERR_INVALID, buf);
  }
  const int D = pool->head_dim;
  int lg = 0;
  while ((1 << lg) < pool->block) ++lg;
  const int64_t heads = int64_t(layer) * pool->num_kv_heads;
  a->q = static_cast<const bf16*>(d_q);
  a->kc = static_cast<const uint8_t*>(pool->k_codes) + heads * pool->num_slots * D;
  a->vc = static_cast<const uint8_t*>(pool->v_codes) + heads * pool->num_slots * D;
  a->scale_stride = pool->num_slots >> lg;
  a->scales = reinterpret_cast<const float2*>(pool->scales) + heads * a->scale_stride;
  a->head_stride = pool->num_slots * D;
  a->num_slots = pool->num_slots;
  a->tma_row_base = heads * pool->num_slots;
  a->block_log2 = lg;
  a->table = d_table;
  a->row_stride = row_stride;
  a->hq = num_q_heads;
  a->group = num_q_heads / pool->num_kv_heads;
  a->scale_log2 = scale * kLog2e;
  a->key_mul = ldexpf(frexpf(a->scale_log2, &a->scale_exp), 1 - kKeyShift);
  --a->scale_exp;
  a->out_bf16 = out_type == RX_OUT_BF16;
  return RX_OK;
}

}  // namespace

namespace rx_internal {

int32_t kv8_attention_error_flags(bool clear) {
  int32_t v = 0;
  cudaMemcpyFromSymbol(&v, g_kv8_att_error, sizeof(v));
  if (clear && v) {
    int32_t z = 0;
    cudaMemcpyToSymbol(g_kv8_att_error, &z, sizeof(z));
  }
  return v;
}

}  // namespace rx_internal

namespace {

void cluster_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, unsigned tiles, int split,
                    int bytes) {
  cfg->gridDim = dim3(tiles * unsigned(split));
  cfg->blockDim = dim3(kTileThreads);
  cfg->dynamicSmemBytes = size_t(bytes);
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(split);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

// CTAs that share a tile's keys: the most, a power of two up to 16, of which the
// device runs all clusters at once and a table row (the host knows its width,
// not the contexts) gives each a part.  20 queries over 8,000 keys, 8 heads: 91
// us with one CTA a tile, 29 so; 200 queries of one head over 21,800 keys: 375
// and 49.  Parts below three key tiles lose (20 queries over 400 keys, 8 heads:
// 19 us unsplit, 21 in two), and so do clusters in more than one wave (168
// tiles of 3,200 keys: 75 us unsplit, 87).
constexpr int kMaxSplitLog2 = 4;
template <int D, bool DECODE>
rx_status cluster_split(int64_t tiles, int64_t key_tiles, int64_t max_ctas, int* split) {
  constexpr auto* kernel = DECODE ? decode8_split_kernel<D> : extend8_split_kernel<D>;
  static std::atomic<bool> done[kMaxDevices];
  static std::atomic<int> fit[kMaxDevices][kMaxSplitLog2 + 1];  // clusters at once, + 1
  *split = 1;
  if (tiles * 2 > rx_internal::sm_count() || key_tiles < 2 * kMinPart) return RX_OK;
  rx_status st = ensure_smem(done, kernel, Tile8<D>::BYTES);
  if (st != RX_OK) return st;
  int dev = -1;
  cudaGetDevice(&dev);
  for (int lg = kMaxSplitLog2; lg >= 1; --lg) {
    if (key_tiles >> lg < kMinPart || tiles << lg > max_ctas) continue;
    int n = fit[dev][lg].load(std::memory_order_relaxed);
    if (n == 0) {
      if (lg > 3 && cudaFuncSetAttribute(kernel,
                                         cudaFuncAttributeNonPortableClusterSizeAllowed,
                                         1) != cudaSuccess)
        cudaGetLastError();
      cudaLaunchConfig_t cfg{};
      cudaLaunchAttribute attr[1];
      cluster_config(&cfg, attr, 1, 1 << lg, Tile8<D>::BYTES);
      int c = 0;
      if (cudaOccupancyMaxActiveClusters(&c, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();  // no cluster of this size
        c = 0;
      }
      n = c + 1;
      fit[dev][lg].store(n, std::memory_order_relaxed);
    }
    if (tiles <= n - 1) {
      *split = 1 << lg;
      break;
    }
  }
  return RX_OK;
}

}  // namespace

extern "C" rx_status rx_kv8_extend_attention(
    const rx_kv8_pool_desc* pool, int32_t layer, const void* d_q, int32_t num_q_heads,
    const int32_t* d_req_to_token, int64_t row_stride, const int32_t* d_req_rows,
    const int32_t* d_prefix_len, const int32_t* d_qo_indptr, const int32_t* d_tile_indptr,
    int32_t R, int64_t num_tiles, float scale, void* d_out, int32_t out_type, float* d_lse,
    rx_stream_t stream) {
  Args8 a{};
  rx_status st = common_args("rx_kv8_extend_attention", pool, layer, d_q, num_q_heads,
                             d_req_to_token, row_stride, scale, out_type, &a);
  if (st != RX_OK) return st;
  const int D = pool->head_dim;
  if (R < 0 || num_tiles < 0 || num_tiles > INT32_MAX / pool->num_kv_heads)
    return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_extend_attention: bad R or num_tiles");
  if (R == 0 || num_tiles == 0) return RX_OK;
  if (!d_q || !d_req_to_token || !d_req_rows || !d_prefix_len || !d_qo_indptr ||
      !d_tile_indptr || !d_out || !d_lse || !aligned16(d_q) || !aligned16(d_out))
    return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_extend_attention: NULL or misaligned");
  a.req_rows = d_req_rows;
  a.prefix_len = d_prefix_len;
  a.qo_indptr = d_qo_indptr;
  a.tile_indptr = d_tile_indptr;
  a.num_req = R;
  a.num_tiles = int(num_tiles);
  a.out = d_out;
  a.lse = d_lse;
  // heads interleaved (the heavy row tiles of every head first, a short
  // tail) for up to 8 waves of CTAs or when a request's keys over all heads
  // stay in L2 while its row tiles run; otherwise head-major, so the CTAs in
  // flight read one head's long key ranges
  a.heads_interleaved = num_tiles * pool->num_kv_heads <= int64_t(8) * rx_internal::sm_count() ||
                        row_stride * pool->num_kv_heads * int64_t(D) * 2 <= (int64_t(32) << 20);
  const unsigned ctas = unsigned(num_tiles * pool->num_kv_heads);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int split = 1;
  const int bn = D == 128 ? Tile8<128>::BN : Tile8<256>::BN;
  const int64_t key_tiles = (row_stride + bn - 1) / bn;
  st = D == 128 ? cluster_split<128, false>(ctas, key_tiles, INT64_MAX, &split)
                : cluster_split<256, false>(ctas, key_tiles, INT64_MAX, &split);
  if (st != RX_OK) return st;
  if (split > 1) {
    Maps8 maps;
    st = make_maps(&maps, pool);
    if (st != RX_OK) return st;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cluster_config(&cfg, attr, ctas, split, D == 128 ? Tile8<128>::BYTES : Tile8<256>::BYTES);
    cfg.stream = s;
    if (D == 128)
      cudaLaunchKernelEx(&cfg, extend8_split_kernel<128>, a, maps);
    else
      cudaLaunchKernelEx(&cfg, extend8_split_kernel<256>, a, maps);
    return rx_internal::launch_status("rx_kv8_extend_attention");
  }
  static std::atomic<bool> done128[kMaxDevices], done256[kMaxDevices];
  st = D == 128 ? ensure_smem(done128, extend8_kernel<128>, Tile8<128>::BYTES)
                : ensure_smem(done256, extend8_kernel<256>, Tile8<256>::BYTES);
  Maps8 maps;
  if (st == RX_OK) st = make_maps(&maps, pool);
  if (st != RX_OK) return st;
  if (D == 128)
    extend8_kernel<128><<<ctas, kTileThreads, Tile8<128>::BYTES, s>>>(a, maps);
  else
    extend8_kernel<256><<<ctas, kTileThreads, Tile8<256>::BYTES, s>>>(a, maps);
  return rx_internal::launch_status("rx_kv8_extend_attention");
}

namespace {

// rx_kv8_decode_attention.  step_counter: a counter of the call's own that is
// zero already (NULL: the one behind the workspace's partials, reset here);
// chained: the launch before is the step's store, whose end the kernels wait for
// on the device, where they need it.
rx_status decode8(
    const rx_kv8_pool_desc* pool, int32_t layer, const void* d_q, int32_t num_q_heads,
    const int32_t* d_req_to_token, int64_t row_stride, const int32_t* d_plan,
    const rx_decode_plan_info* info, int32_t B, int32_t step, float scale, void* d_out,
    int32_t out_type, float* d_lse, void* d_workspace, size_t workspace_bytes,
    rx_stream_t stream, int32_t* step_counter, bool chained) {
  Args8 a{};
  rx_status st = common_args("rx_kv8_decode_attention", pool, layer, d_q, num_q_heads,
                             d_req_to_token, row_stride, scale, out_type, &a);
  if (st != RX_OK) return st;
  if (!info || B < 0 || step < 0)
    return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_decode_attention: bad argument");
  if (B == 0) return RX_OK;
  if (int64_t(workspace_bytes) < info->workspace_bytes || !d_workspace ||
      !aligned16(d_workspace))
    return rx_internal::set_error(
        RX_ERR_INVALID, "rx_kv8_decode_attention: workspace missing, small or misaligned");
  if (!d_q || !d_req_to_token || !d_plan || !d_out || !d_lse || !aligned16(d_q) ||
      !aligned16(d_out))
    return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_decode_attention: NULL or misaligned");
  const int D = pool->head_dim;
  const int64_t hkv = pool->num_kv_heads;
  const int64_t n_small = info->n_work - info->n_work_tc;
  if (info->n_work < 0 || n_small < 0 || info->n_work_tc < 0 || info->n_parts < 0 ||
      info->n_work > INT32_MAX / hkv)
    return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_decode_attention: bad plan info");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // the workspace layout of rx_plan_decode: partial rows, their lse, a counter
  const int64_t o_bytes = (info->n_parts * num_q_heads * int64_t(D) * 4 + 255) / 256 * 256;
  const int64_t l_bytes = (info->n_parts * num_q_heads * 4 + 255) / 256 * 256;
  a.ws_o = static_cast<float*>(d_workspace);
  a.ws_lse = reinterpret_cast<float*>(static_cast<char*>(d_workspace) + o_bytes);
  int32_t* counter =
      reinterpret_cast<int32_t*>(static_cast<char*>(d_workspace) + o_bytes + l_bytes);
  a.work = d_plan + info->off_work;
  a.members = d_plan + info->off_members;
  a.n_small = int(n_small);
  a.step = step;
  const int64_t sms = rx_internal::sm_count();
  const int64_t small_units = n_small * hkv;
  int64_t ctas = (small_units + kWarps - 1) / kWarps;
  if (ctas > sms || (ctas > 0 && info->n_work_tc > 0)) {
    // more units than warps, or warps that start late (beside the tiles):
    // units are taken from a counter, heaviest first
    ctas = std::min(ctas, sms);
    a.counter = step_counter ? step_counter : counter;
    if (!step_counter && cudaMemsetAsync(counter, 0, sizeof(int32_t), s) != cudaSuccess)
      return rx_internal::launch_status("rx_kv8_decode_attention: counter reset");
  }
  a.chained = chained;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (info->n_work_tc > 0) {
    static std::atomic<bool> done128[kMaxDevices], done256[kMaxDevices];
    st = D == 128 ? ensure_smem(done128, decode8_tile_kernel<128>, Tile8<128>::BYTES)
                  : ensure_smem(done256, decode8_tile_kernel<256>, Tile8<256>::BYTES);
    Maps8 maps;
    if (st == RX_OK) st = make_maps(&maps, pool);
    if (st != RX_OK) return st;
    const unsigned n = unsigned(info->n_work_tc * hkv);
    const int bn = D == 128 ? Tile8<128>::BN : Tile8<256>::BN;
    // Sharing the tiles' keys pays when they outlast the streams beside them: by
    // far, on all SMs (193 requests over 8,098 common keys: 92 us unsplit, 49),
    // by less on three eighths, beside the streams (64 over 2,000 and some 460 of
    // their own, d = 256: 65 and 45, and a step of such a run 49 and 41), and not
    // when the streams fill the time (a chat step of 256: 126 us, 136 split).
    // A key tile is about 1.3 us, the plan's keys are read at 5.8 TB/s, and a
    // tile item has kDecodeKeysPerRow keys per query row at most.
    const int64_t chunk =
        std::min(row_stride, std::max<int64_t>(rx_internal::kDecodeMinChunk,
                                               int64_t(rx_internal::kDecodeKeysPerRow) * B *
                                                   a.group));
    const int64_t key_tiles = (chunk + bn - 1) / bn;
    int split = 1;
    const float read_us = float(info->distinct_kv_tokens) * float(hkv) *
                          (2.f * float(D) + 8.f / float(pool->block)) / 5.8e6f;
    const float ratio = 1.3f * float(key_tiles) / read_us;
    if (ratio >= 2.f) {
      const int64_t max_ctas = ratio >= 6.f ? INT64_MAX : sms * 3 / 8;
      st = D == 128 ? cluster_split<128, true>(n, key_tiles, max_ctas, &split)
                    : cluster_split<256, true>(n, key_tiles, max_ctas, &split);
      if (st != RX_OK) return st;
    }
    cudaLaunchConfig_t tc{};
    cudaLaunchAttribute ta[2];
    cluster_config(&tc, ta, n, split, D == 128 ? Tile8<128>::BYTES : Tile8<256>::BYTES);
    tc.stream = s;
    if (split == 1) tc.numAttrs = 0;
    if (chained) ta[tc.numAttrs++] = attr[0];
    if (split > 1)
      cudaLaunchKernelEx(&tc, D == 128 ? decode8_split_kernel<128> : decode8_split_kernel<256>, a,
                         maps);
    else
      cudaLaunchKernelEx(&tc, D == 128 ? decode8_tile_kernel<128> : decode8_tile_kernel<256>, a,
                         maps);
    st = rx_internal::launch_status("rx_kv8_decode_attention: tiles");
    if (st != RX_OK) return st;
  }
  if (ctas > 0) {
    static std::atomic<bool> done128[kMaxDevices], done256[kMaxDevices];
    st = D == 128 ? ensure_smem(done128, stream8_kernel<128>, Pipe8<128>::BYTES)
                  : ensure_smem(done256, stream8_kernel<256>, Pipe8<256>::BYTES);
    if (st != RX_OK) return st;
    cfg.gridDim = dim3(unsigned(ctas));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = D == 128 ? Pipe8<128>::BYTES : Pipe8<256>::BYTES;
    a.beside_tiles = info->n_work_tc > 0;
    cfg.numAttrs = a.beside_tiles || chained ? 1 : 0;
    if (D == 128)
      cudaLaunchKernelEx(&cfg, stream8_kernel<128>, a);
    else
      cudaLaunchKernelEx(&cfg, stream8_kernel<256>, a);
    st = rx_internal::launch_status("rx_kv8_decode_attention: streams");
    if (st != RX_OK) return st;
  }
  cfg.dynamicSmemBytes = 0;
  // launched while the kernels before it run; it waits on the device for their
  // end (a plan without items has none, and its lists may be behind the
  // caller's last kernel)
  cfg.numAttrs = info->n_work > 0 ? 1 : 0;
  const int64_t rows = int64_t(B) * num_q_heads;
  const bool wide = rows < sms * 16;  // eight warps a row
  cfg.gridDim = dim3(unsigned(wide ? rows : (rows + kMergeWarps - 1) / kMergeWarps));
  cfg.blockDim = dim3(kMergeWarps * 32);
  const int32_t* indptr = d_plan + info->off_req_part_indptr;
  const int32_t* parts = d_plan + info->off_req_parts;
  const float* wo = a.ws_o;
  const float* wl = a.ws_lse;
  auto* merge = D == 128 ? (wide ? merge8_kernel<128, 8> : merge8_kernel<128, 1>)
                         : (wide ? merge8_kernel<256, 8> : merge8_kernel<256, 1>);
  cudaLaunchKernelEx(&cfg, merge, indptr, parts, wo, wl, int(num_q_heads), int(B), d_out,
                     int(a.out_bf16), d_lse);
  return rx_internal::launch_status("rx_kv8_decode_attention: merge");
}

}  // namespace

extern "C" rx_status rx_kv8_decode_attention(
    const rx_kv8_pool_desc* pool, int32_t layer, const void* d_q, int32_t num_q_heads,
    const int32_t* d_req_to_token, int64_t row_stride, const int32_t* d_plan,
    const rx_decode_plan_info* info, int32_t B, int32_t step, float scale, void* d_out,
    int32_t out_type, float* d_lse, void* d_workspace, size_t workspace_bytes,
    rx_stream_t stream) {
  return decode8(pool, layer, d_q, num_q_heads, d_req_to_token, row_stride, d_plan, info, B, step,
                 scale, d_out, out_type, d_lse, d_workspace, workspace_bytes, stream, nullptr,
                 false);
}

extern "C" rx_status rx_kv8_extend_batches(const rx_kv8_pool_desc* pool, int32_t layer,
                                           int32_t num_q_heads, const rx_extend_batch* batches,
                                           int32_t n, float scale, const rx_event_t* events,
                                           rx_stream_t stream) {
  if (n < 0 || (n && !batches))
    return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_extend_batches: bad batch list");
  rx_status r = rx_internal::check_kv8_pool(pool, layer);
  if (r != RX_OK) return r;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto mark = [&](int32_t i, int k) -> rx_status {
    if (!events) return RX_OK;
    if (cudaEventRecord(reinterpret_cast<cudaEvent_t>(events[4 * int64_t(i) + k]), s) !=
        cudaSuccess)
      return rx_internal::launch_status("rx_kv8_extend_batches: event record");
    return RX_OK;
  };
  // in batch order on one stream: a batch reads what the ones before it stored
  for (int32_t i = 0; i < n; ++i) {
    const rx_extend_batch& b = batches[i];
    if ((r = mark(i, 0)) != RX_OK) return r;
    r = rx_kv8_store(pool, layer, b.d_new_slots, b.d_k, b.d_v, b.n_new, stream);
    if (r != RX_OK) return r;
    if ((r = mark(i, 1)) != RX_OK || (r = mark(i, 2)) != RX_OK) return r;
    r = rx_kv8_extend_attention(pool, layer, b.d_q, num_q_heads, b.d_req_to_token, b.row_stride,
                                b.d_req_rows, b.d_prefix_len, b.d_qo_indptr, b.d_tile_indptr, b.R,
                                b.num_tiles, scale, b.d_out, RX_OUT_F32, b.d_lse, stream);
    if (r != RX_OK) return r;
    if ((r = mark(i, 3)) != RX_OK) return r;
  }
  return RX_OK;
}

extern "C" rx_status rx_kv8_decode_steps(const rx_kv8_pool_desc* pool, int32_t layer,
                                         int32_t num_q_heads, const int32_t* d_req_to_token,
                                         int64_t row_stride, const rx_decode_step* steps,
                                         int32_t n_steps, int32_t B, float scale,
                                         void* d_workspace, size_t workspace_bytes,
                                         rx_stream_t stream) {
  if (n_steps < 0 || (n_steps && !steps))
    return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_decode_steps: bad step list");
  rx_status r = rx_internal::check_kv8_pool(pool, layer);
  if (r != RX_OK) return r;
  if (num_q_heads <= 0 || num_q_heads % pool->num_kv_heads != 0)
    return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_decode_steps: Hq % Hkv != 0");
  // Every step has its own unit counter, reset together behind the largest
  // step's partials if the workspace has room, and the launches of steps that
  // follow on under one plan are chained: the store is launched while the merge
  // before it runs, and the tiles or streams while the store does.  Each waits on
  // the device for the end of the kernel before it (which did so too) before it
  // reads what that writes or writes what that reads; tiles of shared segments so
  // run beside the end of the step before.  The plan says which segments its steps
  // store into.  Another plan's segments may hold what the steps before stored, so
  // its first step starts when those have ended.
  int64_t region = 0;
  bool own_counters = n_steps > 0 && B > 0;
  for (int32_t i = 0; own_counters && i < n_steps; ++i) {
    const rx_decode_plan_info* inf = steps[i].info;
    own_counters = inf && inf->n_parts >= 0;
    if (!own_counters) break;
    const int64_t o = inf->n_parts * num_q_heads * int64_t(pool->head_dim) * 4;
    const int64_t l = inf->n_parts * num_q_heads * 4;
    region = std::max(region, (o + 255) / 256 * 256 + (l + 255) / 256 * 256);
  }
  own_counters = own_counters && d_workspace && aligned16(d_workspace) &&
                 int64_t(workspace_bytes) >= region + 4 * int64_t(n_steps);
  int32_t* counters =
      own_counters ? reinterpret_cast<int32_t*>(static_cast<char*>(d_workspace) + region) : nullptr;
  if (own_counters && cudaMemsetAsync(counters, 0, 4 * size_t(n_steps),
                                      reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return rx_internal::launch_status("rx_kv8_decode_steps: counters reset");
  for (int32_t i = 0; i < n_steps; ++i) {
    const rx_decode_step& t = steps[i];
    const bool chained = own_counters && i > 0 && t.d_plan == steps[i - 1].d_plan;
    r = rx_internal::kv8_store(pool, layer, t.d_slots, t.d_k, t.d_v, B, stream, chained);
    if (r != RX_OK) return r;
    r = decode8(pool, layer, t.d_q, num_q_heads, d_req_to_token, row_stride, t.d_plan, t.info, B,
                t.step, scale, t.d_out, RX_OUT_F32, t.d_lse, d_workspace, workspace_bytes, stream,
                own_counters ? counters + i : nullptr, chained);
    if (r != RX_OK) return r;
  }
  return RX_OK;
}
