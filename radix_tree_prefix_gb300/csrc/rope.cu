// Norm and position rotation of queries and keys, and their append to the
// pool in the same pass (rx_rope_init, rx_qk_rope, rx_qkv_store).
//
// A head row x of d elements becomes
//   y = x / sqrt(mean(x^2) + eps) * w        (the norm, if any; w or 1 + w)
//   (a, b) -> m (a cos t - b sin t, a sin t + b cos t),  t = position * f_i
// for the pairs (a, b) = (y_i, y_{i + rot/2}) or (y_2i, y_2i+1) of the first
// rot elements; the rest of the row stays, to the bit where nothing is normalised.
// Everything else is held in fp32 and rounded once, to bf16.
//
// Angles: f_i is held as a 64-bit fraction of a turn, so position * f_i
// modulo one turn is one 64-bit integer product that is exact for every
// position (the fraction's own error is 2^-52 of f_i: 2^-23 of a turn at
// position 2^31).  Only the turn's fraction goes to fp32, and its sine and
// cosine are taken within half a turn, where the special-function unit is
// good to 2^-20.5, far below a bf16 rounding (2^-8).  No table of angles is
// read and no position is too far.
//
// Bound by HBM: every row is read once and written once.  A thread holds the
// eight pairs of one share of a head (16 elements in two 16-byte pieces), so
// D/16 threads hold a head and a pair's two elements meet in one thread
// without a shuffle; a warp takes 32/(D/16) heads at a time, computes its
// eight sines and cosines a lane once, and walks its token's heads with them.
// Measured: 32,767 tokens of 40 heads of 128 in 109 us (6.16 TB/s, 91% of a
// copy's rate; 2 us less where the rest of a row was turned by an angle of 0), the
// append of 51,200 tokens of 24 heads of 256 in 224 us (5.6 TB/s, 83%; its writes go
// to nine places), one token 3 us.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include "ptx_util.cuh"
#include "rx.h"
#include "rx_internal.h"

// Bit 0: rx_qkv_store met a slot outside [1, num_slots) (its K and V are not
// stored).  Read by rx_device_check().
static __device__ int32_t g_rope_error;

namespace {

struct RopeArgs {
  rx_rope rope;
  const int32_t* pos;
  const int32_t* slots;
  const uint4* q;  // strides in 16-byte pieces
  const uint4* k;
  const uint4* v;
  uint4* q_out;
  uint4* k_out;  // the pool's layer for a store
  uint4* v_out;
  const uint4* q_weight;
  const uint4* k_weight;
  int64_t T, q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int64_t head_stride;  // pieces between two heads of the pool
  int64_t num_slots;
  int hq, hkv;
  int split;     // warps that share a token's heads
  float eps;
  float offset;  // added to a weight: 0 or 1
  int whole;     // every row starts on a 32-byte boundary
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(rxk::pack_bf16(f[0], f[1]), rxk::pack_bf16(f[2], f[3]),
                    rxk::pack_bf16(f[4], f[5]), rxk::pack_bf16(f[6], f[7]));
}

// One 16-element share of a row: pieces a and b, normalised by the weights w
// (sums: some head of the warp is, and the shuffles of the row sums are the
// whole warp's; norm: this one is) and rotated.  Pair i of the share is (a_i,
// b_i), or INTERLEAVED (a_2i, a_2i+1), then (b_2i, b_2i+1).
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void turn_share(uint4& ua, uint4& ub, bool sums, bool norm,
                                           const uint4 (&w)[2], float eps, float offset,
                                           const float (&cs)[8], const float (&sn)[8]) {
  float a[8], b[8];
  unpack8(ua, a);
  unpack8(ub, b);
  float r = 1.f;
  if (sums) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    r = rsqrtf(ss * (1.f / D) + eps);
  }
  if (norm) {
    float wa[8], wb[8];
    unpack8(w[0], wa);
    unpack8(w[1], wb);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] *= r * (wa[i] + offset);
      b[i] *= r * (wb[i] + offset);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& x = INTERLEAVED ? (i < 4 ? a[2 * (i & 3)] : b[2 * (i & 3)]) : a[i];
    float& y = INTERLEAVED ? (i < 4 ? a[2 * (i & 3) + 1] : b[2 * (i & 3) + 1]) : b[i];
    const float x0 = x, y0 = y;
    x = x0 * cs[i] - y0 * sn[i];
    y = fmaf(x0, sn[i], y0 * cs[i]);
  }
  ua = pack8(a);
  ub = pack8(b);
}

// The first n pairs of a share from the turned pieces, the others as they were (a product
// with a sine of 0 takes an infinity from one element into the next, and loses a zero's sign
// and a NaN's bits).  Of shares whose pairs do not all turn or all stay.
template <bool INTERLEAVED>
__device__ __forceinline__ void keep_rest(uint4& ta, uint4& tb, const uint4& a, const uint4& b,
                                          int n) {
  if constexpr (INTERLEAVED) {  // a pair is a word
    ta = make_uint4(n > 0 ? ta.x : a.x, n > 1 ? ta.y : a.y, n > 2 ? ta.z : a.z,
                    n > 3 ? ta.w : a.w);
    tb = make_uint4(n > 4 ? tb.x : b.x, n > 5 ? tb.y : b.y, n > 6 ? tb.z : b.z,
                    n > 7 ? tb.w : b.w);
  } else {
    auto first = [&](uint32_t t, uint32_t old, int i) {  // elements i and i + 1
      return n > i + 1 ? t : n > i ? __byte_perm(t, old, 0x7610) : old;
    };
    ta = make_uint4(first(ta.x, a.x, 0), first(ta.y, a.y, 2), first(ta.z, a.z, 4),
                    first(ta.w, a.w, 6));
    tb = make_uint4(first(tb.x, b.x, 0), first(tb.y, b.y, 2), first(tb.z, b.z, 4),
                    first(tb.w, b.w, 6));
  }
}

// The sines and cosines of the eight pairs of share c at a position.
__device__ __forceinline__ void angles(const rx_rope& r, int c, int32_t pos, float (&cs)[8],
                                       float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int pair = 8 * c + i;
    cs[i] = 1.f;
    sn[i] = 0.f;
    if (2 * pair < r.rot_dim) {
      // the angle in turns, in [-1/2, 1/2)
      const int64_t turn = int64_t(uint64_t(int64_t(pos)) * r.turns[pair]);
      const float angle = float(int32_t(turn >> 32)) * (6.283185307179586f / 4294967296.f);
      __sincosf(angle, &sn[i], &cs[i]);
      sn[i] *= r.magnitude;
      cs[i] *= r.magnitude;
    }
  }
}

// Where a token's queries, keys and values lie, and where they go (head 0).
struct Rows {
  const uint4* from[3];
  uint4* to[3];
  template <int D, bool STORE>
  __device__ __forceinline__ void set(const RopeArgs& a, int64_t t, int64_t slot) {
    from[0] = a.q + t * a.q_stride;
    from[1] = a.k + t * a.k_stride;
    from[2] = STORE ? a.v + t * a.v_stride : nullptr;
    to[0] = a.q_out + t * a.q_out_stride;
    to[1] = STORE ? a.k_out + slot * (D / 8) : a.k_out + t * a.k_out_stride;
    to[2] = STORE ? a.v_out + slot * (D / 8) : nullptr;
  }
};
// Head h of a token: queries, then keys, then values.
template <int D, bool STORE>
struct Head {
  int kind, i;  // 0: query, 1: key, 2: value; its number among them
  __device__ __forceinline__ Head(const RopeArgs& a, int h) {
    kind = h < a.hq ? 0 : STORE && h >= a.hq + a.hkv ? 2 : 1;
    i = h - (kind > 0 ? a.hq : 0) - (kind > 1 ? a.hkv : 0);
  }
  __device__ __forceinline__ const uint4* from(const Rows& r) const {
    return r.from[kind] + i * (D / 8);
  }
  __device__ __forceinline__ uint4* to(const RopeArgs& a, const Rows& r) const {
    return r.to[kind] + i * (STORE && kind > 0 ? a.head_stride : int64_t(D / 8));
  }
};

// A warp takes a token's heads HPW at a time (or `split` warps share them), the
// next step's rows on their way while one is turned and written.  What counts is
// how many warps an SM holds: small CTAs of 64 registers a thread keep 32 of them
// (a chat turn's append 219 us; three steps ahead with 80 registers 252, and a ring
// of shared memory under warps that walk over tokens 287).
constexpr int kWarps = 2;  // per CTA
template <int D, bool INTERLEAVED, bool STORE, bool PART>
__global__ void __launch_bounds__(kWarps * 32, 16)
    rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int TPH = D / 16;  // threads a head
  constexpr int HPW = 32 / TPH;
  __shared__ Rows rows_of[kWarps];  // (in registers they cost the SM a third of its warps)
  Rows& rows = rows_of[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const int c = lane % TPH;  // share of the head
  const int64_t unit = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t t = unit / a.split;
  if (t >= a.T) return;  // the whole warp
  const int part = int(unit - t * a.split);
  // the share's pieces, in pieces of the row
  int ea = 2 * c, eb = 2 * c + 1;
  if (!INTERLEAVED && 16 * c < a.rope.rot_dim) {
    ea = c;
    eb = a.rope.rot_dim / 16 + c;
  }
  auto load = [&](const uint4* row, uint4& x, uint4& y) {
    if (INTERLEAVED && a.whole) {  // both pieces at once
      asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                   : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w), "=r"(y.x), "=r"(y.y),
                     "=r"(y.z), "=r"(y.w)
                   : "l"(row + ea));
    } else {
      x = row[ea];
      y = row[eb];
    }
  };
  int32_t slot = 1;
  bool keep = true;
  if constexpr (STORE) {
    slot = __ldg(a.slots + t);
    keep = slot >= 1 && slot < a.num_slots;
    if (!keep) {
      atomicOr(&g_rope_error, 1);
      slot = 1;
    }
  }
  if (lane == 0) rows.set<D, STORE>(a, t, slot);
  __syncwarp();
  const bool norm_q = a.q_weight != nullptr, norm_k = a.k_weight != nullptr;
  const int heads = a.hq + a.hkv * (STORE ? 2 : 1);
  const int step = a.split * HPW;
  int h = part * HPW + lane / TPH;
  uint4 nx = {}, ny = {};
  if (h < heads) load(Head<D, STORE>(a, h).from(rows), nx, ny);
  float cs[8], sn[8];
  angles(a.rope, c, a.pos ? __ldg(a.pos + t) : 0, cs, sn);
  const int n = a.rope.rot_dim / 2 - 8 * c;  // pairs of the share that turn (or all, or none)
  const bool turns = n > 0;
#pragma unroll 1
  for (int h0 = part * HPW; h0 < heads; h0 += step, h += step) {
    uint4 x = nx, y = ny;
    if (h + step < heads) load(Head<D, STORE>(a, h + step).from(rows), nx, ny);
    const Head<D, STORE> head(a, h);
    const bool is_q = head.kind == 0, is_v = head.kind == 2, live = h < heads;
    if (!__all_sync(0xffffffffu, is_v || !live)) {
      const bool norm = !is_v && (is_q ? norm_q : norm_k);
      uint4 w[2] = {};
      if (norm) {  // (from L1)
        w[0] = __ldg((is_q ? a.q_weight : a.k_weight) + ea);
        w[1] = __ldg((is_q ? a.q_weight : a.k_weight) + eb);
      }
      uint4 rx = x, ry = y;
      turn_share<D, INTERLEAVED>(rx, ry, norm_q || norm_k, norm, w, a.eps, a.offset, cs, sn);
      if (PART && !norm) keep_rest<INTERLEAVED>(rx, ry, x, y, n);
      if (norm || (turns && !is_v)) {  // (else the share's bits stay as they are)
        x = rx;
        y = ry;
      }
    }
    if (live && (is_q || keep)) {
      uint4* row = head.to(a, rows);
      if (INTERLEAVED && a.whole) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(row + ea),
                     "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(y.x), "r"(y.y), "r"(y.z),
                     "r"(y.w)
                     : "memory");
      } else {
        row[ea] = x;
        row[eb] = y;
      }
    }
  }
}

// Half layout with a rotated part that is no multiple of 16, whose pairs do not
// fall on 16-byte pieces: element by element.
template <int D, bool STORE>
__global__ void __launch_bounds__(kWarps * 32)
    rope_odd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int TPH = D / 16;
  constexpr int HPW = 32 / TPH;
  const int lane = threadIdx.x & 31;
  const int c = lane % TPH, sub = lane / TPH;
  const int64_t unit = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t t = unit / a.split;
  if (t >= a.T) return;  // the whole warp
  const int part = int(unit - t * a.split);
  const int rot = a.rope.rot_dim;
  float cs[8], sn[8];
  angles(a.rope, c, a.pos ? __ldg(a.pos + t) : 0, cs, sn);
  // pair i of the rotated part, then the rest of the row two by two
  auto element = [&](int i, int half) {
    const int pair = 8 * c + i;
    return 2 * pair < rot ? pair + half * (rot / 2) : 2 * pair + half;
  };
  auto load = [&](const uint4* row, uint4& x, uint4& y) {
    const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
    uint32_t p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      p[i] = uint32_t(r[element(i, 0)]) | (uint32_t(r[element(i, 1)]) << 16);
    x = make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                   __byte_perm(p[4], p[5], 0x5410), __byte_perm(p[6], p[7], 0x5410));
    y = make_uint4(__byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632),
                   __byte_perm(p[4], p[5], 0x7632), __byte_perm(p[6], p[7], 0x7632));
  };
  int64_t slot = 1;
  bool keep = true;
  if constexpr (STORE) {
    slot = __ldg(a.slots + t);
    keep = slot >= 1 && slot < a.num_slots;
    if (!keep) {
      atomicOr(&g_rope_error, 1);
      slot = 1;
    }
  }
  Rows rows;
  rows.set<D, STORE>(a, t, slot);
  const bool norm_q = a.q_weight != nullptr, norm_k = a.k_weight != nullptr;
  const int heads = a.hq + a.hkv * (STORE ? 2 : 1);
#pragma unroll 1
  for (int h0 = part * HPW; h0 < heads; h0 += a.split * HPW) {
    const int h = h0 + sub;
    const Head<D, STORE> head(a, h);
    const bool is_q = head.kind == 0, is_v = head.kind == 2, live = h < heads;
    uint4 x = {}, y = {}, w[2] = {};
    if (live) load(head.from(rows), x, y);
    const bool norm = !is_v && (is_q ? norm_q : norm_k);
    if (norm) load(is_q ? a.q_weight : a.k_weight, w[0], w[1]);
    uint4 rx = x, ry = y;
    turn_share<D, false>(rx, ry, norm_q || norm_k, norm, w, a.eps, a.offset, cs, sn);
    if (!norm) keep_rest<false>(rx, ry, x, y, rot / 2 - 8 * c);
    if (!is_v) {
      x = rx;
      y = ry;
    }
    if (live && (is_q || keep)) {
      uint16_t* r = reinterpret_cast<uint16_t*>(head.to(a, rows));
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[element(i, 0)] = uint16_t(xs[i >> 1] >> (16 * (i & 1)));
        r[element(i, 1)] = uint16_t(ys[i >> 1] >> (16 * (i & 1)));
      }
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int D, bool STORE>
void launch(const RopeArgs& a, cudaStream_t s) {
  const int64_t all = (a.T * a.split + kWarps - 1) / kWarps;
  const dim3 block{kWarps * 32};
  const dim3 grid{unsigned(all)};
  const bool half = a.rope.layout == RX_ROPE_HALF;
  if (a.rope.rot_dim % 16 != 0)  // a share has pairs of both kinds
    half ? rope_odd_kernel<D, STORE><<<grid, block, 0, s>>>(a)
         : rope_kernel<D, true, STORE, true><<<grid, block, 0, s>>>(a);
  else
    half ? rope_kernel<D, false, STORE, false><<<grid, block, 0, s>>>(a)
         : rope_kernel<D, true, STORE, false><<<grid, block, 0, s>>>(a);
}

// What both calls check and fill in: the rotation, the norm and the inputs.
rx_status fill(RopeArgs* a, const char* what, const rx_rope* rope, const rx_head_norm* norm,
               int32_t head_dim, const int32_t* d_positions, int64_t T, const void* d_q,
               int64_t q_stride, int32_t hq, const void* d_k, int64_t k_stride, int32_t hkv,
               void* d_q_out, int64_t q_out_stride) {
  static thread_local char buf[160];
  auto bad = [&](const char* why) {
    snprintf(buf, sizeof(buf), "%s: %s", what, why);
    return rx_internal::set_error(RX_ERR_INVALID, buf);
  };
  if (head_dim != 128 && head_dim != 256) return bad("head_dim must be 128 or 256");
  if (T < 0 || T > INT32_MAX) return bad("T < 0, or of 2^31 or more");
  if (hq < 0 || hkv < 0 || int64_t(hq) + 2 * int64_t(hkv) > INT32_MAX / 2)
    return bad("bad head counts");
  if (rope) {
    if (rope->rot_dim < 0 || rope->rot_dim > head_dim || rope->rot_dim % 2)
      return bad("rot_dim must be even and at most head_dim");
    if (rope->layout != RX_ROPE_HALF && rope->layout != RX_ROPE_INTERLEAVED)
      return bad("unknown pair layout");
    if (!isfinite(rope->magnitude)) return bad("the rotation's magnitude is not finite");
    a->rope = *rope;
  } else {
    a->rope.rot_dim = 0;
    a->rope.layout = RX_ROPE_INTERLEAVED;
    a->rope.magnitude = 1.f;
  }
  if (norm) {
    if (!(norm->eps >= 0.f) || !isfinite(norm->eps)) return bad("eps < 0 or not finite");
    if (!aligned16(norm->d_q_weight) || !aligned16(norm->d_k_weight))
      return bad("misaligned norm weight");
    a->q_weight = static_cast<const uint4*>(norm->d_q_weight);
    a->k_weight = static_cast<const uint4*>(norm->d_k_weight);
    a->eps = norm->eps;
    a->offset = norm->plus_one ? 1.f : 0.f;
  }
  if (T == 0) return RX_OK;
  if (!d_positions && a->rope.rot_dim > 0) return bad("NULL positions");
  if (hq && (!d_q || !d_q_out || !aligned16(d_q) || !aligned16(d_q_out)))
    return bad("NULL or misaligned queries");
  if (hkv && (!d_k || !aligned16(d_k))) return bad("NULL or misaligned keys");
  const int64_t qrow = int64_t(hq) * head_dim, krow = int64_t(hkv) * head_dim;
  if (hq && (q_stride < qrow || q_out_stride < qrow || q_stride % 8 || q_out_stride % 8))
    return bad("a query token stride is below Hq * head_dim or not a multiple of 8");
  if (hkv && (k_stride < krow || k_stride % 8))
    return bad("a key token stride is below Hkv * head_dim or not a multiple of 8");
  a->pos = d_positions;
  a->T = T;
  a->hq = hq;
  a->hkv = hkv;
  a->q = static_cast<const uint4*>(d_q);
  a->k = static_cast<const uint4*>(d_k);
  a->q_out = static_cast<uint4*>(d_q_out);
  a->q_stride = q_stride / 8;
  a->k_stride = k_stride / 8;
  a->q_out_stride = q_out_stride / 8;
  return RX_OK;
}

rx_status run(RopeArgs& a, int head_dim, bool store, const char* what, cudaStream_t s) {
  const int hpw = 32 / (head_dim / 16);
  const int heads = a.hq + a.hkv * (store ? 2 : 1);
  if (a.T == 0 || heads == 0) return RX_OK;
  // a warp a token when there are tokens for every SM's warps; fewer tokens are
  // bound by the latency of a warp's walk over its heads, so several share one
  const int64_t steps = (heads + hpw - 1) / hpw;
  const int64_t want = int64_t(rx_internal::sm_count()) * 32;
  a.split = int(std::min(steps, std::max<int64_t>(1, want / a.T)));
  const uintptr_t low = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                        reinterpret_cast<uintptr_t>(a.v) | reinterpret_cast<uintptr_t>(a.q_out) |
                        reinterpret_cast<uintptr_t>(a.k_out) |
                        reinterpret_cast<uintptr_t>(a.v_out) |
                        reinterpret_cast<uintptr_t>(a.q_weight) |
                        reinterpret_cast<uintptr_t>(a.k_weight) |
                        uintptr_t(16 * (a.q_stride | a.k_stride | a.v_stride | a.q_out_stride |
                                        (store ? 0 : a.k_out_stride)));
  a.whole = (low & 31) == 0;
  if (a.T * a.split > int64_t(INT32_MAX) * kWarps)
    return rx_internal::set_error(RX_ERR_INVALID, "rope: too many tokens");
  if (head_dim == 128)
    store ? launch<128, true>(a, s) : launch<128, false>(a, s);
  else
    store ? launch<256, true>(a, s) : launch<256, false>(a, s);
  return rx_internal::launch_status(what);
}

}  // namespace

namespace rx_internal {

int32_t rope_error_flags(bool clear) {
  int32_t v = 0;
  cudaMemcpyFromSymbol(&v, g_rope_error, sizeof(v));
  if (clear && v) {
    int32_t z = 0;
    cudaMemcpyToSymbol(g_rope_error, &z, sizeof(z));
  }
  return v;
}

}  // namespace rx_internal

extern "C" rx_status rx_rope_init(const rx_rope_config* cfg, rx_rope* out) {
  auto bad = [](const char* why) { return rx_internal::set_error(RX_ERR_INVALID, why); };
  if (!cfg || !out) return bad("rx_rope_init: NULL argument");
  const int rot = cfg->rot_dim, kind = cfg->scaling;
  if (rot < 0 || rot % 2 || rot > 2 * RX_ROPE_MAX_PAIRS)
    return bad("rx_rope_init: rot_dim must be even and at most 256");
  if (cfg->layout != RX_ROPE_HALF && cfg->layout != RX_ROPE_INTERLEAVED)
    return bad("rx_rope_init: unknown pair layout");
  if (cfg->reserved != 0) return bad("rx_rope_init: reserved must be 0");
  if (!(cfg->base > 1.0) || !isfinite(cfg->base)) return bad("rx_rope_init: base must be above 1");
  if (kind < RX_ROPE_SCALE_NONE || kind > RX_ROPE_SCALE_WAVELENGTH)
    return bad("rx_rope_init: unknown scaling");
  if (!isfinite(cfg->magnitude) || cfg->magnitude < 0.0)
    return bad("rx_rope_init: magnitude < 0 or not finite");
  const double s = kind == RX_ROPE_SCALE_NONE ? 1.0 : cfg->factor;
  if (!(s >= 1.0) || !isfinite(s)) return bad("rx_rope_init: factor must be at least 1");
  const bool ramp = kind == RX_ROPE_SCALE_PARTS || kind == RX_ROPE_SCALE_WAVELENGTH;
  if (ramp && !(cfg->original_len > 0.0 && isfinite(cfg->original_len) && cfg->low > 0.0 &&
                cfg->high > cfg->low && isfinite(cfg->high)))
    return bad("rx_rope_init: original_len > 0 and 0 < low < high are needed");
  constexpr double kTwoPi = 6.283185307179586476925;
  double base = cfg->base;
  if (kind == RX_ROPE_SCALE_BASE && rot > 2) base *= pow(s, double(rot) / (rot - 2));
  double first = 0.0, last = 0.0;
  if (kind == RX_ROPE_SCALE_PARTS) {
    auto pair = [&](double turns) {
      return rot * log(cfg->original_len / (turns * kTwoPi)) / (2.0 * log(base));
    };
    first = std::max(0.0, floor(pair(cfg->high)));
    last = std::min(double(rot - 1), ceil(pair(cfg->low)));
  }
  rx_rope r;
  memset(&r, 0, sizeof(r));
  for (int i = 0; i < rot / 2; ++i) {
    double f = pow(base, -2.0 * i / rot);
    if (kind == RX_ROPE_SCALE_LINEAR) {
      f /= s;
    } else if (kind == RX_ROPE_SCALE_PARTS) {
      const double w = std::min(1.0, std::max(0.0, (i - first) / std::max(last - first, 0.001)));
      f = f / s * w + f * (1.0 - w);
    } else if (kind == RX_ROPE_SCALE_WAVELENGTH) {
      const double turns = cfg->original_len * f / kTwoPi;
      const double w = std::min(1.0, std::max(0.0, (turns - cfg->low) / (cfg->high - cfg->low)));
      f = f / s * (1.0 - w) + f * w;
    }
    // f <= 1, so a position is less than a turn; the 64-bit fraction holds
    // every bit of the double down to f = 2^-9
    r.turns[i] = uint64_t(ldexp(f / kTwoPi, 64) + 0.5);
  }
  r.magnitude = float(cfg->magnitude > 0.0            ? cfg->magnitude
                      : kind == RX_ROPE_SCALE_PARTS   ? 0.1 * log(s) + 1.0
                                                      : 1.0);
  r.rot_dim = rot;
  r.layout = cfg->layout;
  *out = r;
  return RX_OK;
}

extern "C" rx_status rx_qk_rope(const rx_rope* rope, const rx_head_norm* norm, int32_t head_dim,
                                const int32_t* d_positions, int64_t T, const void* d_q,
                                int64_t q_stride, int32_t num_q_heads, const void* d_k,
                                int64_t k_stride, int32_t num_kv_heads, void* d_q_out,
                                int64_t q_out_stride, void* d_k_out, int64_t k_out_stride,
                                rx_stream_t stream) {
  RopeArgs a{};
  const rx_status st = fill(&a, "rx_qk_rope", rope, norm, head_dim, d_positions, T, d_q, q_stride,
                            num_q_heads, d_k, k_stride, num_kv_heads, d_q_out, q_out_stride);
  if (st != RX_OK || T == 0) return st;
  if (num_kv_heads && (!d_k_out || !aligned16(d_k_out)))
    return rx_internal::set_error(RX_ERR_INVALID, "rx_qk_rope: NULL or misaligned key output");
  if (num_kv_heads &&
      (k_out_stride < int64_t(num_kv_heads) * head_dim || k_out_stride % 8))
    return rx_internal::set_error(
        RX_ERR_INVALID,
        "rx_qk_rope: a key token stride is below Hkv * head_dim or not a multiple of 8");
  a.k_out = static_cast<uint4*>(d_k_out);
  a.k_out_stride = k_out_stride / 8;
  return run(a, head_dim, false, "rx_qk_rope", reinterpret_cast<cudaStream_t>(stream));
}

extern "C" rx_status rx_qkv_store(const rx_pool_desc* pool, int32_t layer, const rx_rope* rope,
                                  const rx_head_norm* norm, const int32_t* d_positions,
                                  const int32_t* d_slots, int64_t T, const void* d_q,
                                  int64_t q_stride, int32_t num_q_heads, const void* d_k,
                                  int64_t k_stride, const void* d_v, int64_t v_stride,
                                  void* d_q_out, int64_t q_out_stride, rx_stream_t stream) {
  rx_status st = rx_internal::check_pool(pool, layer);
  if (st != RX_OK) return st;
  const int32_t hkv = pool->num_kv_heads;
  RopeArgs a{};
  st = fill(&a, "rx_qkv_store", rope, norm, pool->head_dim, d_positions, T, d_q, q_stride,
            num_q_heads, d_k, k_stride, hkv, d_q_out, q_out_stride);
  if (st != RX_OK || T == 0) return st;
  if (!d_slots || !d_v || !aligned16(d_v))
    return rx_internal::set_error(RX_ERR_INVALID, "rx_qkv_store: NULL or misaligned input");
  if (v_stride < int64_t(hkv) * pool->head_dim || v_stride % 8)
    return rx_internal::set_error(
        RX_ERR_INVALID,
        "rx_qkv_store: a value token stride is below Hkv * head_dim or not a multiple of 8");
  const int64_t pieces = pool->head_dim / 8;
  a.head_stride = pool->num_slots * pieces;
  const int64_t off = int64_t(layer) * hkv * a.head_stride;
  a.slots = d_slots;
  a.num_slots = pool->num_slots;
  a.v = static_cast<const uint4*>(d_v);
  a.v_stride = v_stride / 8;
  a.k_out = static_cast<uint4*>(pool->k_pool) + off;
  a.v_out = static_cast<uint4*>(pool->v_pool) + off;
  return run(a, pool->head_dim, true, "rx_qkv_store", reinterpret_cast<cudaStream_t>(stream));
}
