// The 8-bit KV pool's writes and reads: K and V rows quantised to e4m3 as
// they are stored (rx_kv8_store) and read back as bf16 (rx_kv8_load).
//
// A scale belongs to one KV head and one block of 1 .. 64 consecutive slots,
// and is a power of two: the least 2^e with amax <= 448 * 2^e over the
// block's rows.  e4m3 is a floating format, so a power-of-two scale costs no
// precision against amax / 448 (an element's rounding is relative, at most
// 2^-4 of it, down to 2^-6 of the scale, which is amax * 2^-14.8 to amax * 2^-13.8
// as amax is above 224 scales), every division by it is exact, and
// rounding a block's rows again under a larger scale (a token appended to the
// block raised its amax) changes only the rows' smallest elements.
//
// Both kernels are bound by HBM: a row's bytes are read once and written once.
// One row of one head is D / 8 lanes of 16 B (bf16), so a row's maximum is a
// few shuffles and a row is loaded and stored in whole 128 B segments.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdio.h>

#include <algorithm>

#include "kv8.cuh"
#include "ptx_util.cuh"
#include "rx.h"
#include "rx_internal.h"

// Bit 0: rx_kv8_store or rx_kv8_load met a slot outside [1, num_slots); bit
// 6: rx_kv8_store met a value that is not finite; bit 7: it met a block's tokens
// out of slot order.  Read by rx_device_check().
static __device__ int32_t g_kv8_error;

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 2;  // rows of a group of lanes (rows of blocks of one slot, loads)
constexpr uint32_t kInfBits = 0x7f80u;  // bf16 infinity; larger magnitudes are NaN

__device__ __forceinline__ uint32_t abs2(uint32_t x) { return x & 0x7fff7fffu; }
// The larger bf16 of each half, a NaN if either is one.
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t row_max(uint4 x) {
  return max2_nan(max2_nan(abs2(x.x), abs2(x.y)), max2_nan(abs2(x.z), abs2(x.w)));
}
// Largest magnitude (bf16 bits) over the L lanes of a row and both halves.
template <int L>
__device__ __forceinline__ uint32_t reduce_max(uint32_t m) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) m = max2_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  m = max2_nan(m, m >> 16);
  return m & 0xffffu;
}
// 0 in place of a NaN; `inf_too`: also in place of an infinity.
__device__ __forceinline__ uint32_t drop2(uint32_t x, bool inf_too) {
  const uint32_t lo = x & 0x7fffu, hi = (x >> 16) & 0x7fffu;
  if (lo > kInfBits || (inf_too && lo == kInfBits)) x &= 0xffff0000u;
  if (hi > kInfBits || (inf_too && hi == kInfBits)) x &= 0x0000ffffu;
  return x;
}
__device__ __forceinline__ uint4 drop(uint4 x, bool inf_too) {
  return make_uint4(drop2(x.x, inf_too), drop2(x.y, inf_too), drop2(x.z, inf_too),
                    drop2(x.w, inf_too));
}
__device__ __forceinline__ float bf16_bits_to_float(uint32_t b) { return __uint_as_float(b << 16); }

__device__ __forceinline__ uint32_t quant4(uint32_t a, uint32_t b, float inv) {
  const uint32_t lo = kv8::to_e4m3x2(__uint_as_float(a << 16) * inv,
                                     __uint_as_float(a & 0xffff0000u) * inv);
  const uint32_t hi = kv8::to_e4m3x2(__uint_as_float(b << 16) * inv,
                                     __uint_as_float(b & 0xffff0000u) * inv);
  return lo | (hi << 16);
}
__device__ __forceinline__ uint2 quant8(uint4 x, float inv) {
  return make_uint2(quant4(x.x, x.y, inv), quant4(x.z, x.w, inv));
}

struct StoreArgs {
  uint8_t* kc;  // layer base, [Hkv][num_slots][D]
  uint8_t* vc;
  float2* scales;  // layer base, [Hkv][num_slots / block]
  const int32_t* slots;
  const uint4* k;  // [T][Hkv][D] bf16
  const uint4* v;
  int64_t T;
  int64_t num_slots;
  int hkv;
  int block_log2;
  int window;
};

// One slot a block: every row has its own scale.  A group of D / 8 lanes
// takes kRows (token, head) rows, their K and V on their way together.  Two rows
// and a grid of one pass: 8,017 tokens x 8 heads x 128 in 7.8 us in a graph, 10.4
// call after call (one row and CTAs that loop, 9.1 in a graph).
template <int D>
__global__ void __launch_bounds__(kThreads) store_rows_kernel(const StoreArgs a) {
  constexpr int L = D / 8;
  constexpr int GROUPS = kThreads / L;
  const int lane = threadIdx.x % L;
  const int64_t rows = a.T * a.hkv;
  const int64_t base = int64_t(blockIdx.x) * (GROUPS * kRows) + threadIdx.x / L;
  rxk::griddep_launch_dependents();
  rxk::griddep_wait();  // (a chained launch: the kernels before read the pool)
  uint4 k[kRows], v[kRows];
  int32_t slot[kRows];
  int h[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t r = base + j * GROUPS;
    const bool in = r < rows;
    // (fewer than 2^31 rows: checked on the host)
    const uint32_t t = in ? uint32_t(r) / uint32_t(a.hkv) : 0;
    h[j] = in ? int(uint32_t(r) - t * uint32_t(a.hkv)) : -1;
    slot[j] = in ? __ldg(a.slots + t) : 0;
    k[j] = v[j] = make_uint4(0, 0, 0, 0);
    if (in) {
      k[j] = __ldcs(a.k + r * L + lane);
      v[j] = __ldcs(a.v + r * L + lane);
    }
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    uint32_t km = reduce_max<L>(row_max(k[j]));
    uint32_t vm = reduce_max<L>(row_max(v[j]));
    if (__any_sync(0xffffffffu, km >= kInfBits || vm >= kInfBits)) {
      // a NaN is stored as 0 and an infinity as the row's largest code; the
      // scale comes from the finite values
      if (lane == 0 && (km >= kInfBits || vm >= kInfBits)) atomicOr(&g_kv8_error, 64);
      km = reduce_max<L>(row_max(drop(k[j], true)));
      vm = reduce_max<L>(row_max(drop(v[j], true)));
      k[j] = drop(k[j], false);
      v[j] = drop(v[j], false);
    }
    if (h[j] < 0) continue;
    if (slot[j] < 1 || slot[j] >= a.num_slots) {  // never write outside the pool
      if (lane == 0) atomicOr(&g_kv8_error, 1);
      continue;
    }
    const int ke = kv8::scale_exponent(bf16_bits_to_float(km));
    const int ve = kv8::scale_exponent(bf16_bits_to_float(vm));
    const int64_t at = int64_t(h[j]) * a.num_slots + slot[j];
    reinterpret_cast<uint2*>(a.kc + at * D)[lane] = quant8(k[j], kv8::pow2(-ke));
    reinterpret_cast<uint2*>(a.vc + at * D)[lane] = quant8(v[j], kv8::pow2(-ve));
    if (lane == 0) a.scales[at] = make_float2(kv8::pow2(ke), kv8::pow2(ve));
  }
}

// Blocks of 2 .. 64 slots.  The call's tokens of one block stand next to one
// another in slot order (a run); the CTA takes a window of tokens and one of
// (head, K or V), lists the runs that start in the window, and a group of D / 8
// lanes takes one run at a time: its maximum, the block's scale, the rows
// before the run rounded again if the scale grew, then the run's codes.
// Up to kHold rows stay in registers between the two passes, all of them on
// their way at once; the rows of a longer run are read again, from L1 or L2.
// 51,200 tokens x 4 heads x 256 in blocks of 16: 62 us with L2 flushed, 5.1 TB/s
// (every row read twice and a run's slots one after the other, 82.6), 57.4 call
// after call.
constexpr int kHold = 16;
constexpr int kMaxBlock = 64;
constexpr int kMaxWindow = 1024;
template <int D>
__global__ void __launch_bounds__(kThreads) store_runs_kernel(const StoreArgs a) {
  constexpr int L = D / 8;
  constexpr int GROUPS = kThreads / L;
  __shared__ int32_t win[kMaxWindow + kMaxBlock + 1];  // slots of tokens w0 - 1 ..
  __shared__ int32_t starts[kMaxWindow];
  __shared__ int count;
  const int tid = threadIdx.x;
  const int lane = tid % L;
  const int64_t w0 = int64_t(blockIdx.x) * a.window;
  const int h = blockIdx.y >> 1, which = blockIdx.y & 1;
  const int blk = 1 << a.block_log2;
  if (tid == 0) count = 0;
  rxk::griddep_launch_dependents();
  rxk::griddep_wait();  // (a chained launch: the kernels before read the pool)
  for (int i = tid; i < a.window + blk + 1; i += kThreads) {
    const int64_t t = w0 - 1 + i;
    win[i] = t >= 0 && t < a.T ? __ldg(a.slots + t) : -1;  // -1 is in no run
  }
  __syncthreads();
  for (int i = tid; i < a.window && w0 + i < a.T; i += kThreads) {
    const int32_t s = win[i + 1], p = win[i];
    if (s < 1 || s >= a.num_slots) {
      if (blockIdx.y == 0) atomicOr(&g_kv8_error, 1);
    } else if (p < 1 || p >= a.num_slots || (s >> a.block_log2) != (p >> a.block_log2)) {
      starts[atomicAdd(&count, 1)] = i;  // (the order of the runs changes no result)
    } else if (s - 1 != p && blockIdx.y == 0) {
      atomicOr(&g_kv8_error, 128);  // two runs of one block would race: the later one is skipped
    }
  }
  __syncthreads();
  const int n_runs = count;
  const uint4* src = (which ? a.v : a.k) + int64_t(h) * L + lane;
  const int64_t tok = int64_t(a.hkv) * L;  // uint4 per token
  uint8_t* codes = (which ? a.vc : a.kc) + int64_t(h) * a.num_slots * D;
  for (int i0 = 0; i0 < n_runs; i0 += GROUPS) {
    const int i = i0 + tid / L;
    const bool in = i < n_runs;
    const int at = in ? starts[i] : 0;
    const int64_t t0 = w0 + at;
    const int32_t s0 = in ? win[at + 1] : 0;
    const int first = s0 & (blk - 1);
    // the run ends with its block (so within the pool), its slots' order or the
    // call: the group's lanes look at L tokens together
    int n = 0;
    for (int j0 = 0; j0 < blk; j0 += L) {
      const int j = j0 + lane;
      const bool ok = in && j < blk - first && win[at + 1 + j] == s0 + j;
      uint32_t bits = __ballot_sync(0xffffffffu, ok);
      if (L < 32) bits = (bits >> ((tid & 31) / L * L)) & ((1u << (L & 31)) - 1);
      if (n == j0) n += bits == 0xffffffffu ? 32 : __ffs(~bits) - 1;
    }
    float* sc = reinterpret_cast<float*>(
        a.scales + int64_t(h) * (a.num_slots >> a.block_log2) + (s0 >> a.block_log2)) + which;
    float old = in && first > 0 ? *sc : 0.f;
    const uint4* row0 = src + t0 * tok;
    uint4 x[kHold];
#pragma unroll
    for (int j = 0; j < kHold; ++j)
      x[j] = j < n ? __ldg(row0 + j * tok) : make_uint4(0, 0, 0, 0);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kHold; ++j) m = max2_nan(m, row_max(x[j]));
#pragma unroll 8
    for (int j = kHold; j < n; ++j) m = max2_nan(m, row_max(__ldg(row0 + j * tok)));
    m = reduce_max<L>(m);
    const bool bad = m >= kInfBits;
    if (__any_sync(0xffffffffu, bad)) {
      if (bad && lane == 0) atomicOr(&g_kv8_error, 64);
      m = 0;
      for (int j = 0; j < n; ++j) m = max2_nan(m, row_max(drop(__ldg(row0 + j * tok), true)));
      m = reduce_max<L>(m);
#pragma unroll
      for (int j = 0; j < kHold; ++j) x[j] = drop(x[j], false);
    }
    float scale = kv8::pow2(kv8::scale_exponent(bf16_bits_to_float(m)));
    __syncwarp();  // every lane has read the old scale before lane 0 writes
    if (!in) continue;
    // a scale that no store wrote (not positive and finite) counts as none
    if (!(old > 0.f && old < INFINITY)) old = 0.f;
    if (first > 0 && scale > old) {
      const float f = old / scale;
      uint2* row = reinterpret_cast<uint2*>(codes + int64_t(s0 - first) * D) + lane;
      for (int j0 = 0; j0 < first; j0 += 8) {
        uint2 c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < first) c[j] = row[(j0 + j) * L];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j0 + j >= first) break;
          uint32_t q[4];
          const uint32_t w[4] = {c[j].x & 0xffffu, c[j].x >> 16, c[j].y & 0xffffu, c[j].y >> 16};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = kv8::f16x2_to_float2(kv8::to_f16x2(w[e]));
            q[e] = kv8::to_e4m3x2(y.x * f, y.y * f);
          }
          row[(j0 + j) * L] = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        }
      }
    } else if (first > 0) {
      scale = old;
    }
    if (lane == 0) *sc = scale;
    const float inv = 1.f / scale;
    uint2* row = reinterpret_cast<uint2*>(codes + int64_t(s0) * D) + lane;
#pragma unroll
    for (int j = 0; j < kHold; ++j)
      if (j < n) row[j * L] = quant8(x[j], inv);
#pragma unroll 4
    for (int j = kHold; j < n; ++j) {
      uint4 y = __ldg(row0 + j * tok);
      if (bad) y = drop(y, false);
      row[j * L] = quant8(y, inv);
    }
  }
}

// out[t][h] = bf16(code * scale), a lane for 8 codes of K and of V (a store
// instruction of a warp then fills whole sectors), kRows rows of a thread on
// their way together.  32,768 tokens x 8 heads x 128, L2 flushed: 37.5 us, 5.4
// TB/s (four rows and CTAs that loop, 41.6; a lane for 16 codes, whose stores
// fill half a sector each, 49.9).
template <int D>
__global__ void __launch_bounds__(kThreads) load_kernel(const StoreArgs a, uint4* k_out,
                                                        uint4* v_out) {
  constexpr int L = D / 8;
  constexpr int GROUPS = kThreads / L;
  const int lane = threadIdx.x % L;
  const int64_t rows = a.T * a.hkv;
  const int64_t r0 = int64_t(blockIdx.x) * (GROUPS * kRows) + threadIdx.x / L;
  uint2 kc[kRows], vc[kRows];
  float2 s[kRows];
  int32_t slot[kRows];
  int h[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t r = r0 + j * GROUPS;
    // (fewer than 2^31 rows: checked on the host)
    const uint32_t t = r < rows ? uint32_t(r) / uint32_t(a.hkv) : 0;
    h[j] = r < rows ? int(uint32_t(r) - t * uint32_t(a.hkv)) : 0;
    slot[j] = r < rows ? __ldg(a.slots + t) : 1;
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    kc[j] = vc[j] = make_uint2(0, 0);
    s[j] = make_float2(0.f, 0.f);
    if (slot[j] < 1 || slot[j] >= a.num_slots) {  // never read outside the pool: zeros
      if (lane == 0) atomicOr(&g_kv8_error, 1);
    } else if (r0 + j * GROUPS < rows) {
      const int64_t at = int64_t(h[j]) * a.num_slots + slot[j];
      kc[j] = *(reinterpret_cast<const uint2*>(a.kc + at * D) + lane);
      vc[j] = *(reinterpret_cast<const uint2*>(a.vc + at * D) + lane);
      s[j] = a.scales[int64_t(h[j]) * (a.num_slots >> a.block_log2) +
                      (slot[j] >> a.block_log2)];
    }
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t r = r0 + j * GROUPS;
    if (r >= rows) break;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const uint2 x = which ? vc[j] : kc[j];
      const float f = which ? s[j].y : s[j].x;
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = e & 2 ? x.y : x.x;
        const float2 y = kv8::f16x2_to_float2(kv8::to_f16x2((e & 1) ? w >> 16 : w & 0xffffu));
        const __nv_bfloat162 b = __floats2bfloat162_rn(y.x * f, y.y * f);
        o[e] = *reinterpret_cast<const uint32_t*>(&b);
      }
      __stcs((which ? v_out : k_out) + r * L + lane, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

rx_status store_args(const rx_kv8_pool_desc* pool, int32_t layer, const int32_t* d_slots,
                     const void* d_k, const void* d_v, int64_t T, StoreArgs* a) {
  rx_status st = rx_internal::check_kv8_pool(pool, layer);
  if (st != RX_OK) return st;
  if (T < 0) return rx_internal::set_error(RX_ERR_INVALID, "8-bit KV store or load: T < 0");
  if (T > INT32_MAX / pool->num_kv_heads)
    return rx_internal::set_error(RX_ERR_INVALID,
                                  "8-bit KV store or load: 2^31 rows (T x KV heads) or more");
  if (T > 0 && (!d_slots || !d_k || !d_v || !aligned(d_k, 16) || !aligned(d_v, 16)))
    return rx_internal::set_error(RX_ERR_INVALID,
                                  "8-bit KV store or load: NULL or misaligned rows or slots");
  const int64_t head_rows = int64_t(layer) * pool->num_kv_heads;
  int lg = 0;
  while ((1 << lg) < pool->block) ++lg;
  a->kc = static_cast<uint8_t*>(pool->k_codes) + head_rows * pool->num_slots * pool->head_dim;
  a->vc = static_cast<uint8_t*>(pool->v_codes) + head_rows * pool->num_slots * pool->head_dim;
  a->scales = reinterpret_cast<float2*>(pool->scales) + head_rows * (pool->num_slots >> lg);
  a->slots = d_slots;
  a->k = static_cast<const uint4*>(d_k);
  a->v = static_cast<const uint4*>(d_v);
  a->T = T;
  a->num_slots = pool->num_slots;
  a->hkv = pool->num_kv_heads;
  a->block_log2 = lg;
  a->window = 0;
  return RX_OK;
}

}  // namespace

namespace rx_internal {

rx_status check_kv8_pool(const rx_kv8_pool_desc* pool, int32_t layer) {
  if (!pool || !pool->k_codes || !pool->v_codes || !pool->scales)
    return set_error(RX_ERR_INVALID, "8-bit pool descriptor or pool pointer is NULL");
  if (pool->head_dim != 128 && pool->head_dim != 256)
    return set_error(RX_ERR_INVALID, "head_dim must be 128 or 256");
  if (pool->num_kv_heads <= 0 || pool->num_layers <= 0 || pool->num_slots < 2)
    return set_error(RX_ERR_INVALID, "8-bit pool shape invalid");
  if (pool->block < 1 || pool->block > 64 || (pool->block & (pool->block - 1)) ||
      pool->num_slots % pool->block)
    return set_error(RX_ERR_INVALID,
                     "8-bit pool: block must be a power of two up to 64 that divides num_slots");
  // the attention kernels address pool rows with 32-bit TMA coordinates
  if (pool->num_slots > INT32_MAX ||
      int64_t(pool->num_layers) * pool->num_kv_heads > INT32_MAX / pool->num_slots)
    return set_error(RX_ERR_INVALID,
                     "8-bit pool has 2^31 rows (layers x KV heads x slots) or more");
  if (layer < 0 || layer >= pool->num_layers)
    return set_error(RX_ERR_INVALID, "layer out of range");
  if (!aligned(pool->k_codes, 16) || !aligned(pool->v_codes, 16) || !aligned(pool->scales, 8))
    return set_error(RX_ERR_INVALID,
                     "8-bit pool codes must be 16-byte aligned, scales 8-byte aligned");
  return RX_OK;
}

int32_t kv8_store_error_flags(bool clear) {
  int32_t v = 0;
  cudaMemcpyFromSymbol(&v, g_kv8_error, sizeof(v));
  if (clear && v) {
    int32_t z = 0;
    cudaMemcpyToSymbol(g_kv8_error, &z, sizeof(z));
  }
  return v;
}

}  // namespace rx_internal

rx_status rx_internal::kv8_store(const rx_kv8_pool_desc* pool, int32_t layer,
                                 const int32_t* d_slots, const void* d_k, const void* d_v,
                                 int64_t T, rx_stream_t stream, bool chained) {
  StoreArgs a;
  rx_status st = store_args(pool, layer, d_slots, d_k, d_v, T, &a);
  if (st != RX_OK || T == 0) return st;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = chained ? 1 : 0;
  const int D = pool->head_dim;
  const int64_t sms = rx_internal::sm_count();
  if (pool->block == 1) {
    const int64_t per_cta = kThreads / (D / 8) * kRows;
    const int64_t ctas = (T * a.hkv + per_cta - 1) / per_cta;
    cfg.gridDim = dim3(unsigned(ctas));
    cudaLaunchKernelEx(&cfg, D == 128 ? store_rows_kernel<128> : store_rows_kernel<256>, a);
  } else {
    if (a.hkv > 32767)
      return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_store: too many KV heads");
    // a window of as many blocks as the CTA has groups keeps every group at
    // whole blocks; a call too short to fill the SMs so has a token (a decode
    // step: one run each) per group
    const int groups = kThreads / (D / 8);
    const int64_t whole = std::min<int64_t>(int64_t(groups) << a.block_log2, kMaxWindow);
    a.window = int((T + whole - 1) / whole * a.hkv * 2 >= 2 * sms ? whole : groups);
    const int64_t gx = (T + a.window - 1) / a.window;
    if (gx > INT32_MAX) return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_store: T too large");
    cfg.gridDim = dim3(unsigned(gx), unsigned(a.hkv * 2));
    cudaLaunchKernelEx(&cfg, D == 128 ? store_runs_kernel<128> : store_runs_kernel<256>, a);
  }
  return rx_internal::launch_status("rx_kv8_store");
}

extern "C" rx_status rx_kv8_store(const rx_kv8_pool_desc* pool, int32_t layer,
                                  const int32_t* d_slots, const void* d_k, const void* d_v,
                                  int64_t T, rx_stream_t stream) {
  return rx_internal::kv8_store(pool, layer, d_slots, d_k, d_v, T, stream, false);
}

extern "C" rx_status rx_kv8_load(const rx_kv8_pool_desc* pool, int32_t layer,
                                 const int32_t* d_slots, void* d_k, void* d_v, int64_t T,
                                 rx_stream_t stream) {
  StoreArgs a;
  rx_status st = store_args(pool, layer, d_slots, d_k, d_v, T, &a);
  if (st != RX_OK || T == 0) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int D = pool->head_dim;
  const int64_t per_cta = kThreads / (D / 8) * kRows;
  const int64_t ctas = (T * a.hkv + per_cta - 1) / per_cta;
  if (D == 128)
    load_kernel<128><<<unsigned(ctas), kThreads, 0, s>>>(a, static_cast<uint4*>(d_k),
                                                         static_cast<uint4*>(d_v));
  else
    load_kernel<256><<<unsigned(ctas), kThreads, 0, s>>>(a, static_cast<uint4*>(d_k),
                                                         static_cast<uint4*>(d_v));
  return rx_internal::launch_status("rx_kv8_load");
}
