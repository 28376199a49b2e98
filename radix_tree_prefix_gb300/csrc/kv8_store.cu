// The 8-bit KV pool's writes and reads: K and V rows quantised to e4m3 as
// they are stored (rx_kv8_store) and read back as bf16 (rx_kv8_load).
//
// A scale belongs to one KV head and one block of 1 .. 64 consecutive slots,
// and is a power of two: the least 2^e with amax <= 448 * 2^e over the
// block's rows.  e4m3 is a floating format, so a power-of-two scale costs no
// precision against amax / 448 (an element's rounding is relative, at most
// 2^-4 of it, down to amax * 2^-15), every division by it is exact, and
// rounding a block's rows again under a larger scale (a token appended to the
// block raised its amax) changes only the rows' smallest elements.
//
// Both kernels are bound by HBM: a row's bytes are read once and written once.
// One row of one head is D / 8 lanes of 16 B (bf16), so a row's maximum is a
// few shuffles and a row is loaded and stored in whole 128 B segments.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdio.h>

#include "kv8.cuh"
#include "rx.h"
#include "rx_internal.h"

// Bit 0: rx_kv8_store or rx_kv8_load met a slot outside [1, num_slots); bit
// 6: rx_kv8_store met a value that is not finite.  Read by rx_device_check().
static __device__ int32_t g_kv8_error;

namespace {

constexpr int kThreads = 256;
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
// takes one (token, head): its K row and its V row.
template <int D>
__global__ void __launch_bounds__(kThreads) store_rows_kernel(const StoreArgs a) {
  constexpr int L = D / 8;
  const int lane = threadIdx.x % L;
  const int64_t rows = a.T * a.hkv;
  const int64_t step = int64_t(gridDim.x) * (kThreads / L);
  // every lane of a warp runs every iteration (the shuffles need them all)
  for (int64_t base = int64_t(blockIdx.x) * (kThreads / L); base < rows; base += step) {
    const int64_t r = base + threadIdx.x / L;
    const bool in = r < rows;
    const int64_t t = in ? r / a.hkv : 0;
    const int64_t h = in ? r - t * a.hkv : 0;
    const int32_t slot = in ? __ldg(a.slots + t) : 0;
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (in) {
      k = __ldcs(a.k + r * L + lane);
      v = __ldcs(a.v + r * L + lane);
    }
    uint32_t km = reduce_max<L>(row_max(k));
    uint32_t vm = reduce_max<L>(row_max(v));
    if (__any_sync(0xffffffffu, km >= kInfBits || vm >= kInfBits)) {
      // a NaN is stored as 0 and an infinity as the row's largest code; the
      // scale comes from the finite values
      if (lane == 0 && (km >= kInfBits || vm >= kInfBits)) atomicOr(&g_kv8_error, 64);
      km = reduce_max<L>(row_max(drop(k, true)));
      vm = reduce_max<L>(row_max(drop(v, true)));
      k = drop(k, false);
      v = drop(v, false);
    }
    if (!in) continue;
    if (slot < 1 || slot >= a.num_slots) {  // never write outside the pool
      if (lane == 0) atomicOr(&g_kv8_error, 1);
      continue;
    }
    const int ke = kv8::scale_exponent(bf16_bits_to_float(km));
    const int ve = kv8::scale_exponent(bf16_bits_to_float(vm));
    const int64_t at = h * a.num_slots + slot;
    reinterpret_cast<uint2*>(a.kc + at * D)[lane] = quant8(k, kv8::pow2(-ke));
    reinterpret_cast<uint2*>(a.vc + at * D)[lane] = quant8(v, kv8::pow2(-ve));
    if (lane == 0) a.scales[at] = make_float2(kv8::pow2(ke), kv8::pow2(ve));
  }
}

// Blocks of 2 .. 64 slots.  The call's tokens of one block stand next to one
// another in slot order (a run); the block of a CTA takes a window of tokens
// and one of (head, K or V), lists the runs that start in the window, and a
// group of D / 8 lanes takes one run at a time: a pass for its maximum, the
// block's scale, the rows before the run rounded again if the scale grew,
// then a pass that quantises the run's rows (read again, from L1 or L2).
template <int D>
__global__ void __launch_bounds__(kThreads) store_runs_kernel(const StoreArgs a) {
  constexpr int L = D / 8;
  constexpr int GROUPS = kThreads / L;
  __shared__ int32_t starts[kThreads];
  __shared__ int count;
  const int tid = threadIdx.x;
  const int lane = tid % L;
  const int64_t w0 = int64_t(blockIdx.x) * a.window;
  const int h = blockIdx.y >> 1, which = blockIdx.y & 1;
  if (tid == 0) count = 0;
  __syncthreads();
  if (tid < a.window && w0 + tid < a.T) {
    const int64_t t = w0 + tid;
    const int32_t s = __ldg(a.slots + t);
    bool start = true;
    if (t > 0) {
      const int32_t p = __ldg(a.slots + t - 1);
      start = !(p >= 1 && s - 1 == p && (s >> a.block_log2) == (p >> a.block_log2));
    }
    if (s < 1 || s >= a.num_slots) {
      start = false;
      if (blockIdx.y == 0) atomicOr(&g_kv8_error, 1);
    }
    if (start) starts[atomicAdd(&count, 1)] = tid;
  }
  __syncthreads();
  const int n_runs = count;
  const uint4* src = (which ? a.v : a.k) + int64_t(h) * L + lane;
  const int64_t tok = int64_t(a.hkv) * L;  // uint4 per token
  uint8_t* codes = (which ? a.vc : a.kc) + int64_t(h) * a.num_slots * D;
  for (int i0 = 0; i0 < n_runs; i0 += GROUPS) {
    const int i = i0 + tid / L;
    const bool in = i < n_runs;
    const int64_t t0 = w0 + (in ? starts[i] : 0);
    const int32_t s0 = in ? __ldg(a.slots + t0) : 0;
    const int first = s0 & ((1 << a.block_log2) - 1);
    // the run ends with its block, its slots' order, the pool or the call
    int n = 0;
    if (in) {
      const int64_t room = min(int64_t((1 << a.block_log2) - first), a.num_slots - s0);
      const int most = int(min(room, a.T - t0));
      for (n = 1; n < most && __ldg(a.slots + t0 + n) == s0 + n; ++n) {
      }
    }
    uint32_t m = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) m = max2_nan(m, row_max(__ldg(src + (t0 + j) * tok)));
    m = reduce_max<L>(m);
    const bool bad = m >= kInfBits;
    if (__any_sync(0xffffffffu, bad)) {
      if (bad && lane == 0) atomicOr(&g_kv8_error, 64);
      m = 0;
      for (int j = 0; j < n; ++j) m = max2_nan(m, row_max(drop(__ldg(src + (t0 + j) * tok), true)));
      m = reduce_max<L>(m);
    }
    float scale = kv8::pow2(kv8::scale_exponent(bf16_bits_to_float(m)));
    float* sc = reinterpret_cast<float*>(
        a.scales + int64_t(h) * (a.num_slots >> a.block_log2) + (s0 >> a.block_log2)) + which;
    float old = in && first > 0 ? *sc : 0.f;
    __syncwarp();  // every lane has read the old scale before lane 0 writes
    if (!in) continue;
    // a scale that no store wrote (not positive and finite) counts as none
    if (!(old > 0.f && old < INFINITY)) old = 0.f;
    if (first > 0 && scale > old) {
      const float f = old / scale;
      uint2* row = reinterpret_cast<uint2*>(codes + int64_t(s0 - first) * D) + lane;
      for (int j = 0; j < first; ++j, row += L) {
        const uint2 c = *row;
        uint32_t q[4];
        const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = kv8::f16x2_to_float2(kv8::to_f16x2(w[e]));
          q[e] = kv8::to_e4m3x2(x.x * f, x.y * f);
        }
        *row = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      }
    } else if (first > 0) {
      scale = old;
    }
    if (lane == 0) *sc = scale;
    const float inv = 1.f / scale;
    uint2* row = reinterpret_cast<uint2*>(codes + int64_t(s0) * D) + lane;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      uint4 x = __ldg(src + (t0 + j) * tok);
      if (bad) x = drop(x, false);
      row[j * L] = quant8(x, inv);
    }
  }
}

// out[t][h] = bf16(code * scale), a lane for 16 codes of K and of V.
template <int D>
__global__ void __launch_bounds__(kThreads) load_kernel(const StoreArgs a, uint4* k_out,
                                                        uint4* v_out) {
  constexpr int L = D / 16;
  const int64_t total = a.T * a.hkv * L;
  for (int64_t c = int64_t(blockIdx.x) * kThreads + threadIdx.x; c < total;
       c += int64_t(gridDim.x) * kThreads) {
    const int64_t r = c / L;
    const int lane = int(c - r * L);
    const int64_t t = r / a.hkv;
    const int64_t h = r - t * a.hkv;
    const int32_t slot = __ldg(a.slots + t);
    uint4 kc = make_uint4(0, 0, 0, 0), vc = kc;
    float2 s = make_float2(0.f, 0.f);
    if (slot < 1 || slot >= a.num_slots) {  // never read outside the pool: a row of zeros
      if (lane == 0) atomicOr(&g_kv8_error, 1);
    } else {
      const int64_t at = h * a.num_slots + slot;
      kc = *(reinterpret_cast<const uint4*>(a.kc + at * D) + lane);
      vc = *(reinterpret_cast<const uint4*>(a.vc + at * D) + lane);
      s = a.scales[h * (a.num_slots >> a.block_log2) + (slot >> a.block_log2)];
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const uint4 x = which ? vc : kc;
      const float f = which ? s.y : s.x;
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 y =
            kv8::f16x2_to_float2(kv8::to_f16x2((e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu));
        const __nv_bfloat162 b = __floats2bfloat162_rn(y.x * f, y.y * f);
        o[e] = *reinterpret_cast<const uint32_t*>(&b);
      }
      uint4* dst = (which ? v_out : k_out) + r * (D / 8) + lane * 2;
      __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
      __stcs(dst + 1, make_uint4(o[4], o[5], o[6], o[7]));
    }
  }
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

rx_status store_args(const rx_kv8_pool_desc* pool, int32_t layer, const int32_t* d_slots,
                     const void* d_k, const void* d_v, int64_t T, StoreArgs* a) {
  rx_status st = rx_internal::check_kv8_pool(pool, layer);
  if (st != RX_OK) return st;
  if (T < 0) return rx_internal::set_error(RX_ERR_INVALID, "8-bit KV store or load: T < 0");
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
    return set_error(RX_ERR_INVALID, "8-bit pool has 2^31 rows (layers x KV heads x slots) or more");
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

extern "C" rx_status rx_kv8_store(const rx_kv8_pool_desc* pool, int32_t layer,
                                  const int32_t* d_slots, const void* d_k, const void* d_v,
                                  int64_t T, rx_stream_t stream) {
  StoreArgs a;
  rx_status st = store_args(pool, layer, d_slots, d_k, d_v, T, &a);
  if (st != RX_OK || T == 0) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int D = pool->head_dim;
  const int64_t sms = rx_internal::sm_count();
  if (pool->block == 1) {
    const int64_t per_cta = kThreads / (D / 8);
    int64_t ctas = (T * a.hkv + per_cta - 1) / per_cta;
    if (ctas > sms * 8) ctas = sms * 8;
    if (D == 128)
      store_rows_kernel<128><<<unsigned(ctas), kThreads, 0, s>>>(a);
    else
      store_rows_kernel<256><<<unsigned(ctas), kThreads, 0, s>>>(a);
  } else {
    if (a.hkv > 32767)
      return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_store: too many KV heads");
    // long windows keep every group of a CTA in whole blocks; short ones
    // spread a decode step's tokens (one run each) over the SMs
    a.window = T * a.hkv * 2 >= 2 * sms * kThreads ? kThreads : 16;
    const int64_t gx = (T + a.window - 1) / a.window;
    if (gx > INT32_MAX) return rx_internal::set_error(RX_ERR_INVALID, "rx_kv8_store: T too large");
    const dim3 grid(unsigned(gx), unsigned(a.hkv * 2));
    if (D == 128)
      store_runs_kernel<128><<<grid, kThreads, 0, s>>>(a);
    else
      store_runs_kernel<256><<<grid, kThreads, 0, s>>>(a);
  }
  return rx_internal::launch_status("rx_kv8_store");
}

extern "C" rx_status rx_kv8_load(const rx_kv8_pool_desc* pool, int32_t layer,
                                 const int32_t* d_slots, void* d_k, void* d_v, int64_t T,
                                 rx_stream_t stream) {
  StoreArgs a;
  rx_status st = store_args(pool, layer, d_slots, d_k, d_v, T, &a);
  if (st != RX_OK || T == 0) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int D = pool->head_dim;
  int64_t ctas = (T * a.hkv * (D / 16) + kThreads - 1) / kThreads;
  const int64_t cap = int64_t(rx_internal::sm_count()) * 8;
  if (ctas > cap) ctas = cap;
  if (D == 128)
    load_kernel<128><<<unsigned(ctas), kThreads, 0, s>>>(a, static_cast<uint4*>(d_k),
                                                         static_cast<uint4*>(d_v));
  else
    load_kernel<256><<<unsigned(ctas), kThreads, 0, s>>>(a, static_cast<uint4*>(d_k),
                                                         static_cast<uint4*>(d_v));
  return rx_internal::launch_status("rx_kv8_load");
}
