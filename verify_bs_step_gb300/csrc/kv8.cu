// Writing and reading an 8-bit paged K/V cache (sm_103a).
//
// Every (page, layer, k/v, head) run of `block` x D codes has one scale 2^e: with amax the
// largest magnitude of the run's finite values, e is the smallest integer with amax <= QMAX 2^e
// (QMAX 127 for int8, 448 for e4m3), and a value x is held as the code nearest to x 2^-e.
// A power of two keeps the scaling exact, so a code carries one rounding, and it lets a page
// grow token by token: when a new token needs a larger scale, the codes already there move to
// it by an exact power of two and one more rounding, each at least twice as coarse as the one
// before, so all of them together stay below one step of the final scale.
//
// A warp owns one run of consecutive tokens in one page, for one head of K or of V.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv8.h"

namespace vbs {

constexpr int KV8_NT = 256;

template <int FMT> struct Code;
template <> struct Code<VBS_I8> {
  static constexpr float TOP = 0.9921875f;          // QMAX = TOP 2^BITS
  static constexpr int BITS = 7;
  __device__ static __forceinline__ uint8_t enc(float x) {
    x = fminf(fmaxf(x, -127.f), 127.f);             // NaN becomes -127 here: the caller has dealt with it
    return static_cast<uint8_t>(static_cast<int8_t>(__float2int_rn(x)));
  }
  __device__ static __forceinline__ float dec(uint8_t c) { return static_cast<float>(static_cast<int8_t>(c)); }
};
template <> struct Code<VBS_E4M3> {
  static constexpr float TOP = 0.875f;
  static constexpr int BITS = 9;
  __device__ static __forceinline__ uint8_t enc(float x) {
    return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
  }
  __device__ static __forceinline__ float dec(uint8_t c) {
    __nv_fp8_e4m3 f;
    f.__x = c;
    return static_cast<float>(f);
  }
};

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exp2i(float s) { return (__float_as_int(s) >> 23) - 127; }   // of a power of two

// The smallest e with amax <= TOP 2^BITS 2^e, clamped (amax finite, >= 0).
template <int FMT> __device__ __forceinline__ int scale_exp(float amax) {
  int x = 0;
  const float m = frexpf(amax, &x);
  const int e = x - Code<FMT>::BITS + (m > Code<FMT>::TOP ? 1 : 0);
  return amax > 0.f ? max(KV8_E_LO, min(KV8_E_HI, e)) : KV8_E_LO;
}

// True if token i continues the page run of token i - 1.
__device__ __forceinline__ bool continues(const int64_t* slots, int64_t i, int64_t s, int block) {
  return i > 0 && s % block != 0 && slots[i - 1] == s - 1;
}

template <int FMT, typename T>
__global__ void __launch_bounds__(KV8_NT) kv8_append_kernel(const Kv8Geom g, const Kv8Src src, int64_t n,
                                                            const int64_t* __restrict__ slots) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * KV8_NT + threadIdx.x) >> 5;
  if (item >= n * 2 * g.H) return;
  const int64_t i = item / (2 * g.H);
  const int kv = static_cast<int>(item % (2 * g.H)) / g.H, h = static_cast<int>(item % g.H);
  const int64_t s = slots[i];
  if (s < 0) return;
  if (s >= g.NB * g.block) {                        // not a slot of this cache: nothing is written
    if (lane == 0) set_status(g.status, VBS_EINVAL);
    return;
  }
  if (continues(slots, i, s, g.block)) return;
  const int64_t page = s / g.block;
  const int off = static_cast<int>(s - page * g.block);
  int len = 1;
  while (off + len < g.block && i + len < n && slots[i + len] == s + len) ++len;

  const void* base = kv ? src.v : src.k;
  const int64_t tok = kv ? src.v_tok : src.k_tok;
  const int64_t p0 = i * tok + h * (kv ? src.v_head : src.k_head);
  float amax = 0.f;
  bool odd = false;
  for (int t = 0; t < len; ++t)
    for (int d = lane; d < g.D; d += 32) {
      const float x = fabsf(Elem<T>::load(base, p0 + t * tok + d));
      if (x <= 3.402823466e38f) amax = fmaxf(amax, x);
      else odd = true;                              // NaN or infinity
    }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, m));
  if (odd) set_status(g.status, VBS_EINPUT);
  int e = scale_exp<FMT>(amax);
  const int64_t run = g.run(page, kv, h);
  uint8_t* codes = reinterpret_cast<uint8_t*>(g.pool) + run * g.block * g.D;
  if (off > 0) {
    const int e_old = exp2i(g.scales[run]);
    if (e_old < e) {
      const float f = e_old - e < -126 ? 0.f : pow2i(e_old - e);
      for (int d = lane; d < off * g.D; d += 32) codes[d] = Code<FMT>::enc(Code<FMT>::dec(codes[d]) * f);
    } else {
      e = e_old;
    }
    __syncwarp();
  }
  const float inv = pow2i(-e);
  for (int t = 0; t < len; ++t)
    for (int d = lane; d < g.D; d += 32) {
      const float x = Elem<T>::load(base, p0 + t * tok + d);
      codes[(off + t) * g.D + d] = x == x ? Code<FMT>::enc(x * inv) : 0;
    }
  if (lane == 0) g.scales[run] = pow2i(e);
}

template <int FMT>
__global__ void __launch_bounds__(KV8_NT) kv8_read_kernel(const Kv8Geom g, int64_t n, const int64_t* __restrict__ slots,
                                                          uint16_t* k_out, uint16_t* v_out) {
  const int per = g.D / 16;
  const int64_t total = n * 2 * g.H * per;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * KV8_NT + threadIdx.x; x < total;
       x += static_cast<int64_t>(gridDim.x) * KV8_NT) {
    const int c = static_cast<int>(x % per);
    const int64_t y = x / per;
    const int h = static_cast<int>(y % g.H);
    const int64_t z = y / g.H;
    const int kv = static_cast<int>(z & 1);
    const int64_t i = z >> 1;
    const int64_t s = slots[i];
    uint4 q = make_uint4(0, 0, 0, 0);
    float sc = 0.f;
    if (s >= 0 && s < g.NB * g.block) {
      const int64_t page = s / g.block, run = g.run(page, kv, h);
      q = *reinterpret_cast<const uint4*>(g.pool + (run * g.block + (s - page * g.block)) * g.D + c * 16);
      sc = g.scales[run];
    } else if (s >= 0) {
      set_status(g.status, VBS_EINVAL);
    }
    const uint8_t* b = reinterpret_cast<const uint8_t*>(&q);
    __nv_bfloat162 o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)                     // exact: a code has at most 7 bits
      o[j] = __floats2bfloat162_rn(Code<FMT>::dec(b[2 * j]) * sc, Code<FMT>::dec(b[2 * j + 1]) * sc);
    uint4* dst = reinterpret_cast<uint4*>((kv ? v_out : k_out) + (i * g.H + h) * g.D + c * 16);
    dst[0] = reinterpret_cast<const uint4*>(o)[0];
    dst[1] = reinterpret_cast<const uint4*>(o)[1];
  }
}

int launch_kv8_append(const Kv8Geom& g, const Kv8Src& src, int64_t n, const int64_t* slots, int, cudaStream_t s) {
  if (n == 0) return VBS_OK;
  const int64_t grid = (n * 2 * g.H + KV8_NT / 32 - 1) / (KV8_NT / 32);
  if (grid >= (int64_t{1} << 31)) return VBS_EINVAL;
  const unsigned gr = static_cast<unsigned>(grid);
  if (g.fmt == VBS_I8) {
    if (src.dtype == VBS_BF16) kv8_append_kernel<VBS_I8, bf16_t><<<gr, KV8_NT, 0, s>>>(g, src, n, slots);
    else kv8_append_kernel<VBS_I8, float><<<gr, KV8_NT, 0, s>>>(g, src, n, slots);
  } else {
    if (src.dtype == VBS_BF16) kv8_append_kernel<VBS_E4M3, bf16_t><<<gr, KV8_NT, 0, s>>>(g, src, n, slots);
    else kv8_append_kernel<VBS_E4M3, float><<<gr, KV8_NT, 0, s>>>(g, src, n, slots);
  }
  return cudaGetLastError() == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

int launch_kv8_read(const Kv8Geom& g, int64_t n, const int64_t* slots, void* k_out, void* v_out, int num_sms,
                    cudaStream_t s) {
  if (n == 0) return VBS_OK;
  const int64_t total = n * 2 * g.H * (g.D / 16);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((total + KV8_NT - 1) / KV8_NT, static_cast<int64_t>(num_sms) * 32));
  auto* k = static_cast<uint16_t*>(k_out);
  auto* v = static_cast<uint16_t*>(v_out);
  if (g.fmt == VBS_I8) kv8_read_kernel<VBS_I8><<<grid, KV8_NT, 0, s>>>(g, n, slots, k, v);
  else kv8_read_kernel<VBS_E4M3><<<grid, KV8_NT, 0, s>>>(g, n, slots, k, v);
  return cudaGetLastError() == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

}  // namespace vbs
