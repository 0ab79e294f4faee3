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
// A warp owns one page's tokens in the call, for one head of K or of V: a run of consecutive slots, and what follows it
// past skipped tokens (rare, element by element).  Where the rows can be
// loaded 16 bytes at a time it holds up to 16 tokens x 128 dims in registers between the maximum and the
// rounding (longer runs are read again, from L2), with all loads in flight at once.  What bounds it is the
// stream of the rows in and the codes out: 64 prompts of 1000 tokens, 8 heads x 128 dims, bf16 to int8, take 76 us
// (262 MB read, 131 written: 5.2 TB/s, 77 % of the measured copy; 4 CTAs an SM instead of 3 took 83); a single
// token's step is latency: slot, scale, row (256 rows x 8 heads: 10 us).

#include "codes.cuh"
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

// A page continued at slot `off` with rows that need the exponent e: the larger of that and the page's own; when
// it grows, the codes before `off` are rounded to it.
template <int FMT> __device__ __forceinline__ int regrow(const Kv8Geom& g, int64_t run, int off, int e, int lane) {
  const int e_old = exp2i(g.scales[run]);
  __syncwarp();                                     // read by all lanes before lane 0 writes the new one
  if (e_old >= e) return e_old;
  const float f = e_old - e < -126 ? 0.f : pow2i(e_old - e);
  uint4* codes = reinterpret_cast<uint4*>(g.pool + run * g.block * g.D);
  for (int d = lane; d < off * g.D / 16; d += 32) {
    const uint4 q = codes[d];
    u32 w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      float2 lo, hi;
      decode4<FMT>(w[y], lo, hi);
      w[y] = encode4<FMT>(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
    }
    codes[d] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return e;
}

// The larger magnitudes of two pairs of bf16, a NaN before all.
__device__ __forceinline__ u32 max_abs2(u32 a, u32 b) {
  const __nv_bfloat162 x = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&a));
  const __nv_bfloat162 y = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b));
  const __nv_bfloat162 z = __hmax2_nan(x, y);
  return *reinterpret_cast<const u32*>(&z);
}

// One run, element by element: rows of any alignment, and runs that hold NaN, infinities or values past the largest scale.
template <int FMT, typename T>
__device__ __noinline__ void append_elements(const Kv8Geom& g, const void* base, int64_t tok, int64_t p0, int64_t run,
                                             int off, int len, int lane) {
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
  uint8_t* codes = reinterpret_cast<uint8_t*>(g.pool) + run * g.block * g.D;
  if (off > 0) e = regrow<FMT>(g, run, off, e, lane);
  const float inv = pow2i(-e);
  for (int t = 0; t < len; ++t)
    for (int d = lane; d < g.D; d += 32) {
      const float x = Elem<T>::load(base, p0 + t * tok + d);
      codes[(off + t) * g.D + d] = x == x ? Code<FMT>::enc(x * inv) : 0;
    }
  if (lane == 0) g.scales[run] = pow2i(e);
}

// Whether a slot is one of this cache's (others are skipped).
__device__ __forceinline__ bool held(const Kv8Geom& g, int64_t s) { return s >= 0 && s < g.NB * g.block; }
// Whether `s` goes on in the page of slot `from`, past it.
__device__ __forceinline__ bool goes_on(const Kv8Geom& g, int64_t s, int64_t from, int64_t page) {
  return s > from && s < (page + 1) * g.block;
}

// What follows the run at token t in its page past skipped tokens: runs one after the other, each as if it were a call of
// its own.  kvh: the head of K (0..H-1) or V (H..2H-1).
template <int FMT, typename T>
__device__ __noinline__ void append_rest(const Kv8Geom& g, const Kv8Src& src, int kvh, int64_t t, int64_t n,
                                         const int64_t* slots, int lane) {
  const int kv = kvh >= g.H ? 1 : 0, h = kvh - kv * g.H;
  const void* base = kv ? src.v : src.k;
  const int64_t tok = kv ? src.v_tok : src.k_tok, head = h * (kv ? src.v_head : src.k_head);
  const int64_t page = slots[t] / g.block, run = g.run(page, kv, h);
  int64_t from = -1;                                // the last slot written; -1: the run at t is still to come
  while (t < n) {
    const int64_t s = t + lane < n ? slots[t + lane] : -1;
    const u32 m = __ballot_sync(FULL, held(g, s));
    if (m == 0) {
      t += 32;
      continue;
    }
    const int f = __ffs(m) - 1;
    const int64_t s0 = shfl64(static_cast<u64>(s), f);
    if (!goes_on(g, s0, from, page)) return;
    t += f;
    const int off = static_cast<int>(s0 - page * g.block);
    int len = 1;
    while (off + len < g.block) {
      const int64_t k = t + len + lane;
      const u32 more = __ballot_sync(FULL, k < n && off + len + lane < g.block && slots[k] == s0 + len + lane);
      const int got = more == FULL ? 32 : __ffs(~more) - 1;
      len += got;
      if (got < 32) break;
    }
    __syncwarp();                                   // the run before: its codes and scale, written by other lanes
    if (from >= 0) append_elements<FMT, T>(g, base, tok, t * tok + head, run, off, len, lane);
    t += len;
    from = s0 + len - 1;
  }
}

// A CTA looks at 32 tokens; its warps (and those of the CTAs beside it along y) share out the pages whose tokens begin
// there, each for every head of K and V: a run of consecutive slots first, then what skipped tokens part from it.
template <int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(KV8_NT, Elem<T>::BYTES == 2 ? 3 : 2) kv8_append_kernel(
    const __grid_constant__ Kv8Geom g, const __grid_constant__ Kv8Src src, int64_t n,
    const int64_t* __restrict__ slots) {
  constexpr int EPC = 16 / Elem<T>::BYTES;          // elements in 16 bytes
  constexpr int NR = 16 * 128 / EPC / 32;           // 16-byte pieces a lane holds: 16 tokens x 128 dims a warp
  const int lane = threadIdx.x & 31;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 32, i = i0 + lane;
  const int64_t s = i < n ? slots[i] : -1;
  const int64_t s_back = i0 > 0 ? slots[i - 32] : -1, s_fore = i + 32 < n ? slots[i + 32] : -1;
  const bool valid = held(g, s);
  int64_t page = 0;
  int off = 0;
  if (s >= 0 && !valid) set_status(g.status, VBS_EINVAL);     // not a slot of this cache: nothing is written
  if (valid) {
    page = s / g.block;
    off = static_cast<int>(s - page * g.block);
  }
  const u32 valids = __ballot_sync(FULL, valid);
  // the slot before, skipped tokens apart: where it lies in the same page, the token belongs to its run or follows it
  const u32 below = valids & ((1u << lane) - 1u);
  int64_t prev = static_cast<int64_t>(shfl64(static_cast<u64>(s), below ? 31 - __clz(below) : 0));
  u32 back = __ballot_sync(FULL, held(g, s_back));
  const bool beside = lane > 0 ? (below >> (lane - 1)) != 0 : (back >> 31) != 0;    // no skipped one between
  int64_t last = static_cast<int64_t>(shfl64(static_cast<u64>(s_back), back ? 31 - __clz(back) : 0));
  if (back == 0 && valids != 0 && __shfl_sync(FULL, off, __ffs(valids) - 1) > 0) {  // further back, for the first one
    for (int64_t k = i0 - 64; back == 0 && k >= 0; k -= 32) {
      last = slots[k + lane];
      back = __ballot_sync(FULL, held(g, last));
      last = static_cast<int64_t>(shfl64(static_cast<u64>(last), back ? 31 - __clz(back) : 0));
    }
  }
  if (below == 0) prev = back ? last : -1;
  const bool follows = valid && prev >= page * g.block && goes_on(g, s, prev, page);
  const bool cont = follows && beside && prev == s - 1;
  const u32 conts = __ballot_sync(FULL, cont), resumes = __ballot_sync(FULL, follows && !cont);
  const u32 firsts = __ballot_sync(FULL, valid && !follows);
  // the last run: how far it goes beyond the 32, and whether its page goes on past skipped tokens
  int ext = 0;
  bool far = false;
  if (valids != 0) {
    const int l = 31 - __clz(valids);
    const int64_t s_l = shfl64(static_cast<u64>(s), l), end = (shfl64(static_cast<u64>(page), l) + 1) * g.block;
    const int room = static_cast<int>(end - 1 - s_l);
    int64_t v = s_fore;
    for (int got = l == 31 ? 32 : 0; got == 32 && ext < room;) {
      if (ext > 0) v = i + 32 + ext < n ? slots[i + 32 + ext] : -1;
      const u32 on = __ballot_sync(FULL, ext + lane < room && v == s_l + 1 + ext + lane);
      got = on == FULL ? 32 : __ffs(~on) - 1;
      ext += got;
    }
    for (int64_t k = i0 + 32 + ext; ext < room && k < n; k += 32) {
      if (k > i0 + 32) v = k + lane < n ? slots[k + lane] : -1;
      const u32 m = __ballot_sync(FULL, held(g, v));
      if (m == 0) continue;
      const int64_t next = shfl64(static_cast<u64>(v), __ffs(m) - 1);
      far = next > s_l && next < end;
      break;
    }
  }
  const int per = 2 * g.H, runs = __popc(firsts);
  const int step = gridDim.y * (KV8_NT / 32);
  u32 heads = firsts;
  int at = 0;                                       // runs taken off `heads` so far
  for (int x = blockIdx.y * (KV8_NT / 32) + (threadIdx.x >> 5); x < runs * per; x += step) {
    for (; at < x / per; ++at) heads &= heads - 1;
    const int p = __ffs(heads) - 1, kvh = x % per, kv = kvh >= g.H ? 1 : 0, h = kvh - kv * g.H;
    const int64_t pg = shfl64(static_cast<u64>(page), p);
    const int o = __shfl_sync(FULL, off, p);
    int len = __ffs(~(p < 31 ? conts >> (p + 1) : 0u));       // 1 + the tokens that go on
    if (p + len == 32) len += ext;
    const void* base = kv ? src.v : src.k;
    const int64_t tok = kv ? src.v_tok : src.k_tok;
    const int64_t p0 = (i0 + p) * tok + h * (kv ? src.v_head : src.k_head);
    const int64_t run = g.run(pg, kv, h);
    if (!VEC) {
      append_elements<FMT, T>(g, base, tok, p0, run, o, len, lane);
      continue;
    }
    const int cpr = g.D / EPC, total = len * cpr;   // 16-byte pieces of a row, of the run
    const int t0 = lane / cpr, q0 = lane - t0 * cpr;          // a lane's first piece; from one to its next:
    const int dt = 32 / cpr, dc = 32 - dt * cpr;
    const int64_t row = tok * Elem<T>::BYTES, ahead = dt * row + dc * 16, wrap = row - cpr * 16;
    const char* const first = static_cast<const char*>(base) + p0 * Elem<T>::BYTES + t0 * row + q0 * 16;
    const char* at_q = first;
    int c_q = q0;
    uint4 q[NR];
    // the lane's next pieces, the first of them piece c0 + lane of the run, into q
    auto load = [&](int c0) {
      const int left = total - c0 - lane;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        q[r] = make_uint4(0, 0, 0, 0);
        if (r * 32 < left) q[r] = ld_stream16(at_q);
        at_q += ahead;
        if (dc != 0) {
          c_q += dc;
          if (c_q >= cpr) {
            c_q -= cpr;
            at_q += wrap;
          }
        }
      }
    };
    u32 top = 0;                                    // the largest magnitude's bits (NaN and infinities above all)
    for (int c0 = 0; c0 < total; c0 += NR * 32) {
      load(c0);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if (Elem<T>::BYTES == 2) {
          top = max_abs2(top, max_abs2(max_abs2(q[r].x, q[r].y), max_abs2(q[r].z, q[r].w)));
        } else {
          top = max(max(max(top, q[r].x & 0x7fffffffu), q[r].y & 0x7fffffffu),
                    max(q[r].z & 0x7fffffffu, q[r].w & 0x7fffffffu));
        }
      }
    }
    if (Elem<T>::BYTES == 2) top = max(top & 0xffff0000u, top << 16);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(FULL, top, m));
    if (top > 0x7f7fffffu) {                        // NaN or infinity
      append_elements<FMT, T>(g, base, tok, p0, run, o, len, lane);
      continue;
    }
    const float amax = __uint_as_float(top);
    int e = scale_exp<FMT>(amax);
    if (amax * pow2i(-e) > Code<FMT>::TOP * (1 << Code<FMT>::BITS)) {       // past the largest scale: clamped there
      append_elements<FMT, T>(g, base, tok, p0, run, o, len, lane);
      continue;
    }
    if (o > 0) e = regrow<FMT>(g, run, o, e, lane);
    const u64 inv = pair(pow2i(-e), pow2i(-e));
    uint8_t* codes = reinterpret_cast<uint8_t*>(g.pool) + (run * g.block + o) * g.D + lane * EPC;
    at_q = first;
    c_q = q0;
    for (int c0 = 0; c0 < total; c0 += NR * 32) {
      if (total > NR * 32) load(c0);
      const int left = total - c0 - lane;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if (r * 32 >= left) continue;
        float v[EPC];
        Vec16<T>::unpack(q[r], v);
        const u32 w0 = encode4_scaled<FMT>(v[0], v[1], v[2], v[3], inv);
        if (EPC == 8) {
          const u32 w1 = encode4_scaled<FMT>(v[EPC - 4], v[EPC - 3], v[EPC - 2], v[EPC - 1], inv);
          *reinterpret_cast<uint2*>(codes + r * 256) = make_uint2(w0, w1);
        } else {
          *reinterpret_cast<u32*>(codes + r * 128) = w0;
        }
      }
      codes += NR * 32 * EPC;
    }
    if (lane == 0) g.scales[run] = pow2i(e);
  }
  if (resumes == 0 && !far) return;
  // pages that go on past skipped tokens (rare): by the warp that wrote the run before (in a loop of its own: in the
  // one above its state cost registers, 76 to 82 us for 64 prompts of 1000 tokens)
  heads = firsts;
  at = 0;
  for (int x = blockIdx.y * (KV8_NT / 32) + (threadIdx.x >> 5); x < runs * per; x += step) {
    for (; at < x / per; ++at) heads &= heads - 1;
    append_rest<FMT, T>(g, src, x % per, i0 + __ffs(heads) - 1, n, slots, lane);
  }
}

// A warp a token: its 2 H D codes, 16 a lane, as bf16; a lane's 32 bytes go out in one store where they may (WIDE:
// 81 us against 87 when that was tried).  The chain of slot, codes and stores bounds a warp, so that many warps with two
// pieces a lane do better than fewer with four: 64 prompts of 1000 tokens, 8 heads x 128 dims, take 72 us (131 MB read,
// 262 written: 5.4 TB/s) against 79.
constexpr int KV8_RD = 2;                           // pieces of 16 codes that a lane of the reading kernel holds
template <int FMT, bool WIDE>
__global__ void __launch_bounds__(KV8_NT, 6) kv8_read_kernel(const Kv8Geom g, int64_t n, const int64_t* __restrict__ slots,
                                                          uint16_t* k_out, uint16_t* v_out) {
  const int lane = threadIdx.x & 31, per = g.D / 16, all = 2 * g.H * per;
  const int dk = 32 / per, dc = 32 - dk * per;
  const int64_t stride = (static_cast<int64_t>(gridDim.x) * KV8_NT) >> 5;
  int64_t i = (static_cast<int64_t>(blockIdx.x) * KV8_NT + threadIdx.x) >> 5;
  int64_t next = i < n ? slots[i] : -1;
  for (; i < n; i += stride) {
    const int64_t s = next;
    if (i + stride < n) next = slots[i + stride];
    const bool held = s >= 0 && s < g.NB * g.block;
    if (s >= 0 && !held && lane == 0) set_status(g.status, VBS_EINVAL);
    const int64_t page = !held ? 0 : s <= UINT32_MAX ? static_cast<u32>(s) / static_cast<u32>(g.block) : s / g.block;
    const int64_t run0 = g.run(page, 0, 0);
    const char* codes = g.pool + (run0 * g.block + (held ? s - page * g.block : 0)) * g.D;
    const int64_t head = static_cast<int64_t>(g.block) * g.D;
    for (int j0 = blockIdx.y * KV8_RD * 32 + lane; j0 < all; j0 += gridDim.y * KV8_RD * 32) {
      int kvh = j0 / per, c = j0 - kvh * per;
      uint4 q[KV8_RD];
      float sc[KV8_RD];
      uint16_t* out[KV8_RD];
#pragma unroll
      for (int r = 0; r < KV8_RD; ++r) {
        q[r] = make_uint4(0, 0, 0, 0);
        sc[r] = 0.f;
        if (held && j0 + r * 32 < all) {
          q[r] = ld_stream16(codes + kvh * head + c * 16);
          sc[r] = g.scales[run0 + kvh];
        }
        out[r] = (kvh < g.H ? k_out : v_out) + (i * g.H + (kvh < g.H ? kvh : kvh - g.H)) * g.D + c * 16;
        kvh += dk;
        c += dc;
        if (c >= per) {
          c -= per;
          ++kvh;
        }
      }
#pragma unroll
      for (int r = 0; r < KV8_RD; ++r) {
        if (j0 + r * 32 >= all) continue;
        const u32 w[4] = {q[r].x, q[r].y, q[r].z, q[r].w};
        u32 o[8];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          float2 lo, hi;
          decode4<FMT>(w[y], lo, hi);
          const __nv_bfloat162 x = __floats2bfloat162_rn(lo.x * sc[r], lo.y * sc[r]);   // exact: a code has at most 7 bits
          const __nv_bfloat162 z = __floats2bfloat162_rn(hi.x * sc[r], hi.y * sc[r]);
          o[2 * y] = *reinterpret_cast<const u32*>(&x);
          o[2 * y + 1] = *reinterpret_cast<const u32*>(&z);
        }
        if (WIDE) {
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out[r]), "r"(o[0]), "r"(o[1]),
                       "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]) : "memory");
        } else {
          reinterpret_cast<uint4*>(out[r])[0] = make_uint4(o[0], o[1], o[2], o[3]);
          reinterpret_cast<uint4*>(out[r])[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    }
  }
}

template <int FMT, typename T>
static int launch_append(const Kv8Geom& g, const Kv8Src& src, bool vec, int64_t n, const int64_t* slots, int num_sms,
                         cudaStream_t s) {
  // enough warps for a step of single tokens, where every token is a run; a prompt has a run a page
  const int64_t chunks = (n + 31) / 32;
  if (chunks >= (int64_t{1} << 31)) return VBS_EINVAL;
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(8 * g.H, 4 * num_sms / chunks));
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(y));
  if (vec) kv8_append_kernel<FMT, T, true><<<grid, KV8_NT, 0, s>>>(g, src, n, slots);
  else kv8_append_kernel<FMT, T, false><<<grid, KV8_NT, 0, s>>>(g, src, n, slots);
  return cudaGetLastError() == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

int launch_kv8_append(const Kv8Geom& g, const Kv8Src& src, int64_t n, const int64_t* slots, int num_sms, cudaStream_t s) {
  if (n == 0) return VBS_OK;
  const int es = src.dtype == VBS_BF16 ? 2 : 4;
  const bool vec = ((reinterpret_cast<uintptr_t>(src.k) | reinterpret_cast<uintptr_t>(src.v)) & 15) == 0 &&
                   (src.k_tok | src.k_head | src.v_tok | src.v_head) * es % 16 == 0;
  if (g.fmt == VBS_I8)
    return src.dtype == VBS_BF16 ? launch_append<VBS_I8, bf16_t>(g, src, vec, n, slots, num_sms, s)
                                 : launch_append<VBS_I8, float>(g, src, vec, n, slots, num_sms, s);
  return src.dtype == VBS_BF16 ? launch_append<VBS_E4M3, bf16_t>(g, src, vec, n, slots, num_sms, s)
                               : launch_append<VBS_E4M3, float>(g, src, vec, n, slots, num_sms, s);
}

int launch_kv8_read(const Kv8Geom& g, int64_t n, const int64_t* slots, void* k_out, void* v_out, int num_sms,
                    cudaStream_t s) {
  if (n == 0) return VBS_OK;
  // few tokens: a token's codes are shared out over CTAs as well (256 tokens of 2048 codes: 11 to 9 us)
  const int64_t x = std::min<int64_t>((n + KV8_NT / 32 - 1) / (KV8_NT / 32), static_cast<int64_t>(num_sms) * 32);
  const int64_t parts = (2 * static_cast<int64_t>(g.H) * g.D / 16 + 32 * KV8_RD - 1) / (32 * KV8_RD);
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>({parts, 4 * num_sms / x, 65535}));
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(y));
  auto* k = static_cast<uint16_t*>(k_out);
  auto* v = static_cast<uint16_t*>(v_out);
  const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31) == 0;
  if (g.fmt == VBS_I8) {
    if (wide) kv8_read_kernel<VBS_I8, true><<<grid, KV8_NT, 0, s>>>(g, n, slots, k, v);
    else kv8_read_kernel<VBS_I8, false><<<grid, KV8_NT, 0, s>>>(g, n, slots, k, v);
  } else {
    if (wide) kv8_read_kernel<VBS_E4M3, true><<<grid, KV8_NT, 0, s>>>(g, n, slots, k, v);
    else kv8_read_kernel<VBS_E4M3, false><<<grid, KV8_NT, 0, s>>>(g, n, slots, k, v);
  }
  return cudaGetLastError() == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

}  // namespace vbs
