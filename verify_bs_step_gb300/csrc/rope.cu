// Rotary positions of queries and keys, with the write into a 16-bit paged cache (sm_103a).
//
// A token at position p turns the pair (a, b) of dims by p f: a' = a cos - b sin, b' = b cos + a sin, where the pair is
// (i, i + rot / 2) or (2 i, 2 i + 1) and f its frequency.  Frequencies are held as turns a position in units of 2^-64,
// so that p f modulo a turn is one 64-bit product that wraps, off by 2^-32 of a turn at position 2^31; what is left of the
// nearest quarter of a turn goes to sincospi in fp32.  Products and sums are fp32; a value is rounded once, to its
// output's type.
//
// A warp takes a token and some of its heads (queries, keys and values in one line): it works out the token's angles
// once, two or so a lane, into shared memory, and every lane keeps those of its 16 dims in registers over the heads.
// The first heads' rows are on their way before the angles are worked out.  What bounds it is the rows' stream in and
// out: 64000 tokens x (32 query, 8 + 8 K/V heads) x 128, rotated, written and put into the cache, take 266 us (787 MB read,
// 860 written: 6.2 TB/s, 91 % of the measured copy).  A step of few tokens is one chain of loads, and takes a warp for
// every few heads (256 rows: 3.9 us; 4 rows: 2.6).

#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.cuh"
#include "rope.h"

namespace vbs {

constexpr int RP_NT = 256, RP_W = RP_NT / 32;
constexpr int RP_PAIRS = ROPE_MAX_D / 2;

// Where a head of the line (queries, keys, values) is read and written.
struct RopeHead {
  const void* in;
  void* out;                         // NULL: none
  uint16_t* cache;                   // NULL: none
  bool turned;
};

__device__ __forceinline__ float2 turn_of(unsigned long long turns, int pos, float amp) {
  const unsigned long long t = turns * static_cast<unsigned long long>(static_cast<long long>(pos));
  // the nearest quarter of a turn, and what is left, at most an eighth: fp32 holds that to 2^-28 turns
  const unsigned q = static_cast<unsigned>((t + (1ull << 61)) >> 62);
  const long long rest = static_cast<long long>(t - (static_cast<unsigned long long>(q) << 62));
  float s, c;
  sincospif(static_cast<float>(static_cast<int>(rest >> 30)) * 1.1641532182693481e-10f, &s, &c);   // half turns: 2^-33
  const float x = q & 1 ? -s : c, y = q & 1 ? c : s;
  return q & 2 ? make_float2(-x * amp, -y * amp) : make_float2(x * amp, y * amp);
}

template <typename T> __device__ __forceinline__ T* elem_ptr(const void* p, int64_t i) {
  return reinterpret_cast<T*>(const_cast<void*>(p)) + i;
}

// The cache row of a token's slot (K of head 0), or NULL.
__device__ __forceinline__ uint16_t* cache_row(const Kv16Geom& g, int64_t slot) {
  if (slot == -1) return nullptr;
  if (slot < 0 || slot >= g.NB * g.block) {
    set_status(g.status, VBS_EINVAL);
    return nullptr;
  }
  const int64_t page = slot / g.block;
  const int off = static_cast<int>(slot - page * g.block);
  return g.pool + (((page * g.L + g.layer) * 2 * g.H) * g.block + off) * g.D;
}

template <typename T>
__device__ __forceinline__ RopeHead head_of(const RopeArgs& a, int64_t tok, uint16_t* row, int h) {
  const int64_t hs = static_cast<int64_t>(a.kv.block) * a.kv.D;     // from head to head of a page
  if (h < a.q.heads)
    return {elem_ptr<T>(a.q.in, tok * a.q.in_tok + h * a.q.in_head), elem_ptr<T>(a.q.out, tok * a.q.out_tok + h * a.q.out_head),
            nullptr, true};
  h -= a.q.heads;
  if (h < a.k.heads)
    return {elem_ptr<T>(a.k.in, tok * a.k.in_tok + h * a.k.in_head),
            a.k.out ? elem_ptr<T>(a.k.out, tok * a.k.out_tok + h * a.k.out_head) : nullptr, row ? row + h * hs : nullptr, true};
  h -= a.k.heads;
  return {elem_ptr<T>(a.v.in, tok * a.v.in_tok + h * a.v.in_head), nullptr, row ? row + (a.kv.H + h) * hs : nullptr, false};
}

// Eight consecutive elements, as they are held.
template <typename T> struct Eight;
template <> struct Eight<bf16_t> {
  uint4 x;
  __device__ __forceinline__ void load(const void* p, int d) { x = *reinterpret_cast<const uint4*>(elem_ptr<bf16_t>(p, d)); }
  __device__ __forceinline__ void store(void* p, int d) const { *reinterpret_cast<uint4*>(elem_ptr<bf16_t>(p, d)) = x; }
  __device__ __forceinline__ uint4 bf16() const { return x; }
  __device__ __forceinline__ void get(float (&f)[8]) const { Vec16<bf16_t>::unpack(x, f); }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    u32* w = &x.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const u32*>(&h);
    }
  }
};
template <> struct Eight<float> {
  float4 x, y;
  __device__ __forceinline__ void load(const void* p, int d) {
    x = *reinterpret_cast<const float4*>(elem_ptr<float>(p, d));
    y = *reinterpret_cast<const float4*>(elem_ptr<float>(p, d + 4));
  }
  __device__ __forceinline__ void store(void* p, int d) const {
    *reinterpret_cast<float4*>(elem_ptr<float>(p, d)) = x;
    *reinterpret_cast<float4*>(elem_ptr<float>(p, d + 4)) = y;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    x = make_float4(f[0], f[1], f[2], f[3]);
    y = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ uint4 bf16() const {
    Eight<bf16_t> e;
    float f[8];
    get(f);
    e.set(f);
    return e.x;
  }
};

// A lane's 16 dims: two runs of 8 at d0 and d1, which hold the pairs' first and second dims (HALF) or 8 pairs
// side by side; past the rotated dims, two runs that are copied.
template <typename T, bool HALF> struct Unit {
  Eight<T> lo, hi;
  __device__ __forceinline__ void turn(const float2 (&cs)[8]) {
    float a[8], b[8];
    lo.get(a);
    hi.get(b);
    if (HALF) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = a[i], y = b[i];
        a[i] = fmaf(x, cs[i].x, -y * cs[i].y);
        b[i] = fmaf(y, cs[i].x, x * cs[i].y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
        a[2 * i] = fmaf(x, cs[i].x, -y * cs[i].y);
        a[2 * i + 1] = fmaf(y, cs[i].x, x * cs[i].y);
        b[2 * i] = fmaf(z, cs[i + 4].x, -w * cs[i + 4].y);
        b[2 * i + 1] = fmaf(w, cs[i + 4].x, z * cs[i + 4].y);
      }
    }
    lo.set(a);
    hi.set(b);
  }
};

// VEC: D and rot are multiples of 16 and all rows 16-byte aligned.  A warp takes `passes` passes of 32 / (D / 16) heads
// of its token, from part * passes on.
template <typename T, bool HALF>
__global__ void __launch_bounds__(RP_NT) rope_vec_kernel(const RopeArgs a, int parts, int passes) {
  constexpr int AHEAD = 4;                          // heads whose rows a lane has on their way
  __shared__ float2 table[RP_W][RP_PAIRS];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t id = static_cast<int64_t>(blockIdx.x) * RP_W + wid;
  const int64_t tok = id / parts;
  if (tok >= a.n) return;
  const int part = static_cast<int>(id - tok * parts);
  const int U = a.D / 16, HP = 32 / U;              // units a head, heads a pass
  const int hl = lane / U, u = lane - hl * U;
  const int all = a.q.heads + a.k.heads + a.v.heads;
  const int h0 = part * passes * HP, h1 = min(all, h0 + passes * HP);
  const bool spun = u * 16 < a.r.rot;               // this lane's dims are rotated
  const int d0 = HALF && spun ? u * 8 : u * 16;
  const int d1 = HALF && spun ? a.r.rot / 2 + u * 8 : u * 16 + 8;
  const int pos = a.pos ? a.pos[tok] : 0;
  uint16_t* row = a.kv.pool ? cache_row(a.kv, a.slots[tok]) : nullptr;
  if (pos < 0) return;

  auto fetch = [&](Unit<T, HALF>& x, int h) {
    if (hl < HP && h < h1) {
      const RopeHead at = head_of<T>(a, tok, row, h);
      x.lo.load(at.in, d0);
      x.hi.load(at.in, d1);
    }
  };
  Unit<T, HALF> x[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) fetch(x[i], h0 + i * HP + hl);

  float2 cs[8];
  if (a.r.rot > 0) {
    for (int i = lane; i < a.r.rot / 2; i += 32) table[wid][i] = turn_of(a.r.turns[i], pos, a.r.amp);
    __syncwarp();
    if (spun) {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = table[wid][u * 8 + i];
    }
  }
  for (int hb = h0; hb < h1; hb += AHEAD * HP) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int h = hb + i * HP + hl;
      if (hl < HP && h < h1) {
        const RopeHead at = head_of<T>(a, tok, row, h);
        if (at.turned && spun) x[i].turn(cs);
        if (at.out) {
          x[i].lo.store(at.out, d0);
          x[i].hi.store(at.out, d1);
        }
        if (at.cache) {
          *reinterpret_cast<uint4*>(at.cache + d0) = x[i].lo.bf16();
          *reinterpret_cast<uint4*>(at.cache + d1) = x[i].hi.bf16();
        }
      }
      fetch(x[i], h + AHEAD * HP);
    }
  }
}

template <typename T> __device__ __forceinline__ void put(T* p, float x);
template <> __device__ __forceinline__ void put(float* p, float x) { *p = x; }
template <> __device__ __forceinline__ void put(bf16_t* p, float x) { p->bits = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// Rows of any alignment and size, a pair or an element a lane at a time.
template <typename T>
__global__ void __launch_bounds__(RP_NT) rope_any_kernel(const RopeArgs a) {
  __shared__ float2 table[RP_W][RP_PAIRS];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * RP_W + wid;
  if (tok >= a.n) return;
  const int pos = a.pos ? a.pos[tok] : 0;
  uint16_t* row = a.kv.pool ? cache_row(a.kv, a.slots[tok]) : nullptr;
  if (pos < 0) return;
  const int half = a.r.rot / 2;
  for (int i = lane; i < half; i += 32) table[wid][i] = turn_of(a.r.turns[i], pos, a.r.amp);
  __syncwarp();
  const int all = a.q.heads + a.k.heads + a.v.heads;
  for (int h = blockIdx.y; h < all; h += gridDim.y) {
    const RopeHead at = head_of<T>(a, tok, row, h);
    const T* in = reinterpret_cast<const T*>(at.in);
    T* out = reinterpret_cast<T*>(at.out);
    bf16_t* cache = reinterpret_cast<bf16_t*>(at.cache);
    const int spun = at.turned ? half : 0;
    for (int i = lane; i < spun; i += 32) {
      const int d0 = a.r.layout == VBS_ROPE_HALF ? i : 2 * i, d1 = a.r.layout == VBS_ROPE_HALF ? half + i : 2 * i + 1;
      const float x = Elem<T>::load(in, d0), y = Elem<T>::load(in, d1);
      const float2 cs = table[wid][i];
      const float p = fmaf(x, cs.x, -y * cs.y), q = fmaf(y, cs.x, x * cs.y);
      if (out) {
        put(out + d0, p);
        put(out + d1, q);
      }
      if (cache) {
        put(cache + d0, p);
        put(cache + d1, q);
      }
    }
    for (int d = 2 * spun + lane; d < a.D; d += 32) {
      const float x = Elem<T>::load(in, d);
      if (out) out[d] = in[d];
      if (cache) put(cache + d, x);
    }
  }
}

static bool rows_vec(const RopeRows& r, int elem) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(r.in) | reinterpret_cast<uintptr_t>(r.out);
  return r.heads == 0 || ((p & 15) == 0 && (r.in_tok | r.in_head) * elem % 16 == 0 &&
                          (r.out == nullptr || (r.out_tok | r.out_head) * elem % 16 == 0));
}

template <typename T>
static int launch_rope_as(const RopeArgs& a, int num_sms, cudaStream_t s) {
  const int all = a.q.heads + a.k.heads + a.v.heads, elem = Elem<T>::BYTES;
  if (a.D % 16 == 0 && a.r.rot % 16 == 0 && rows_vec(a.q, elem) && rows_vec(a.k, elem) && rows_vec(a.v, elem)) {
    const int HP = 32 / (a.D / 16), passes = (all + HP - 1) / HP;
    // few tokens: their heads over more warps, until the GPU has some 32 warps an SM
    const int per = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(passes, a.n * passes / (32 * num_sms))));
    const int parts = (passes + per - 1) / per;
    const int64_t grid = (a.n * parts + RP_W - 1) / RP_W;
    if (grid >= int64_t{1} << 31) return VBS_EINVAL;
    return launch_dependent(a.r.layout == VBS_ROPE_HALF ? rope_vec_kernel<T, true> : rope_vec_kernel<T, false>,
                            dim3(static_cast<unsigned>(grid)), dim3(RP_NT), 0, s, a, parts, per);
  }
  const int64_t grid = (a.n + RP_W - 1) / RP_W;
  if (grid >= int64_t{1} << 31) return VBS_EINVAL;
  const int over = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(all, 4 * num_sms / grid)));
  return launch_dependent(rope_any_kernel<T>, dim3(static_cast<unsigned>(grid), over), dim3(RP_NT), 0, s, a);
}

int launch_rope(const RopeArgs& a, int num_sms, cudaStream_t s) {
  if (a.n == 0) return VBS_OK;
  return a.dtype == VBS_BF16 ? launch_rope_as<bf16_t>(a, num_sms, s) : launch_rope_as<float>(a, num_sms, s);
}

}  // namespace vbs
