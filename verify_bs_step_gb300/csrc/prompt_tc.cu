// Attention of packed prompts to themselves: tcgen05 tiles (sm_103a).
//
// An item is 2 x 128 query rows of one K/V head (2 TT tokens in their packed order, whatever requests they are of, the
// heads of a group side by side) over the positions that any of them sees, PT_N at a time:
//   S = Q K^T     tcgen05.mma, Q and K in shared memory (128-byte swizzle), S in TMEM, one buffer a row tile;
//   softmax       four warps a row tile, one thread a row: S from TMEM to registers, weights back to TMEM as bf16;
//   O += P V      tcgen05.mma, P from TMEM, V in shared memory as it comes, O in TMEM.
// The two row tiles share K and V, and one's products run while the other's softmax does.  A warp each loads K (and Q)
// and V by TMA, issues the products, and works out the next item (which positions each of its tokens sees).
//
// A row sees the positions [x, y): its request's first token up to its own (causal) or its request's last.  Tiles
// that some row does not see whole are masked row by row; there V may hold infinities or NaN that no weight of 0
// makes harmless, so that such elements are put to 0 for the product, and added to the rows that see them at the end.
//
// The running reference of the softmax only moves when a row's maximum has grown by 2^8 (in the weights'
// own units): until then weights up to 256 are as good in bf16 as weights up to 1, and O stays where it is.
// The weights' bf16 rounding is the one rounding besides the result's; their sum is taken before it.

#include <climits>

#include <cuda_bf16.h>

#include "pairs.cuh"
#include "prompt.h"
#include "tc.cuh"

namespace vbs {

constexpr int PT_M = 128;                 // query rows a tile
constexpr int PT_N = 128;                 // positions a tile
constexpr int PT_SM = 256;                // softmax threads: one a row of both tiles
constexpr int PT_NT = PT_SM + 128;        // and warps for K, V, the products and the items
constexpr int PT_CU = 4096;               // request starts held in shared memory
constexpr int PT_STMAX = 4;

struct PtArgs {
  PromptArgs p;
  int G, TT;                              // heads a group, tokens a row tile
  int tiles;                              // of 2 TT tokens
  bool out16;                             // stores of 16 bytes
};

template <int DP> struct PtCfg {
  static constexpr int SLABS = DP / 64;                    // 64 dims: 128 bytes a row
  static constexpr int QB = SLABS * PT_M * 128;            // one row tile of Q
  static constexpr int TB = SLABS * PT_N * 128;            // one tile of K or V
  static constexpr int ST = DP == 64 ? 4 : 2;              // stages of K, and of V
  static constexpr size_t SMEM = 2 * QB + 2 * ST * TB + PT_CU * 4 + 1024;
};

// Rings of barriers: kf, vf (a tile has landed), ke, ve (it is not read any more); per row tile: s (scores are done),
// p (weights are written), o (an item's sums are done), of (they have been read).  q, qe: an item's Q has landed, is not
// read any more.  itf, ite: an item is worked out, is done with.  end: every product that was issued is done.
struct PtBars {
  u64 kf[PT_STMAX], ke[PT_STMAX], vf[PT_STMAX], ve[PT_STMAX], s[2], p[2], o[2], of[2], q, qe, itf[2], ite[2], end;
};

struct PtItem {
  int tok, h;                             // first token; h < 0: no more items
  int base;                               // the first position
  int n;                                  // tiles of positions
  int j0[2], j1[2];                       // a row tile's
  int f0[2], f1[2];                       // of them, those that every row sees whole
};

// Whether every row that works on tile j sees all of it: its V is used as it is.
__device__ __forceinline__ bool seen_whole(const PtItem& it, int j) {
  return (j < it.j0[0] || j >= it.j1[0] || (j >= it.f0[0] && j < it.f1[0])) &&
         (j < it.j0[1] || j >= it.j1[1] || (j >= it.f0[1] && j < it.f1[1]));
}

__device__ __forceinline__ void tma_load3(u32 dst, const CUtensorMap* map, u64* bar, int x, int h, int t) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(map), "r"(x), "r"(h), "r"(t), "r"(smem_u32(bar)) : "memory");
}

// request_of with one start in `every` at hand, in shared memory.
__device__ __forceinline__ int2 request_of(const PromptArgs& a, const int* cu, int every, int t) {
  int lo = 0, hi = a.B / every + 1;       // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (cu[m] <= t) lo = m;
    else hi = m;
  }
  int b = lo * every;
  if (every > 1)
    while (b < a.B && b < lo * every + every && a.cu[b + 1] <= t) ++b;
  if (b >= a.B) return make_int2(0, 0);
  const int s = every == 1 ? cu[b] : a.cu[b], e = every == 1 ? cu[b + 1] : a.cu[b + 1];
  return s >= 0 && s <= t && e > t && e <= a.N ? make_int2(s, e) : make_int2(0, 0);
}

template <int DP>
__global__ void __launch_bounds__(PT_NT, 1) prompt_tc_kernel(const __grid_constant__ CUtensorMap qmap,
                                                            const __grid_constant__ CUtensorMap kmap,
                                                            const __grid_constant__ CUtensorMap vmap, const PtArgs a) {
  using C = PtCfg<DP>;
  constexpr int ST = C::ST;
  extern __shared__ unsigned char pt_smem_raw[];
  __shared__ __align__(8) PtBars bars;
  __shared__ u32 tmem_base;
  __shared__ volatile int gone;
  __shared__ volatile int odd;                            // an infinity or NaN of V was put to 0 (stays so)
  __shared__ PtItem ring[2];
  __shared__ int2 span[2][2 * PT_M];                      // positions [x, y) of an item's tokens

  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  unsigned char* smem = pt_smem_raw + ((1024 - (smem_u32(pt_smem_raw) & 1023)) & 1023);
  const u32 q_a = smem_u32(smem), k_a = q_a + 2 * C::QB, v_a = k_a + ST * C::TB;
  int* cu = reinterpret_cast<int*>(smem + 2 * C::QB + 2 * ST * C::TB);
  const PromptArgs& p = a.p;
  const int every = (p.B + 1 + PT_CU - 1) / PT_CU;        // one start in `every` is held
  const int items = a.tiles * p.H;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bars.kf[i], 1);
      mbar_init(&bars.ke[i], 1);
      mbar_init(&bars.vf[i], 1);
      mbar_init(&bars.ve[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s[i], 1);
      mbar_init(&bars.p[i], PT_M);
      mbar_init(&bars.o[i], 1);
      mbar_init(&bars.of[i], PT_M);
      mbar_init(&bars.itf[i], 1);
      mbar_init(&bars.ite[i], PT_SM / 32 + 3);
    }
    mbar_init(&bars.q, 1);
    mbar_init(&bars.qe, 1);
    mbar_init(&bars.end, 1);
    fence_mbar_init();
    gone = 0;
    odd = 0;
  }
  if (wid == PT_SM / 32 + 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  for (int i = tid; i * every <= p.B; i += PT_NT) cu[i] = p.cu[i * every];
  if (blockIdx.x == 0)
    for (int b = tid; b < p.B; b += PT_NT)
      if (p.cu[b] < 0 || p.cu[b] > p.cu[b + 1] || p.cu[b + 1] > p.N) set_status(p.status, VBS_EINVAL);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const u32 tm = tmem_base, tm_s = tm, tm_o = tm + 2 * PT_N;

  // the item in ring slot t & 1, once it is there; done with it, one arrival a warp
  auto item_at = [&](int t) { return tc_wait(&bars.itf[t & 1], (t >> 1) & 1, &gone, p.status); };

  if (wid < PT_SM / 32) {
    // ---- softmax: thread = row ----
    const int X = wid >> 2, r = tid & (PT_M - 1);          // row tile, row
    const u32 tl = static_cast<u32>((wid & 3) * 32) << 16;  // its TMEM lanes
    const u32 ts = tm_s + X * PT_N + tl, to = tm_o + X * DP + tl;
    const bool neg = p.scale < 0.f;
    // (a scale of 0 stays above it, so that a masked -inf stays one)
    const float sc = fmaxf(fabsf(p.scale) * LOG2E_F, 1.17549435e-38f);
    const int tok_r = r / a.G, g = r - tok_r * a.G;
    bool ok = true;
    int T = 0, S = 0, O = 0;                              // K/V tiles, score tiles and items of this row tile so far
    for (int t = 0;; ++t) {
      ok = __all_sync(FULL, item_at(t));
      const PtItem& it = ring[t & 1];
      if (!ok || it.h < 0) break;
      const int2 sp = r < a.TT * a.G ? span[t & 1][X * a.TT + tok_r] : make_int2(0, 0);
      const int x0 = sp.x - it.base, x1 = sp.y - it.base;  // counted from the item's first position
      const int j0 = it.j0[X], j1 = it.j1[X];
      float m = -INFINITY, l = 0.f;                       // the reference (in scaled units), the sum of weights
      for (int j = j0; j < j1; ++j, ++S) {
        ok = __all_sync(FULL, tc_wait(&bars.s[X], S & 1, &gone, p.status));
        if (!ok) break;
        tc_fence_after();
        float s[PT_N];
#pragma unroll
        for (int c = 0; c < PT_N; c += 32) tc_ld32(ts + c, s + c);
        tc_wait_ld();
        if (neg) {
#pragma unroll
          for (int i = 0; i < PT_N; ++i) s[i] = -s[i];
        }
        const int from = x0 - j * PT_N, left = x1 - j * PT_N;
        if (__any_sync(FULL, from > 0 || left < PT_N)) {
#pragma unroll
          for (int i = 0; i < PT_N; ++i)
            if (i < from || i >= left) s[i] = -INFINITY;
        }
        float top[4] = {fmaxf(s[0], s[1]), fmaxf(s[2], s[3]), fmaxf(s[4], s[5]), fmaxf(s[6], s[7])};
#pragma unroll
        for (int i = 8; i < PT_N; i += 2) top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], s[i], s[i + 1]);
        const float mx = max3(fmaxf(top[0], top[1]), top[2], top[3]) * sc;
        const bool grow = mx > m + 8.f;                   // also in a row's first tile: m = -inf
        if (__any_sync(FULL, grow)) {
          const float to_m = grow ? mx : m;
          const float corr = grow ? (m == -INFINITY ? 0.f : ex2(m - to_m)) : 1.f;
          if (j > j0) {
            // O holds the tiles before (S of this one was issued after their products, and is done)
#pragma unroll
            for (int c = 0; c < DP; c += 16) {
              float o[16];
              tc_ld16(to + c, o);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; i += 2) unpair(mul2(pair(o[i], o[i + 1]), pair(corr, corr)), o[i], o[i + 1]);
              tc_st16(to + c, o);
            }
          }
          l *= corr;
          m = to_m;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        // scale and reference go into one fma, whose product is not rounded as the reference was: for
        // large scores the difference is more than a weight can bear, and the product is rounded first
        float f = sc;
        if (__any_sync(FULL, fabsf(ref) > 65536.f)) {
#pragma unroll
          for (int i = 0; i < PT_N; ++i) s[i] *= sc;
          f = 1.f;
        }
        u64 sum[2] = {0, 0};
        const u64 f2 = pair(f, f), r2 = pair(-ref, -ref);
#pragma unroll
        for (int c = 0; c < PT_N; c += 32) {
          float pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x, y;
            unpair(fma2(pair(s[c + 2 * i], s[c + 2 * i + 1]), f2, r2), x, y);
            x = ex2(x);
            y = ex2(y);
            sum[i & 1] = add2(sum[i & 1], pair(x, y));
            __nv_bfloat162 w = __floats2bfloat162_rn(x, y);
            pk[i] = *reinterpret_cast<float*>(&w);
          }
          tc_st16(ts + c / 2, pk);                        // the weights stand where scores were
        }
        float l0, l1;
        unpair(add2(sum[0], sum[1]), l0, l1);
        l += l0 + l1;
        // V where a row does not see the whole tile: the first row tile that works on it looks it through
        const bool mine = X == 0 || j < it.j0[0] || j >= it.j1[0];
        if (mine && !seen_whole(it, j)) {
          const int st = (T + j) % ST;
          ok = tc_wait(&bars.vf[st], ((T + j) / ST) & 1, &gone, p.status);
          ok = __all_sync(FULL, ok);
          if (!ok) break;
#pragma unroll
          for (int sl = 0; sl < C::SLABS; ++sl) {
            uint4* row = reinterpret_cast<uint4*>(smem + (v_a - q_a) + st * C::TB + sl * (PT_N * 128) + r * 128);
            u32 worst = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint4 w = row[(c + r) & 7];           // (eight rows meet eight different chunks)
              worst = max_abs2(max_abs2(max_abs2(worst, w.x), max_abs2(w.y, w.z)), w.w);
            }
            if ((worst & 0x7f80u) == 0x7f80u || (worst & 0x7f800000u) == 0x7f800000u) {
              for (int c = 0; c < 8; ++c) {
                uint4 w = row[c];
                u32* e = &w.x;
                for (int i = 0; i < 4; ++i) {
                  if ((e[i] & 0x7f80u) == 0x7f80u) e[i] &= 0xffff0000u;
                  if ((e[i] & 0x7f800000u) == 0x7f800000u) e[i] &= 0x0000ffffu;
                }
                row[c] = w;
              }
              odd = 1;
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&bars.p[X]);
      }
      T += it.n;
      if (!ok) break;
      if (j1 > j0) {
        ok = __all_sync(FULL, tc_wait(&bars.o[X], O & 1, &gone, p.status));
        if (!ok) break;
        ++O;
        tc_fence_after();
        // ---- out ----
        const bool live = sp.y > sp.x;
        const float inv = 1.f / l;                        // (0 / 0 where every score is -inf: NaN)
        uint16_t* out = p.o + static_cast<int64_t>(it.tok + X * a.TT + tok_r) * p.o_tok +
                        static_cast<int64_t>(it.h * a.G + g) * p.o_head;
        const bool look = odd;
#pragma unroll
        for (int c = 0; c < DP; c += 32) {
          float o[32];
          tc_ld32(to + c, o);
          tc_wait_ld();
          if (look) {
            // what was put to 0, in the tiles that not every row sees whole
            for (int j = j0; j < j1; ++j) {
              if (seen_whole(it, j)) continue;
              const int y1 = min(x1, (j + 1) * PT_N);
              for (int y = max(x0, j * PT_N); y < y1; ++y) {
                const uint16_t* v = p.v + static_cast<int64_t>(it.base + y) * p.v_tok + it.h * p.v_head + c;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float z = c + i < p.D ? bf16_lo(v[i]) : 0.f;
                  if (!(fabsf(z) < INFINITY)) o[i] += z;
                }
              }
            }
          }
          if (live) {
            u32 w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
              w[i] = *reinterpret_cast<const u32*>(&b);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              if (c + i >= p.D) break;
              if (a.out16) {
                *reinterpret_cast<uint4*>(out + c + i) = make_uint4(w[i / 2], w[i / 2 + 1], w[i / 2 + 2], w[i / 2 + 3]);
              } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) out[c + i + k] = static_cast<uint16_t>(w[i / 2 + k / 2] >> (k & 1 ? 16 : 0));
              }
            }
          }
        }
        tc_fence_before();
        mbar_arrive(&bars.of[X]);                         // O may be written again
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.ite[t & 1]);
    }
    tc_wait_st();                                         // (weights of a tile that was given up)
    tc_fence_before();
  } else if (wid < PT_SM / 32 + 2) {
    // ---- loads: one lane each for Q and K, and for V ----
    if (lane == 0) {
      const bool kq = wid == PT_SM / 32;
      u64 *full = kq ? bars.kf : bars.vf, *empty = kq ? bars.ke : bars.ve;
      const CUtensorMap* map = kq ? &kmap : &vmap;
      const u32 dst = kq ? k_a : v_a;
      int T = 0, t = 0;                                   // tiles and items on their way
      bool ok = true;
      while (ok && item_at(t) && ring[t & 1].h >= 0) {
        const PtItem it = ring[t & 1];
        if (kq) {
          if (t > 0 && !tc_wait(&bars.qe, (t - 1) & 1, &gone, p.status)) break;
          const bool two = it.j1[1] > it.j0[1], one = it.j1[0] > it.j0[0];
          mbar_expect_tx(&bars.q, ((one ? 1 : 0) + (two ? 1 : 0)) * C::SLABS * 128 * a.G * a.TT);
#pragma unroll
          for (int X = 0; X < 2; ++X)
            if (X ? two : one)
              for (int x = 0; x < C::SLABS; ++x)
                tma_load3(q_a + X * C::QB + x * PT_M * 128, &qmap, &bars.q, x * 64, it.h * a.G, it.tok + X * a.TT);
        }
        ++t;
        for (int j = 0; j < it.n; ++j, ++T) {
          const int st = T % ST;
          ok = T < ST || tc_wait(&empty[st], ((T / ST) & 1) ^ 1, &gone, p.status);
          if (!ok) break;
          mbar_expect_tx(&full[st], C::TB);
          for (int x = 0; x < C::SLABS; ++x)
            tma_load3(dst + st * C::TB + x * PT_N * 128, map, &full[st], x * 64, it.h, it.base + j * PT_N);
        }
        if (ok) mbar_arrive(&bars.ite[(t - 1) & 1]);
      }
      // no copy is in flight when the CTA ends, also where it gave up: the last ones have landed
      for (int j = max(0, T - ST); j < T; ++j) mbar_wait(&full[j % ST], (j / ST) & 1, 1u << 16);
      if (kq && t > 0) mbar_wait(&bars.q, (t - 1) & 1, 1u << 16);
    }
    __syncwarp();
  } else if (wid == PT_SM / 32 + 2) {
    // ---- products: one elected thread waits and issues ----
    if (elect_one()) {
      const u64 dq = tc_desc(q_a, 16), dk = tc_desc(k_a, 16), dv = tc_desc(v_a, PT_N * 128);
      int T = 0, S[2] = {0, 0}, O[2] = {0, 0};            // K/V tiles; score tiles and items of a row tile
      bool ok = true;
      for (int t = 0; ok && item_at(t) && ring[t & 1].h >= 0; ++t) {
        const PtItem it = ring[t & 1];
        auto on = [&](int X, int j) { return j >= it.j0[X] && j < it.j1[X]; };
        auto scores = [&](int X, int j) {                 // S of the row tile over the item's tile j
          const u64 d = dk + static_cast<u64>((T + j) % ST * (C::TB >> 4)), e = dq + static_cast<u64>(X * (C::QB >> 4));
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            tc_mma_ss(tm_s + X * PT_N, e + (((k >> 2) * (PT_M * 128) + (k & 3) * 32) >> 4),
                      d + (((k >> 2) * (PT_N * 128) + (k & 3) * 32) >> 4), tc_idesc(PT_N, false), k > 0);
          tc_commit(&bars.s[X]);
        };
        auto k_done = [&](int j) {                        // both row tiles' S of tile j are issued
          tc_commit(&bars.ke[(T + j) % ST]);
          if (j + 1 == it.n) tc_commit(&bars.qe);
        };
        ok = tc_wait(&bars.q, t & 1, &gone, p.status) && tc_wait(&bars.kf[T % ST], (T / ST) & 1, &gone, p.status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int X = 0; X < 2; ++X)
          if (on(X, 0)) scores(X, 0);
        k_done(0);
        for (int j = 0; j < it.n; ++j) {
          const int st = (T + j) % ST;
          ok = tc_wait(&bars.vf[st], ((T + j) / ST) & 1, &gone, p.status);
#pragma unroll
          for (int X = 0; X < 2; ++X) {
            if (!ok) break;
            if (on(X, j)) {
              // the item before has read its O
              if (j == it.j0[X] && O[X] > 0) ok = tc_wait(&bars.of[X], (O[X] - 1) & 1, &gone, p.status);
              ok = ok && tc_wait(&bars.p[X], S[X] & 1, &gone, p.status);
              if (!ok) break;
              ++S[X];
              tc_fence_after();
              const u64 d = dv + static_cast<u64>(st * (C::TB >> 4));
#pragma unroll
              for (int k = 0; k < PT_N / 16; ++k)
                tc_mma_ts(tm_o + X * DP, tm_s + X * PT_N + k * 8, d + (k * 2048 >> 4), tc_idesc(DP, true),
                          j > it.j0[X] || k > 0);
              if (j + 1 == it.j1[X]) {
                tc_commit(&bars.o[X]);
                ++O[X];
              }
            }
            if (j + 1 < it.n) {
              if (X == 0) {
                ok = tc_wait(&bars.kf[(T + j + 1) % ST], ((T + j + 1) / ST) & 1, &gone, p.status);
                if (!ok) break;
                tc_fence_after();
              }
              if (on(X, j + 1)) scores(X, j + 1);
            }
          }
          if (!ok) break;
          tc_commit(&bars.ve[st]);
          if (j + 1 < it.n) k_done(j + 1);
        }
        if (!ok) break;
        T += it.n;
        mbar_arrive(&bars.ite[t & 1]);
      }
      // the products in flight read shared memory and TMEM: all are done before either goes, also where the CTA gave up
      tc_commit(&bars.end);
      mbar_wait(&bars.end, 0, 1u << 16);
    }
    __syncwarp();
  } else {
    // ---- items: the last tokens first, which see the most ----
    int t = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < items + static_cast<int>(gridDim.x); i += gridDim.x) {
      const bool last = i >= items;
      PtItem x;
      x.h = last ? -1 : i % p.H;
      x.tok = last ? 0 : (a.tiles - 1 - i / p.H) * 2 * a.TT;
      int2 sp[2 * PT_M / 32];
      int y0[2] = {INT_MAX, INT_MAX}, y1[2] = {0, 0}, z0[2] = {0, 0}, z1[2] = {INT_MAX, INT_MAX};   // of x and y of the spans
#pragma unroll
      for (int k = 0; k < 2 * PT_M / 32; ++k) {
        const int w = k * 32 + lane, tok = x.tok + w;
        sp[k] = make_int2(0, 0);
        if (last || w >= 2 * a.TT || tok >= p.N) continue;
        sp[k] = request_of(p, cu, every, tok);
        if (sp[k].y <= sp[k].x) continue;
        if (p.causal) sp[k].y = tok + 1;
        const int X = w >= a.TT ? 1 : 0;
        y0[X] = min(y0[X], sp[k].x);
        y1[X] = max(y1[X], sp[k].y);
        z0[X] = max(z0[X], sp[k].x);
        z1[X] = min(z1[X], sp[k].y);
      }
#pragma unroll
      for (int X = 0; X < 2; ++X) {
        y0[X] = __reduce_min_sync(FULL, y0[X]);
        y1[X] = __reduce_max_sync(FULL, y1[X]);
        z0[X] = __reduce_max_sync(FULL, z0[X]);
        z1[X] = __reduce_min_sync(FULL, z1[X]);
      }
      x.base = min(y0[0], y0[1]);
      x.n = 0;
#pragma unroll
      for (int X = 0; X < 2; ++X) {
        const bool some = y1[X] > 0;
        x.j0[X] = some ? (y0[X] - x.base) / PT_N : 0;
        x.j1[X] = some ? (y1[X] - x.base + PT_N - 1) / PT_N : 0;
        x.f0[X] = some ? (z0[X] - x.base + PT_N - 1) / PT_N : 0;
        x.f1[X] = some ? (z1[X] - x.base) / PT_N : 0;
        x.n = max(x.n, x.j1[X]);
      }
      if (!last && x.n == 0) continue;                    // tokens of no request
      if (t >= 2) ok = __all_sync(FULL, tc_wait(&bars.ite[t & 1], ((t >> 1) - 1) & 1, &gone, p.status));
      if (!ok) break;
#pragma unroll
      for (int k = 0; k < 2 * PT_M / 32; ++k) span[t & 1][k * 32 + lane] = sp[k];
      if (lane == 0) ring[t & 1] = x;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.itf[t & 1]);
      ++t;
    }
  }
  __syncthreads();
  tc_fence_after();
  if (wid == PT_SM / 32 + 2)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512) : "memory");
}

// ---------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------

// [N][heads][D] bf16 with strides that are multiples of 16 bytes, as boxes of `tok` tokens x `head` heads x 64 dims
static bool encode(CUtensorMap* map, const uint16_t* x, const PromptArgs& p, int heads, int64_t tok_s, int64_t head_s, int head,
                   int tok) {
  const EncodeFn fn = tensor_map_encode();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(p.N)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? head_s * 2 : 16),
                                 static_cast<cuuint64_t>(p.N > 1 ? tok_s * 2 : 16)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(head), static_cast<cuuint32_t>(tok)}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(x), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool prompt_tc_takes(const PromptArgs& p) {
  auto stride_ok = [](int64_t s, int64_t extent) { return extent == 1 || (s > 0 && s % 8 == 0 && s < (int64_t{1} << 38)); };
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v);
  return p.D <= 128 && p.Hq / p.H <= PT_M && (at & 15) == 0 && stride_ok(p.q_tok, p.N) && stride_ok(p.q_head, p.Hq) &&
         stride_ok(p.k_tok, p.N) && stride_ok(p.k_head, p.H) && stride_ok(p.v_tok, p.N) && stride_ok(p.v_head, p.H) &&
         tensor_map_encode() != nullptr;
}

template <int DP>
static int launch_tc(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const PtArgs& a, int num_sms,
                     cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};
  if (!smem_attr_once(prompt_tc_kernel<DP>, static_cast<int>(PtCfg<DP>::SMEM), attr_done)) return VBS_ECUDA;
  const int grid = std::min(a.tiles * a.p.H, num_sms);
  prompt_tc_kernel<DP><<<grid, PT_NT, PtCfg<DP>::SMEM, s>>>(qm, km, vm, a);
  return cudaGetLastError() == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

int launch_prompt_tc(const PromptArgs& p, int num_sms, cudaStream_t s) {
  const int G = p.Hq / p.H, TT = PT_M / G;
  CUtensorMap qm, km, vm;
  if (!encode(&qm, p.q, p, p.Hq, p.q_tok, p.q_head, G, TT) || !encode(&km, p.k, p, p.H, p.k_tok, p.k_head, 1, PT_N) ||
      !encode(&vm, p.v, p, p.H, p.v_tok, p.v_head, 1, PT_N))
    return VBS_ECUDA;
  const PtArgs a{p, G, TT, (p.N + 2 * TT - 1) / (2 * TT),
                 (reinterpret_cast<uintptr_t>(p.o) & 15) == 0 && (p.o_tok | p.o_head) % 8 == 0};
  return p.D <= 64 ? launch_tc<64>(qm, km, vm, a, num_sms, s) : launch_tc<128>(qm, km, vm, a, num_sms, s);
}

}  // namespace vbs
