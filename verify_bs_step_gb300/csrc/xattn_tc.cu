// Cross attention of many query rows: tcgen05 tiles (sm_103a).
//
// A CTA takes 128 of the query rows that share one sentence's K/V head (token by token, the heads of a
// group side by side) over all of the sentence's positions, TC_N at a time:
//   S = Q K^T     tcgen05.mma, Q and K in shared memory (128-byte swizzle), S in TMEM, two or three buffers;
//   softmax       four warps, one thread a row: S from TMEM to registers, weights back to TMEM as bf16;
//   O += P V      tcgen05.mma, P from TMEM, V in shared memory as it comes (positions are the contraction,
//                 so V is the transposed operand), O in TMEM.
// One warp brings K and V in by TMA (128-byte swizzle, zeros past head_dim and past the tensor's end), one
// issues the products: S of the tiles ahead is issued before it waits for the weights of this one.
//
// The running reference of the softmax only moves when a row's maximum has grown by 2^8 (in the weights'
// own units): until then weights up to 256 are as good in bf16 as weights up to 1, and O stays where it is.
// The weights' bf16 rounding is the one rounding besides the result's; their sum is taken before it.
//
// What bounds it: the chain of one tile in one CTA (wait for S, 64 scores a thread to registers, maximum,
// exponentials, weights back, signal: some 1340 clocks of a 128 x 64 tile), not a pipe: at head_dim 64 the products
// take 256 of the 740 clocks that a tile costs an SM, the exponentials 256.  Two CTAs an SM, 256 TMEM columns each,
// fill each other's waits; TMEM has no room for a third.  Persistent CTAs take the items longest sentence first
// where that pays.  16 x 16 heads x 64, 1024 rows over 1000..2048 positions: 145 us (706 TFLOP/s, 37 % of the measured
// peak); 4 x 8 heads x 128, 500 rows x 4 heads a group over 500..4000: 78 us (945 TFLOP/s, 50 %).
// Measured and not kept: two threads a row (159 us, its vote a tile), a lane that waits for its warp (173), K and V
// loads that block in turn (162), one CTA an SM (230).

#include <cuda_bf16.h>

#include "attn.h"
#include "pairs.cuh"
#include "tc.cuh"
#include "xattn_tc.h"

namespace vbs {

constexpr int TC_M = 128;                 // query rows a CTA
constexpr int TC_N = 64;                  // positions a tile
constexpr int TC_STMAX = 4;               // stages of K, and of V, at most
constexpr int TC_SM = 128;                // softmax threads: one a row
constexpr int TC_SW = TC_SM / 32;         // softmax warps
constexpr int TC_SORT = 1024;             // sentences that can be put in order of length
constexpr int TC_NT = TC_SM + 64;         // and a load warp, a product warp
constexpr int TC_COLS = 256;              // TMEM columns: S (3 x TC_N or 2 x TC_N) and O (64 or 128)

struct TcArgs {
  QO io;
  const int32_t* len;
  int* status;
  int S, B, W, H, D, G, M;
  int tiles;                              // of TC_M rows
  bool q16, out16;                        // 16-byte loads of q, stores of out
  bool sorted;                            // longest sentences first
};

template <int DP> struct TcCfg {
  static constexpr int SLABS = DP / 64;                    // 64 dims: 128 bytes a row
  static constexpr int QB = SLABS * TC_M * 128;
  static constexpr int TB = SLABS * TC_N * 128;            // one tile of K or V
  static constexpr int ST = DP == 64 ? 4 : 2;              // stages: what two CTAs' shared memory holds
  static constexpr int NB = DP == 64 ? 3 : 2;              // S buffers, beside O in 256 TMEM columns
  static constexpr int NQ = DP == 64 ? 2 : 1;              // Q buffers: the next item's rows come in early
  static constexpr size_t SMEM = NQ * QB + 2 * ST * TB + 1024;
};

__device__ __forceinline__ void tma_load(u32 dst, const CUtensorMap* map, u64* bar, int x, int s, int h, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(map), "r"(x), "r"(s), "r"(h), "r"(b), "r"(smem_u32(bar)) : "memory");
}

// Rings of barriers: kf, vf (a tile's K or V has landed), s (its scores are done: so its K stage is free) and pv
// (its products are in O: so its V stage is free), one per stage, and p (its weights are written),
// one per S buffer.  Who waits
// for a tile's phase knows that the ring's turn before it is over, so that a barrier stands in the phase
// waited for or in the next, and its parity tells them apart.  q, qe, of: an item's Q has landed, is not read
// any more, its O has been read.  end: every product that was issued is done.
struct TcBars {
  u64 q[2], qe[2], of, kf[TC_STMAX], vf[TC_STMAX], s[TC_STMAX], pv[TC_STMAX], p[3], end;
};

// The t-th item of this CTA, or -1: items are the sentences' (head, row tile) pairs, longest sentences first;
// the CTAs take them in turn, back and forth, so that every CTA gets long and short ones.
__device__ __forceinline__ int item_of(int t, int items) {
  const int i = t * gridDim.x + (t & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  return i < items ? i : -1;
}

template <int DP>
__global__ void __launch_bounds__(TC_NT, 2) xattn_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                                                           const __grid_constant__ CUtensorMap vmap, const TcArgs a) {
  using C = TcCfg<DP>;
  constexpr int ST = C::ST;
  extern __shared__ unsigned char tc_smem_raw[];
  __shared__ __align__(8) TcBars bars;
  __shared__ u32 tmem_base;
  __shared__ volatile int gone;
  __shared__ uint16_t order[TC_SORT];                     // sentences, longest first
  __shared__ int64_t q_at[TC_M];                          // element offsets of the item's query rows, -1: none

  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  unsigned char* smem = tc_smem_raw + ((1024 - (smem_u32(tc_smem_raw) & 1023)) & 1023);
  const u32 q_a = smem_u32(smem), k_a = q_a + C::NQ * C::QB, v_a = k_a + ST * C::TB;

  if (tid == 0) {
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(&bars.q[i], 32);
      mbar_init(&bars.qe[i], 1);
    }
    mbar_init(&bars.of, TC_SM);
    mbar_init(&bars.end, 1);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bars.kf[i], 1);
      mbar_init(&bars.vf[i], 1);
      mbar_init(&bars.s[i], 1);
      mbar_init(&bars.pv[i], 1);
    }
    for (int i = 0; i < C::NB; ++i) mbar_init(&bars.p[i], TC_SM);
    fence_mbar_init();
    gone = 0;
  }
  if (wid == TC_SW + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)), "r"(TC_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (a.sorted)
    for (int x = tid; x < a.B; x += TC_NT) {
      const int mine = a.len[x];
      int rank = 0;
      for (int y = 0; y < a.B; ++y) {
        const int other = a.len[y];
        rank += other > mine || (other == mine && y < x) ? 1 : 0;
      }
      order[rank] = static_cast<uint16_t>(x);
    }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const u32 tm = tmem_base, tm_s = tm, tm_o = tm + C::NB * TC_N;

  struct Item { int b, h, rows0, len, n; };                // n: tiles of positions; b < 0: no more items
  const int items = a.B * a.H * a.tiles;
  auto item_at = [&](int t) {
    Item it{-1, 0, 0, 0, 0};
    const int i = item_of(t, items);
    if (i < 0) return it;
    const int bh = i / a.tiles, x = bh / a.H;
    it.rows0 = (i - bh * a.tiles) * TC_M;
    it.h = bh - x * a.H;
    it.b = a.sorted ? order[x] : x;
    it.len = a.len[it.b];
    if (it.len < 0 || it.len > a.S) {
      set_status(a.status, VBS_EINVAL);
      it.len = it.len < 0 ? 0 : a.S;
    }
    it.n = static_cast<int>((static_cast<u32>(it.len) + TC_N - 1) / TC_N);
    return it;
  };

  if (wid < TC_SW) {
    // ---- softmax: thread = row ----
    const u32 row = static_cast<u32>(wid * 32) << 16;
    const bool neg = a.io.scale < 0.f;
    // (a scale of 0 stays above it, so that a masked -inf stays one)
    const float sc = fmaxf(fabsf(a.io.scale) * LOG2E_F, 1.17549435e-38f);
    bool ok = true;
    int T = 0;                                     // tiles so far: all barriers count on across items
    Item next = item_at(0);
    for (int t = 1; ok && next.b >= 0; ++t) {
      const Item it = next;
      next = item_at(t);
      float m = -INFINITY, l = 0.f;                // the reference (in scaled units), the sum of weights
      for (int j = 0; j < it.n; ++j, ++T) {
        ok = tc_wait(&bars.s[T % ST], (T / ST) & 1, &gone, a.status);
        ok = __all_sync(FULL, ok);
        if (!ok) break;
        tc_fence_after();
        const u32 sa = tm_s + (T % C::NB) * TC_N + row;
        float s[TC_N];
        tc_ld32(sa, s);
        tc_ld32(sa + 32, s + 32);
        tc_wait_ld();
        if (neg) {
#pragma unroll
          for (int i = 0; i < TC_N; ++i) s[i] = -s[i];
        }
        const int left = it.len - j * TC_N;
        if (left < TC_N) {                         // the sentence ends in this tile
#pragma unroll
          for (int i = 0; i < TC_N; ++i)
            if (i >= left) s[i] = -INFINITY;
        }
        float top[4] = {fmaxf(s[0], s[1]), fmaxf(s[2], s[3]), fmaxf(s[4], s[5]), fmaxf(s[6], s[7])};
#pragma unroll
        for (int i = 8; i < TC_N; i += 2) top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], s[i], s[i + 1]);
        const float mx = max3(fmaxf(top[0], top[1]), top[2], top[3]) * sc;
        const bool grow = mx > m + 8.f;            // also in the first tile: m = -inf
        if (__any_sync(FULL, grow)) {
          const float to = grow ? mx : m;
          const float corr = grow ? (m == -INFINITY ? 0.f : ex2(m - to)) : 1.f;
          if (j > 0) {                             // O holds the tiles before
            ok = tc_wait(&bars.pv[(T - 1) % ST], ((T - 1) / ST) & 1, &gone, a.status);
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < DP; c += 16) {
              float o[16];
              tc_ld16(tm_o + row + c, o);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; i += 2) unpair(mul2(pair(o[i], o[i + 1]), pair(corr, corr)), o[i], o[i + 1]);
              tc_st16(tm_o + row + c, o);
            }
          }
          l *= corr;
          m = to;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        // scale and reference go into one fma, whose product is not rounded as the reference was: for
        // large scores the difference is more than a weight can bear, and the product is rounded first
        float f = sc;
        if (__any_sync(FULL, fabsf(ref) > 65536.f)) {
#pragma unroll
          for (int i = 0; i < TC_N; ++i) s[i] *= sc;
          f = 1.f;
        }
        u64 sum[2] = {0, 0};
        const u64 f2 = pair(f, f), r2 = pair(-ref, -ref);
#pragma unroll
        for (int c = 0; c < TC_N; c += 32) {
          float pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x, y;
            unpair(fma2(pair(s[c + 2 * i], s[c + 2 * i + 1]), f2, r2), x, y);
            x = ex2(x);
            y = ex2(y);
            sum[i & 1] = add2(sum[i & 1], pair(x, y));
            __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
            pk[i] = *reinterpret_cast<float*>(&p);
          }
          tc_st16(sa + c / 2, pk);                 // the weights stand where scores were
        }
        float l0, l1;
        unpair(add2(sum[0], sum[1]), l0, l1);
        l += l0 + l1;
        if (left < TC_N) {
          // positions past the end: their weights are 0, and V's rows have to be finite
          const int st = T % ST;
          ok = tc_wait(&bars.vf[st], (T / ST) & 1, &gone, a.status);
          for (int x = tid; x < (TC_N - left) * 8 * C::SLABS; x += TC_SM) {
            const int c = x & 7, vr = left + (x >> 3) % (TC_N - left), sl = (x >> 3) / (TC_N - left);
            *reinterpret_cast<uint4*>(smem + (v_a - q_a) + st * C::TB + sl * (TC_N * 128) + vr * 128 + c * 16) =
                make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          ok = __all_sync(FULL, ok);
          if (!ok) break;
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&bars.p[T % C::NB]);
      }
      if (ok && it.n > 0) ok = tc_wait(&bars.pv[(T - 1) % ST], ((T - 1) / ST) & 1, &gone, a.status);
      ok = __all_sync(FULL, ok);
      if (!ok) break;
      tc_fence_after();

      // ---- out ----
      const int rho = it.rows0 + tid;
      const int gq = rho % a.G, i = rho / a.G % a.io.n_q, w = rho / a.G / a.io.n_q;
      uint16_t* out = a.io.o + static_cast<int64_t>(it.b * a.W + w) * a.io.o_row + i * a.io.o_tok +
                      (it.h * a.G + gq) * a.io.o_head;
      const float inv = 1.f / l;                   // (0 / 0 where every score is -inf: NaN)
      u32 x[DP / 2];
#pragma unroll
      for (int c = 0; c < DP; c += 16) {
        float o[16];
        if (it.n > 0) {
          tc_ld16(tm_o + row + c, o);
          tc_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const __nv_bfloat162 p = it.n > 0 ? __floats2bfloat162_rn(o[k] * inv, o[k + 1] * inv)
                                            : __floats2bfloat162_rn(0.f, 0.f);
          x[(c + k) / 2] = *reinterpret_cast<const u32*>(&p);
        }
      }
      if (it.n > 0) {
        tc_fence_before();
        mbar_arrive(&bars.of);                     // O may be written again
      }
      if (rho < a.M) {
#pragma unroll
        for (int c = 0; c < DP; c += 8) {
          if (c >= a.D) break;
          if (a.out16) {
            *reinterpret_cast<uint4*>(out + c) = make_uint4(x[c / 2], x[c / 2 + 1], x[c / 2 + 2], x[c / 2 + 3]);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) out[c + k] = static_cast<uint16_t>(x[c / 2 + k / 2] >> (k & 1 ? 16 : 0));
          }
        }
      }
      __syncwarp();
    }
    tc_wait_st();                                  // (weights of a tile that was given up)
    tc_fence_before();
  } else if (wid == TC_SW) {
    // ---- loads: Q by the whole warp, K and V by one lane, each as far ahead as its stages go ----
    int T0 = 0, done = 0;                          // tiles before this item; items with tiles so far
    int kt = 0, vt = 0;                            // tiles of K and of V that lane 0 has loaded
    bool ok = true;
    for (int t = 0;; ++t) {
      const Item it = item_at(t);
      if (it.b < 0) break;
      if (it.n == 0) continue;
      // where the rows stand (four a lane, divided out once), then 16 bytes of them at a time
      for (int r = lane; r < TC_M; r += 32) {
        const int rho = it.rows0 + r;
        const int gq = rho % a.G, i = rho / a.G % a.io.n_q, w = rho / a.G / a.io.n_q;
        const int64_t at = static_cast<int64_t>(it.b * a.W + w) * a.io.q_row + i * a.io.q_tok +
                           (it.h * a.G + gq) * a.io.q_head;
        q_at[r] = rho < a.M ? at : -1;
      }
      __syncwarp();                                // each lane reads what the others wrote
      const int qb = done % C::NQ;
      ok = done < C::NQ || tc_wait(&bars.qe[qb], (done / C::NQ - 1) & 1, &gone, a.status);
      ok = __all_sync(FULL, ok);
      if (!ok) break;
#pragma unroll 8
      for (int idx = lane; idx < TC_M * (DP / 8); idx += 32) {
        const int r = idx / (DP / 8), c = idx % (DP / 8);
        const int64_t at = q_at[r];
        const bool live = at >= 0 && c * 8 < a.D;
        const uint16_t* q = live ? a.io.q + at + c * 8 : a.io.q;
        const u32 to = qb * C::QB + (c >> 3) * (TC_M * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        if (a.q16) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(q_a + to), "l"(q), "r"(live ? 16 : 0) : "memory");
        } else {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (live) {
            x.x = q[0] | static_cast<u32>(q[1]) << 16;
            x.y = q[2] | static_cast<u32>(q[3]) << 16;
            x.z = q[4] | static_cast<u32>(q[5]) << 16;
            x.w = q[6] | static_cast<u32>(q[7]) << 16;
          }
          *reinterpret_cast<uint4*>(smem + to) = x;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      int jk = 0, jv = 0;
      auto feed = [&](int most) {                  // loads tiles until `most` of each are on their way
        for (u32 idle = 0; (jk < most || jv < most) && idle < TC_SPIN && !gone;) {
          bool moved = false;
          if (jk < most) {
            const int T = T0 + jk, st = T % ST;
            if (T < ST || mbar_test(&bars.s[st], ((T / ST) & 1) ^ 1)) {
              mbar_expect_tx(&bars.kf[st], C::TB);
              for (int x = 0; x < C::SLABS; ++x)
                tma_load(k_a + st * C::TB + x * TC_N * 128, &kmap, &bars.kf[st], x * 64, jk * TC_N, it.h, it.b);
              ++jk;
              moved = true;
            }
          }
          if (jv < most) {
            const int T = T0 + jv, st = T % ST;
            if (T < ST || mbar_test(&bars.pv[st], ((T / ST) & 1) ^ 1)) {
              mbar_expect_tx(&bars.vf[st], C::TB);
              for (int x = 0; x < C::SLABS; ++x)
                tma_load(v_a + st * C::TB + x * TC_N * 128, &vmap, &bars.vf[st], x * 64, jv * TC_N, it.h, it.b);
              ++jv;
              moved = true;
            }
          }
          idle = moved ? 0 : idle + 1;
        }
        if ((jk < most || jv < most) && !gone) {
          gone = 1;
          set_status(a.status, VBS_ETIMEOUT);
        }
        return jk >= most && jv >= most;
      };
      // the first K goes out before Q is waited for, where its stage is free
      if (lane == 0 && (T0 < ST || mbar_test(&bars.s[T0 % ST], ((T0 / ST) & 1) ^ 1))) {
        const int st = T0 % ST;
        mbar_expect_tx(&bars.kf[st], C::TB);
        for (int x = 0; x < C::SLABS; ++x)
          tma_load(k_a + st * C::TB + x * TC_N * 128, &kmap, &bars.kf[st], x * 64, 0, it.h, it.b);
        jk = 1;
      }
      __syncwarp();
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&bars.q[qb]);
      if (lane == 0) ok = feed(it.n);
      ok = __all_sync(FULL, ok);
      kt = T0 + jk;
      vt = T0 + jv;
      T0 += it.n;
      ++done;
      if (!ok) break;
    }
    // no copy is in flight when the CTA ends, also where it gave up: the last ones have landed
    if (lane == 0) {
      for (int j = max(0, kt - ST); j < kt; ++j) mbar_wait(&bars.kf[j % ST], (j / ST) & 1, 1u << 16);
      for (int j = max(0, vt - ST); j < vt; ++j) mbar_wait(&bars.vf[j % ST], (j / ST) & 1, 1u << 16);
    }
  } else {
    // ---- products: one elected thread waits and issues ----
    if (elect_one()) {
      const u64 dq = tc_desc(q_a, 16), dk = tc_desc(k_a, 16), dv = tc_desc(v_a, TC_N * 128);
      int T = 0, done = 0;
      bool ok = true;
      Item next = item_at(0);
      for (int t = 1; ok && next.b >= 0; ++t) {
        const Item it = next;
        next = item_at(t);
        if (it.n == 0) continue;
        const int qb = done % C::NQ;
        const u64 dqi = dq + static_cast<u64>(qb * (C::QB >> 4));
        auto scores = [&](int j) {                 // S of the item's tile j
          const int X = T + j, st = X % ST;
          if (!tc_wait(&bars.kf[st], (X / ST) & 1, &gone, a.status)) return false;
          tc_fence_after();
          const u64 d = dk + static_cast<u64>(st * (C::TB >> 4));
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            tc_mma_ss(tm_s + (X % C::NB) * TC_N, dqi + (((k >> 2) * (TC_M * 128) + (k & 3) * 32) >> 4),
                      d + (((k >> 2) * (TC_N * 128) + (k & 3) * 32) >> 4), tc_idesc(TC_N, false), k > 0);
          tc_commit(&bars.s[st]);
          if (j + 1 == it.n) tc_commit(&bars.qe[qb]);  // Q may be loaded again
          return true;
        };
        ok = tc_wait(&bars.q[qb], (done / C::NQ) & 1, &gone, a.status);
        for (int j = 0; j < C::NB - 1 && j < it.n; ++j) ok = ok && scores(j);
        // the item before has read its O
        ok = ok && (done == 0 || tc_wait(&bars.of, (done - 1) & 1, &gone, a.status));
        for (int j = 0; j < it.n && ok; ++j) {
          if (j + C::NB - 1 < it.n) ok = scores(j + C::NB - 1);
          const int X = T + j, st = X % ST;
          ok = ok && tc_wait(&bars.vf[st], (X / ST) & 1, &gone, a.status);
          ok = ok && tc_wait(&bars.p[X % C::NB], (X / C::NB) & 1, &gone, a.status);
          if (!ok) break;
          tc_fence_after();
          const u64 d = dv + static_cast<u64>(st * (C::TB >> 4));
#pragma unroll
          for (int k = 0; k < TC_N / 16; ++k)
            tc_mma_ts(tm_o, tm_s + (X % C::NB) * TC_N + k * 8, d + (k * 2048 >> 4), tc_idesc(DP, true), j > 0 || k > 0);
          tc_commit(&bars.pv[st]);
        }
        T += it.n;
        ++done;
      }
      // the products in flight read shared memory and TMEM: all are done before either goes, also where the CTA gave up
      tc_commit(&bars.end);
      mbar_wait(&bars.end, 0, 1u << 16);
    }
    __syncwarp();
  }
  __syncthreads();
  tc_fence_after();
  if (wid == TC_SW + 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(TC_COLS) : "memory");
}

// ---------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------

// [B][H][S][D] bf16 with any strides that are multiples of 16 bytes, as tiles of TC_N positions x 64 dims
static bool encode(CUtensorMap* map, const uint16_t* p, const EncKV& e, int64_t sent, int64_t pos, int64_t head) {
  const EncodeFn fn = tensor_map_encode();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(e.D), static_cast<cuuint64_t>(e.S), static_cast<cuuint64_t>(e.H),
                              static_cast<cuuint64_t>(e.B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(e.S > 1 ? pos * 2 : 16),
                                 static_cast<cuuint64_t>(e.H > 1 ? head * 2 : 16),
                                 static_cast<cuuint64_t>(e.B > 1 ? sent * 2 : 16)};
  const cuuint32_t box[4] = {64, TC_N, 1, 1}, step[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(p), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Microseconds of the tiles at full lengths: 0.56 a tile and CTA in turn.
static double tiles_us(int64_t items, int S, int num_sms) {
  return ((S - 1) / TC_N + 1) * 0.56 * std::max(1.0, static_cast<double>(items) / (2 * num_sms));
}

// Longest sentences first shares the work out better, but every CTA ranks all the sentences for it, some 7.2e-5 B^2 us.
// Sorted / unsorted in us, sentences x heads, rows x positions up to:
//   64 x 8, 40 x 2000   40.5 / 54.8;   512 x 8, 40 x 2000   238 / 265;   512 x 8 (head_dim 128), 300 x 600   489 / 534
//   1024 x 1, 20 x 400  113.5 / 39.1;  256 x 1, 128 x 400  20.0 / 15.2;  1024 x 8, 40 x 2000   497 / 448
// The ranking is worth a tenth of the time that the tiles take; the choice is within 10 % of the better on 77 such shapes.
static bool sort_pays(int B, int64_t items, int S, int num_sms) {
  return B > 1 && B <= TC_SORT && 7.2e-5 * B * B < 0.1 * tiles_us(items, S, num_sms);
}

bool xattn_tc_takes(const EncKV& e, const QO& io, int num_sms) {
  const int64_t M = static_cast<int64_t>(e.W) * io.n_q * (io.Hq / e.H);
  if (e.D > 128 || e.S < 1 || M <= 16 || static_cast<double>(e.B) * e.H * M > 1e9) return false;
  // The tiles walk a sentence's positions one after the other, the split kernel shares them out but pays for
  // every 32 rows again.  Both sides in us, tiles / split, measured at full lengths (head_dim 64, then 128):
  //   1 head, 32 rows x 1024 positions    14.8 / 15.0, 17.0 / 20.5;   x 8192   75.8 / 17.9, 81 / 23.5
  //   32 heads, 128 rows x 1024           16.1 / 24.9, 18.7 / 28.8;   x 8192   79.0 / 69.7, 91 / 113
  //   256 heads, 32 rows x 1024           18.0 / 30.0, 28.8 / 45.9;   512 rows x 8192   342 / 1786, 415 / 3111
  // (and up to 16 rows, where the split kernel needs one mma tile, 14.9 / 10.8 and 92 / 100 at the ends).
  // Where the split kernel does not split (up to SP_WHOLE units) it wins on short sentences as long as its CTAs are
  // resident at once, and by less where they share an SM:
  //   up to 152 segments of 32 rows x 32    5.4 / 7.5 (split / tiles), 6.2 / 9.5;   x 256   8.1 / 8.6, 10.6 / 10.5
  //   256 segments x 128                    8.7 / 8.9, 10.5 / 11.4;                 x 256   11.3 / 10.5, 14.0 / 12.8
  //   512 segments x 32                     11.4 / 9.1, 14.4 / 11.0
  const bool wide = e.D > 64;
  const double heads = static_cast<double>(e.B) * e.H, tiles = heads * ((M + TC_M - 1) / TC_M);
  const double tc = (wide ? 8.0 : 6.0) + tiles_us(static_cast<int64_t>(tiles), e.S, num_sms);
  const double alone = wide ? std::min(24.0, std::max(12.0, 6.0 + e.S / 70.0))
                            : std::min(18.0, std::max(9.3, 5.0 + e.S / 100.0));
  const double split = alone + heads * ((M + 31) / 32) * ((e.S - 1) / 16 + 1) * (wide ? 0.0015 : 0.00085);
  if (e.S <= 16 * SP_WHOLE) {
    const double segments = heads * ((M + 31) / 32);
    if (segments <= 2 * num_sms && e.S <= (wide ? 256 : 384) / (segments > num_sms ? 2 : 1)) return false;
  } else if (tc > split) {
    return false;
  }
  auto stride_ok = [](int64_t s, int64_t extent) { return extent == 1 || (s > 0 && s % 8 == 0 && s < (int64_t{1} << 38)); };
  return ((reinterpret_cast<uintptr_t>(e.k) | reinterpret_cast<uintptr_t>(e.v)) & 15) == 0 && stride_ok(e.k_sent, e.B) &&
         stride_ok(e.k_pos, e.S) && stride_ok(e.k_head, e.H) && stride_ok(e.v_sent, e.B) && stride_ok(e.v_pos, e.S) &&
         stride_ok(e.v_head, e.H) && tensor_map_encode() != nullptr;
}

template <int DP>
static int launch_tc(const CUtensorMap& km, const CUtensorMap& vm, const TcArgs& a, int num_sms, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};
  if (!smem_attr_once(xattn_tc_kernel<DP>, static_cast<int>(TcCfg<DP>::SMEM), attr_done)) return VBS_ECUDA;
  const int grid = std::min(a.B * a.H * a.tiles, 2 * num_sms);
  xattn_tc_kernel<DP><<<grid, TC_NT, TcCfg<DP>::SMEM, s>>>(km, vm, a);
  return cudaGetLastError() == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

int launch_xattn_tc(const EncKV& e, const QO& io, int num_sms, cudaStream_t s) {
  CUtensorMap km, vm;
  if (!encode(&km, e.k, e, e.k_sent, e.k_pos, e.k_head) || !encode(&vm, e.v, e, e.v_sent, e.v_pos, e.v_head)) return VBS_ECUDA;
  auto eights = [](const void* p, int64_t r, int64_t t, int64_t h) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (r | t | h) % 8 == 0;
  };
  const int G = io.Hq / e.H, M = e.W * io.n_q * G;
  const TcArgs a{io, e.len, e.status, e.S, e.B, e.W, e.H, e.D, G, M, (M + TC_M - 1) / TC_M,
                 eights(io.q, io.q_row, io.q_tok, io.q_head), eights(io.o, io.o_row, io.o_tok, io.o_head),
                 sort_pays(e.B, static_cast<int64_t>(e.B) * e.H * ((M + TC_M - 1) / TC_M), e.S, num_sms)};
  return e.D <= 64 ? launch_tc<64>(km, vm, a, num_sms, s) : launch_tc<128>(km, vm, a, num_sms, s);
}

}  // namespace vbs
