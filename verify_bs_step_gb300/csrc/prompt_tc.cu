// Attention of packed prompts to themselves: tcgen05 tiles (sm_103a).
//
// An item is 2 x 128 query rows (128 at head_dim above 128, and where there are few) of one K/V head (2 TT tokens in
// their packed order, whatever requests they are of, the heads of a group side by side) over the positions that any of
// them sees, PT_N at a time (where there are few rows, each of two chains takes half of the positions):
//   S = Q K^T     tcgen05.mma, Q and K in shared memory (128-byte swizzle), S in TMEM, one buffer a row tile;
//   softmax       four warps a row tile, one thread a row: S from TMEM to registers, weights back to TMEM as bf16;
//   O += P V      tcgen05.mma, P from TMEM, V in shared memory as it comes, O in TMEM.
// The row tiles share K and V.  Of the other warps one loads K and V by TMA, one a row tile issues its products, four
// look through V (below) and bring results out, and one works out the next items (which positions each token sees) and
// loads their Q.
// The grid has a block an item, but a CTA goes on with the items of blocks that have not started (cluster launch
// control), so that CTAs share the work out whatever the requests' lengths, the longest rows first.
//
// A row sees the positions [x, y): its request's first token up to its own (causal) or its request's last.  Scores past
// them are set to -inf in TMEM, in the tiles that some row does not see whole.  There V may hold infinities or NaN that
// a weight of 0 does not make harmless: such elements are put to 0 for the product, and added at the end, times their
// weights, to the rows that see them.
//
// The running reference of the softmax only moves when a row's maximum has grown by 2^8 (in the weights'
// own units): until then weights up to 256 are as good in bf16 as weights up to 1, and O stays where it is.
// The weights' bf16 rounding is the one rounding besides the result's; their sum is taken before it.
//
// What bounds it is a row tile's chain: a tile of 128 x 128 at head_dim 128 costs 1100 to 1500 clocks of softmax (512 of
// them exponentials, at 32 a clock and SM), the second half of its product with V and the next scores 768, and some 330 from
// an instruction to its barrier, while S and P share their 128 TMEM columns; two chains fill 60 to 65 % of the tensor pipe
// (16001 tokens x 32 heads: 1.37 to 1.47 ms by the clock that power leaves, 1420 TFLOP/s and more, 75 % of the measured
// burst).  Requests of 1000 tokens add an item's start and end, some 6000 of 20000 clocks (64 of them: 540 us, 970 TFLOP/s);
// 128 sentences of up to 256 tokens, 8 heads x 64, take 39 us.  TMEM is full: two S and two O of 128 columns.
// What counted on the way: all roles' code of a tile together has to stay short, or one warp's pushes another's out of the
// instruction cache (unexecuted paths alone cost 733 against 633 us); results through shared memory (a lane a row took 6000
// clocks an item); weights handed over in halves; a warp a row tile for the products; an item's V, results and next
// item on warps of their own.  Measured and not kept: a lock around a row tile's products (1491 against 1466 us), whole warps
// that issue (1665 against 1462), results and V in an event loop (735 against 690), each row tile's own K and V where the two
// see different requests (no gain, and longer code), Q taken to the L2 ahead of its load (561 against 557), the halves of a
// tile that no row of a warp sees left out (571 against 549: the code), masks and maxima in one pass (553 against 549).

#include <climits>

#include <cuda_bf16.h>

#include "launch.cuh"
#include "pairs.cuh"
#include "prompt.h"
#include "tc.cuh"

namespace vbs {

constexpr int PT_M = 128;                 // query rows a tile
constexpr int PT_N = 128;                 // positions a tile
constexpr int PT_SM = 256;                // softmax threads: one a row of both tiles
constexpr int PT_OUT = 128;               // threads that look through V and bring results out
constexpr int PT_NT = PT_SM + PT_OUT + 128;   // and warps for the loads, each row tile's products, and the items
constexpr int PT_W_OUT = PT_SM / 32, PT_W_LOAD = PT_W_OUT + PT_OUT / 32, PT_W_MMA = PT_W_LOAD + 1;
constexpr int PT_RING = 4;                // items on their way
constexpr int PT_CU = 2048;               // request starts held in shared memory
// Below so many requests every CTA looks at all of them while it waits for its first scores, from here on a launch before the
// tiles does (us a call, the first / the second: 5000 requests of 2000 tokens x 4 heads 12.5 / 16.2; and, the CTAs looking
// before they start, 21333 of 64000 x 8 80 / 74, 100000 of 2000 x 4 63 / 24).
constexpr int PT_LOOK = 8192;
constexpr int PT_STMAX = 4;
// Items of this many tiles and more: the row tiles' products go in turn, so that one's run while the other's softmax
// does.  Left alone both fall into step and wait together (16001 tokens: 1605 us alone, 1432 in turn; 64 x 1000, whose
// items have up to 9 tiles: 567 alone, 553 in turn from 5 tiles on, 559 from 7; 128 sentences up to 256: 43 alone, 45 in
// turn from 3 on).
constexpr int PT_TURNS = 5;
// registers a thread: 65,536 / 512 at launch, then the softmax threads take what the others leave
constexpr int PT_REGS = 128, PT_REGS_SM = 168, PT_REGS_OUT = 104, PT_REGS_REST = 72;
static_assert(PT_SM * PT_REGS_SM + PT_OUT * PT_REGS_OUT + 128 * PT_REGS_REST <= PT_NT * PT_REGS, "registers of the block");

struct PtArgs {
  PromptArgs p;
  int G, TT;                              // heads a group, tokens a row tile
  int per, tiles;                         // an item's tokens, TT or 2 TT; items a K/V head
  int batch, many;                        // the grid's first `many` blocks stand for `batch` items each, the others for one
  bool out16;                             // stores of 16 bytes
};

template <int DP> struct PtCfg {
  static constexpr int SLABS = DP / 64;                    // 64 dims: 128 bytes a row
  static constexpr int QB = SLABS * PT_M * 128;            // one row tile of Q
  static constexpr int TB = SLABS * PT_N * 128;            // one tile of K or V
  static constexpr int X = DP == 256 ? 1 : 2;              // row tiles an item: what fits TMEM
  static constexpr int ST = DP == 64 ? 4 : (DP == 128 ? 2 : 1);   // stages of K, and of V
  static constexpr int OUT = 32 * 64;                      // a warp's rows of 32 dims on their way out
  static constexpr size_t SMEM = X * QB + 2 * ST * TB + PT_CU * 4 + PT_OUT / 32 * OUT + 1024;
};

// Rings of barriers: kf, vf (a tile has landed), ke, ve (it is not read any more); vx and vc in place of vf where not
// every row sees the whole tile (it has landed, has been looked through): a barrier's phases count its own uses alone, so
// that who waits for one is never two behind.  Per row tile: q, qe (an item's Q has
// landed, is not read any more), s (scores are done), p (the weights of half a tile are written), o (an item's sums are
// done), of (they have been read), go (it is its turn to issue).  itf, ite: an item is worked out, is done with.  near:
// the load of its last tile begins.  claim: the answer of a claim is there.
// end: every product that was issued is done.
struct PtBars {
  u64 kf[PT_STMAX], ke[PT_STMAX], vf[PT_STMAX], ve[PT_STMAX], q[2], qe[2], s[2], p[2][2], o[2], of[2], vx[PT_STMAX],
      vc[PT_STMAX], go[2], itf[PT_RING], ite[PT_RING], near[PT_RING], claim, end;
};

struct PtItem {
  int tok, h;                             // first token; h < 0: no more items
  int base;                               // the first position
  int n;                                  // tiles of positions
  int y1[2];                              // the end of what a row tile sees, counted from the first position
  int j0[2], j1[2];                       // its tiles
  int w0, w1;                             // tiles that every row of both sees whole: their V is used as it is
  int odd0, odd1;                         // the first and the last tile of whose V elements were put to 0; none: odd0 > odd1
};

// Steps of 16 positions of tile j that a row tile sees some of.
__device__ __forceinline__ int steps_of(int y1, int j) { return min(PT_N, y1 - j * PT_N + 15) >> 4; }

// Adds to a chain's 32 sums of a lane's row r of row tile X, from dim c on, the elements of V in its tiles j0 .. j1 - 1 that
// were put to 0 for the product and that the row sees, times their weights relative to the chain's reference (0 times an
// infinity is NaN, as in the product): they are outside the tiles that every row sees whole.  By a converged warp, whose
// lanes look for such positions 32 at a time.
__device__ __forceinline__ void add_odd(const PtArgs& a, const PtItem& it, const int2* spans, int X, int r, int j0, int j1,
                                        float ref, int c, float* o) {
  const PromptArgs& p = a.p;
  const int lane = threadIdx.x & 31, t = X * a.TT + r / a.G;
  const int2 sp = r < a.TT * a.G ? spans[t] : make_int2(0, 0);
  const int x0 = sp.y > sp.x ? sp.x - it.base : INT_MAX, x1 = sp.y > sp.x ? sp.y - it.base : 0;
  const int first = __reduce_min_sync(FULL, x0), end = __reduce_max_sync(FULL, x1);
  const uint16_t* q = p.q + static_cast<int64_t>(it.tok + t) * p.q_tok + static_cast<int64_t>(it.h * a.G + r % a.G) * p.q_head;
  u32 nan = sp.y > sp.x ? 0u : ~0u;                       // the sums that are NaN, and stay so (or are none)
  for (int i = 0; i < 32; ++i) nan |= o[i] == o[i] && c + i < p.D ? 0u : 1u << i;
  for (int j = j0; j < j1; ++j) {
    if (j >= it.w0 && j < it.w1) continue;
    const int y1 = min(end, (j + 1) * PT_N);
    for (int y = max(first, j * PT_N); y < y1; y += 32) {
      if (__all_sync(FULL, nan == ~0u)) return;
      u32 bad = 0;                                        // of the lane's position
      if (y + lane < y1) {
        const uint16_t* v = p.v + static_cast<int64_t>(it.base + y + lane) * p.v_tok + it.h * p.v_head + c;
        for (int i = 0; i < 32 && c + i < p.D; i += 8) {
          float f[8];
          Vec16<bf16_t>::unpack(*reinterpret_cast<const uint4*>(v + i), f);
          for (int e = 0; e < 8; ++e) bad |= fabsf(f[e]) < INFINITY ? 0u : 1u << (i + e);
        }
      }
      for (u32 which = __ballot_sync(FULL, bad != 0); which != 0; which &= which - 1) {
        const int n = y + __ffs(which) - 1;
        u32 dims = __shfl_sync(FULL, bad, n - y) & ~nan;
        if (dims == 0 || n < x0 || n >= x1) continue;
        const uint16_t* k = p.k + static_cast<int64_t>(it.base + n) * p.k_tok + it.h * p.k_head;
        float s = 0.f, f[8], g[8];
        for (int d = 0; d < p.D; d += 8) {
          Vec16<bf16_t>::unpack(*reinterpret_cast<const uint4*>(q + d), f);
          Vec16<bf16_t>::unpack(*reinterpret_cast<const uint4*>(k + d), g);
          for (int e = 0; e < 8; ++e) s = fmaf(f[e], g[e], s);
        }
        const float w = ex2(s * (p.scale * LOG2E_F) - ref);
        const uint16_t* v = p.v + static_cast<int64_t>(it.base + n) * p.v_tok + it.h * p.v_head + c;
        for (; dims != 0; dims &= dims - 1) {
          const int i = __ffs(dims) - 1;
          o[i] += bf16_lo(v[i]) * w;
          nan |= o[i] == o[i] ? 0u : 1u << i;
        }
      }
      __syncwarp();
    }
  }
}

// The same for all sums of a row, in TMEM from `to` on (both: of two chains, side by side), with the row tiles' or chains'
// references.  (A function of its own, loads and stores too: inline, though it hardly ever runs, it cost 5 % where items
// are short: 2000 requests of 64000 tokens.)
template <int DP, bool SPLIT>
__device__ __noinline__ void add_odd_all(const PtArgs& a, const PtItem& it, const int2* spans, int X, int r, u32 to, bool both,
                                         const float* ref0, const float* ref1) {
  const int odd0 = __shfl_sync(FULL, it.odd0, 0), odd1 = __shfl_sync(FULL, it.odd1, 0), half = (it.n + 1) / 2;
#pragma unroll 1
  for (int c = 0; c < (both ? 2 * DP : DP); c += 32) {
    const int Y = SPLIT ? c / DP : X;
    float o[32];
    tc_ld32(to + c, o);
    tc_wait_ld();
    add_odd(a, it, spans, X, r, max(odd0, SPLIT ? Y * half : it.j0[X]), min(odd1 + 1, SPLIT ? (Y ? it.n : half) : it.j1[X]),
            Y ? *ref1 : *ref0, c % DP, o);
    tc_st32(to + c, o);
  }
  tc_wait_st();
}

__device__ __forceinline__ void tma_load3(u32 dst, const CUtensorMap* map, u64* bar, int x, int h, int t) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(map), "r"(x), "r"(h), "r"(t), "r"(smem_u32(bar)) : "memory");
}

// The last request from b (which starts at or before token t, or is taken for it) to `last` that starts at or before t: by
// steps that double and then halve, as any number of requests may be empty and start there too.
__device__ __forceinline__ int request_after(const int* cu, int b, int last, int t) {
  int step = 1;
  while (step <= last - b && cu[b + step] <= t) {
    b += step;
    step *= 2;
  }
  for (; step > 0; step >>= 1)
    if (step <= last - b && cu[b + step] <= t) b += step;
  return b;
}
// The last request that starts at or before token t, or 0, by a converged warp; one start in `every` is at hand in shared
// memory.
__device__ __forceinline__ int request_before(const PromptArgs& a, const int* cu, int every, int t, int lane) {
  int lo = 0, n = a.B / every + 1;        // it is among the n held from lo on: the last of them not above t
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const u32 below = __ballot_sync(FULL, at < n && cu[lo + at] <= t);
    const int k = max(0, 31 - __clz(below)) * step;
    lo += k;
    n = min(step, n - k);
  }
  return every > 1 ? request_after(a.cu, lo * every, min(a.B, lo * every + every - 1), t) : lo;
}
// Request b's first token and its end; 0, 0 where it is not within the tokens.
__device__ __forceinline__ int2 request_at(const PromptArgs& a, const int* cu, int every, int b) {
  if (b >= a.B) return make_int2(0, 0);
  const int s = every == 1 ? cu[b] : a.cu[b], e = every == 1 ? cu[b + 1] : a.cu[b + 1];
  return s >= 0 && s < e && e <= a.N ? make_int2(s, e) : make_int2(0, 0);
}

// Claims a block of the grid that has not started, in place of its launch (16 bytes of answer, counted by `bar`).
__device__ __forceinline__ void claim_block(uint4* answer, u64* bar) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (the answer before has been read)
  mbar_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
               ::"r"(smem_u32(answer)), "r"(smem_u32(bar)) : "memory");
}
// The claimed block, or -1.
__device__ __forceinline__ int claimed_block(const uint4* answer) {
  u32 got, x;
  asm volatile("{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
               "ld.shared.b128 h, [%2];\n\t"
               "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
               "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
               "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
               : "=r"(got), "=r"(x) : "r"(smem_u32(answer)) : "memory");
  return got ? static_cast<int>(x) : -1;
}

// tc_wait in little code.  Some waits are as long as an item, 128 tokens of whose prompt take up to 3 us: the limit grows by
// a try, some 0.1 us, for each token there is.
__device__ __forceinline__ bool pt_wait(u64* bar, u32 parity, volatile int* gone, const PromptArgs& p) {
#pragma unroll 1
  for (u32 i = 0; !mbar_wait(bar, parity, 1); ++i)
    if (__builtin_expect(i >= TC_SPIN + p.N || *gone, 0)) {
      *gone = 1;
      set_status(p.status, VBS_ETIMEOUT);
      return false;
    }
  return true;
}

// Tells where a request is not within the tokens: threads `at`, `at` + `step`, ... of all that look.
__device__ __forceinline__ void check_requests(const PromptArgs& p, const int* cu, int at, int step) {
  for (int b = at; b < p.B; b += step)
    if (cu[b] < 0 || cu[b] > cu[b + 1] || cu[b + 1] > p.N) set_status(p.status, VBS_EINVAL);
}
// For so many requests that the tiles' CTAs do not look themselves.
__global__ void __launch_bounds__(256) prompt_starts_kernel(const PromptArgs p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  check_requests(p, p.cu, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

// SPLIT: an item is one row tile, the first and the second half of whose positions the two chains take; their sums are
// joined when they are brought out.
template <int DP, bool SPLIT>
__global__ void __launch_bounds__(PT_NT, 1) prompt_tc_kernel(const __grid_constant__ CUtensorMap qmap,
                                                            const __grid_constant__ CUtensorMap kmap,
                                                            const __grid_constant__ CUtensorMap vmap, const PtArgs a) {
  using C = PtCfg<DP>;
  constexpr int ST = C::ST, STEP = SPLIT ? 2 : 1;
  static_assert(!SPLIT || C::X == 2, "a chain each");
  extern __shared__ unsigned char pt_smem_raw[];
  __shared__ __align__(8) PtBars bars;
  __shared__ u32 tmem_base;
  __shared__ volatile int gone;
  __shared__ __align__(16) uint4 claim;
  __shared__ PtItem ring[PT_RING];
  __shared__ int2 span[PT_RING][2 * PT_M];                // positions [x, y) of an item's tokens
  __shared__ float sums[2][2][PT_M];                      // of a row's weights, by the row tile's items in turn
  __shared__ float refs[2][2][PT_M];                      // and what they are relative to

  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  unsigned char* smem = pt_smem_raw + ((1024 - (smem_u32(pt_smem_raw) & 1023)) & 1023);
  const u32 q_a = smem_u32(smem), k_a = q_a + C::X * C::QB, v_a = k_a + ST * C::TB;
  unsigned char* out_s = smem + C::X * C::QB + 2 * ST * C::TB;
  int* cu = reinterpret_cast<int*>(out_s + PT_OUT / 32 * C::OUT);
  const PromptArgs& p = a.p;
  const int every = (p.B + 1 + PT_CU - 1) / PT_CU;        // one start in `every` is held

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bars.kf[i], 1);
      mbar_init(&bars.ke[i], 2);
      mbar_init(&bars.vf[i], 1);
      mbar_init(&bars.ve[i], 2);
      mbar_init(&bars.vx[i], 1);
      mbar_init(&bars.vc[i], PT_OUT);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q[i], 1);
      mbar_init(&bars.go[i], 1);
      mbar_init(&bars.qe[i], 1);
      mbar_init(&bars.s[i], 1);
      mbar_init(&bars.p[i][0], PT_M);
      mbar_init(&bars.p[i][1], PT_M);
      mbar_init(&bars.o[i], 1);
      mbar_init(&bars.of[i], PT_OUT);
    }
    for (int i = 0; i < PT_RING; ++i) {
      mbar_init(&bars.itf[i], 1);
      mbar_init(&bars.near[i], 1);
      mbar_init(&bars.ite[i], (PT_SM + PT_OUT) / 32 + 3);
    }
    mbar_init(&bars.claim, 1);
    mbar_init(&bars.end, 2);
    fence_mbar_init();
    gone = 0;
  }
  if (wid == PT_W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // a dependent launch: set up before, reads and writes nothing before its predecessor's end
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = tid; i * every <= p.B; i += PT_NT) cu[i] = p.cu[i * every];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const u32 tm = tmem_base, tm_s = tm, tm_o = tm + 2 * PT_N;

  // the place among an item's tiles of positions of the j-th that is loaded; a chain takes every STEP-th
  auto place = [](int n, int j) { return SPLIT ? (j & 1) * ((n + 1) / 2) + (j >> 1) : j; };
  auto item_at = [&](int t) { return pt_wait(&bars.itf[t % PT_RING], (t / PT_RING) & 1, &gone, p); };

  if (wid < PT_W_OUT) {
    // ---- softmax: thread = row ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PT_REGS_SM));
    const int X = wid >> 2, r = tid & (PT_M - 1);          // row tile, row
    const u32 tl = static_cast<u32>((wid & 3) * 32) << 16;  // its TMEM lanes
    // every CTA looks at the requests while it waits for its first scores: no block is certain to be launched, as others may
    // claim its items
    if (p.B < PT_LOOK) check_requests(p, every == 1 ? cu : p.cu, tid, PT_SM);
    const u32 ts = tm_s + X * PT_N + tl, to = tm_o + X * DP + tl;
    const bool neg = p.scale < 0.f;
    // (a scale of 0 stays above it, so that a masked -inf stays one)
    const float sc = fmaxf(fabsf(p.scale) * LOG2E_F, 1.17549435e-38f);
    const int tok_r = r / a.G;
    bool ok = true;
    int S = 0, O = 0;                                     // score tiles and items of this row tile so far
    for (int t = 0;; ++t) {
      ok = __all_sync(FULL, item_at(t));
      const PtItem& it = ring[t % PT_RING];
      if (!ok || it.h < 0) break;
      const int2 sp = r < a.TT * a.G ? span[t % PT_RING][(SPLIT ? 0 : X) * a.TT + tok_r] : make_int2(0, 0);
      // counted from the item's first position; rows that are not there see all of it (they are not written)
      const int x0 = sp.y > 0 ? sp.x - it.base : 0, x1 = sp.y > 0 ? sp.y - it.base : INT_MAX / 2;
      const int j0 = it.j0[X], j1 = it.j1[X];
      // the reference (in scaled units), the sum of weights.  Rows that are not there, whose scores are what shared memory
      // and TMEM held before, have NaN, which stays one and is never above a limit: they have no say in the votes below
      float m = sp.y > 0 ? -INFINITY : __int_as_float(0x7fffffff), l = 0.f;
      for (int j = j0; j < j1; j += STEP, ++S) {
        const int y = place(it.n, j) * PT_N, from = x0 - y, left = x1 - y;
        ok = __all_sync(FULL, pt_wait(&bars.s[X], S & 1, &gone, p));
        if (!ok) break;
        tc_fence_after();
        // (the code of a tile is kept short, in loops over its halves: of several warps' long code one pushes the other's
        // out of the instruction cache, tile by tile)
        if (__any_sync(FULL, from > 0 || left < PT_N) || neg) {
          // scores that a row does not see become -inf where they stand (and all change their sign under a negative
          // scale), where there are such
          const int least = __reduce_min_sync(FULL, left), late = __reduce_max_sync(FULL, from);
#pragma unroll 1
          for (int c = 0; c < PT_N; c += 32) {
            if (least >= c + 32 && late <= c && !neg) continue;
            const int lo = max(0, from - c), hi = left - c;
            u32 see = hi >= 32 ? ~0u : (hi <= 0 ? 0u : (1u << hi) - 1u);
            see = lo >= 32 ? 0u : see & (~0u << lo);
            float x[32];
            tc_ld32(ts + c, x);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = see >> i & 1u ? (neg ? -x[i] : x[i]) : -INFINITY;
            tc_st32(ts + c, x);
          }
          tc_wait_st();
        }
        float mx = -INFINITY, s[64];
#pragma unroll 1
        for (int c = 0; c < PT_N; c += 64) {
          tc_ld32(ts + c, s);
          tc_ld32(ts + c + 32, s + 32);
          tc_wait_ld();
          float x[4] = {mx, fmaxf(s[0], s[1]), fmaxf(s[2], s[3]), fmaxf(s[4], s[5])};
#pragma unroll
          for (int i = 6; i < 64; i += 2) x[(i >> 1) & 3] = max3(x[(i >> 1) & 3], s[i], s[i + 1]);
          mx = max3(fmaxf(x[0], x[1]), x[2], x[3]);
        }
        mx *= sc;
        float f = sc;
        const bool grow = mx > m + 8.f;                   // also in the first tile that a row sees: m = -inf
        if (__any_sync(FULL, grow || (fabsf(m) > 65536.f && m > -INFINITY))) {
          const float to_m = grow ? mx : m, corr = grow ? (m == -INFINITY ? 0.f : ex2(m - to_m)) : 1.f;
          if (j > j0) {
            // O holds the tiles before (S of this one was issued after their products, and is done)
#pragma unroll 1
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
          // scale and reference go into one fma, whose product is not rounded as the reference was: for
          // large scores the difference is more than a weight can bear, and the product is rounded first
          if (__any_sync(FULL, fabsf(m) > 65536.f && m > -INFINITY)) {
            f = 1.f;
#pragma unroll 1
            for (int c = 0; c < PT_N; c += 16) {
              float o[16];
              tc_ld16(ts + c, o);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= sc;
              tc_st16(ts + c, o);
            }
            tc_wait_st();
            tc_ld32(ts + 64, s);
            tc_ld32(ts + 96, s + 32);
            tc_wait_ld();
          }
          tc_wait_st();
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const u64 f2 = pair(f, f), r2 = pair(-ref, -ref);
        u64 sum[2] = {0, 0};
        // the second half first: its scores are still at hand (1388 us to 1366 for 16001 tokens)
#pragma unroll 1
        for (int c = 64; c >= 0; c -= 64) {
          if (c == 0) {
            tc_ld32(ts, s);
            tc_ld32(ts + 32, s + 32);
            tc_wait_ld();
          }
#pragma unroll
          for (int h = 0; h < 64; h += 32) {
            float pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x, y;
              unpair(fma2(pair(s[h + 2 * i], s[h + 2 * i + 1]), f2, r2), x, y);
              x = ex2(x);
              y = ex2(y);
              sum[i & 1] = add2(sum[i & 1], pair(x, y));
              __nv_bfloat162 w = __floats2bfloat162_rn(x, y);
              pk[i] = *reinterpret_cast<float*>(&w);
            }
            tc_st16(ts + c + h / 2, pk);                  // the weights stand where scores were
          }
          if (c == 0) {
            float l0, l1;
            unpair(add2(sum[0], sum[1]), l0, l1);
            l += l0 + l1;
            if (j + STEP >= j1) {
              sums[O & 1][X][r] = l;
              refs[O & 1][X][r] = m;
            }
          }
          tc_wait_st();
          tc_fence_before();
          mbar_arrive(&bars.p[X][c >> 6]);
        }
      }
      if (!ok) break;
      if (j1 > j0) ++O;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.ite[t % PT_RING]);
    }
    tc_wait_st();                                         // (weights of a tile that was given up)
    tc_fence_before();
  } else if (wid < PT_W_LOAD) {
    // ---- V where not every row sees the whole tile (thread = position), and results (thread = row) ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PT_REGS_OUT));
    const int r = tid & (PT_M - 1), tok_r = r / a.G, g = r - tok_r * a.G;
    const u32 tl = static_cast<u32>((wid & 3) * 32) << 16;
    unsigned char* mine = out_s + (wid - PT_W_OUT) * C::OUT;
    auto wait = [&](u64* bar, u32 parity) { return __all_sync(FULL, pt_wait(bar, parity, &gone, p)) != 0; };
    u32 turn = 0, o_turn = 0;                             // of each stage's vx, and of the row tiles' o
    int T = 0;
    bool ok = true;
    int looked = 0;                                       // tiles of the next item that have been looked through
    for (int t = 0; ok; ++t) {
      if (!wait(&bars.itf[t % PT_RING], (t / PT_RING) & 1)) break;
      if (ring[t % PT_RING].h < 0) break;
#pragma unroll 1
      for (int u = t; u <= t + 1 && ok; ++u) {
        // the next item's first tiles too, where it is there, so that they do not wait for this one's results
        if (u > t && !__all_sync(FULL, mbar_wait(&bars.itf[u % PT_RING], (u / PT_RING) & 1, 1))) break;
        const PtItem& it = ring[u % PT_RING];
        if (it.h < 0) break;
        const int e = u == t ? it.n : min(it.n, ST / 2);
#pragma unroll 1
        for (int j = u == t ? looked : 0; j < e; ++j) {
          if (place(it.n, j) >= it.w0 && place(it.n, j) < it.w1) continue;
          const int st = (T + j) % ST;
          ok = wait(&bars.vx[st], turn >> st & 1);
          if (!ok) break;
          turn ^= 1u << st;
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
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint4 w = row[c];
                u32* e = &w.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if ((e[i] & 0x7f80u) == 0x7f80u) e[i] &= 0xffff0000u;
                  if ((e[i] & 0x7f800000u) == 0x7f800000u) e[i] &= 0x0000ffffu;
                }
                row[c] = w;
              }
              atomicMin(&ring[u % PT_RING].odd0, place(it.n, j));
              atomicMax(&ring[u % PT_RING].odd1, place(it.n, j));
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          mbar_arrive(&bars.vc[st]);
        }
        if (u == t) T += it.n;
        looked = u == t ? 0 : e;
      }
      const PtItem& it = ring[t % PT_RING];
#pragma unroll 1
      for (int X = 0; X < (SPLIT ? 1 : 2) && ok; ++X) {
        if (it.j1[X] <= it.j0[X]) continue;
        ok = wait(&bars.o[X], o_turn >> X & 1);
        if (!ok) break;
        const bool both = SPLIT && it.n > 1;
        if (both) {
          ok = wait(&bars.o[1], o_turn >> 1);
          if (!ok) break;
        }
        tc_fence_after();
        const u32 to = tm_o + X * DP + tl;
        if (__builtin_expect(__any_sync(FULL, it.odd0 <= it.odd1), 0))
          add_odd_all<DP, SPLIT>(a, it, span[t % PT_RING], X, r, to, both, &refs[o_turn & 1][0][r], &refs[o_turn >> 1][1][r]);
        float inv, other = 0.f;                           // what the sums are multiplied by (0 / 0 where every score is -inf: NaN)
        if (SPLIT) {
          const float m0 = refs[o_turn & 1][0][r], m1 = both ? refs[o_turn >> 1][1][r] : -INFINITY;
          const float l1 = both ? sums[o_turn >> 1][1][r] : 0.f, m = fmaxf(m0, m1), ref = m == -INFINITY ? 0.f : m;
          inv = ex2(m0 - ref);
          other = ex2(m1 - ref);
          const float k = 1.f / (sums[o_turn & 1][0][r] * inv + l1 * other);
          inv *= k;
          other *= k;
          o_turn ^= both ? 3u : 1u;
        } else {
          inv = 1.f / sums[o_turn >> X & 1][X][r];
          o_turn ^= 1u << X;
        }
        const int2 sp = r < a.TT * a.G ? span[t % PT_RING][X * a.TT + tok_r] : make_int2(0, 0);
        uint16_t* out = sp.y > sp.x ? p.o + static_cast<int64_t>(it.tok + X * a.TT + tok_r) * p.o_tok +
                                          static_cast<int64_t>(it.h * a.G + g) * p.o_head
                                    : nullptr;
        // 32 dims at a time through shared memory, so that a warp stores 64 bytes of 8 rows at once (a lane a row
        // takes 32 lines a store)
        uint16_t* at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = reinterpret_cast<uint16_t*>(shfl64(reinterpret_cast<u64>(out), i * 8 + lane / 4));
#pragma unroll 1
        for (int c = 0; c < DP; c += 32) {
          float o[32], o1[32];
          tc_ld32(to + c, o);
          if (both) tc_ld32(to + DP + c, o1);
          tc_wait_ld();
          if (c + 32 == DP) {
            tc_fence_before();
            mbar_arrive(&bars.of[X]);                     // O may be written again
            if (both) mbar_arrive(&bars.of[1]);
          }
          if (SPLIT) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= inv;
            if (both) {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = fmaf(o1[i], other, o[i]);
            }
          }
          __syncwarp();                                   // the 32 dims before have been read
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u32 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float f = SPLIT ? 1.f : inv;
              const __nv_bfloat162 b = __floats2bfloat162_rn(o[8 * i + 2 * k] * f, o[8 * i + 2 * k + 1] * f);
              w[k] = *reinterpret_cast<const u32*>(&b);
            }
            *reinterpret_cast<uint4*>(mine + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
          const int d = c + lane % 4 * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = i * 8 + lane / 4;
            const unsigned char* x = mine + row * 64 + ((lane % 4 ^ (row >> 1 & 3)) << 4);
            if (!at[i] || d >= p.D) continue;
            if (a.out16) {
              *reinterpret_cast<uint4*>(at[i] + d) = *reinterpret_cast<const uint4*>(x);
            } else {
#pragma unroll 1
              for (int k = 0; k < 8; ++k) at[i][d + k] = reinterpret_cast<const uint16_t*>(x)[k];
            }
          }
        }
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&bars.ite[t % PT_RING]);
    }
    tc_fence_before();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PT_REGS_REST));
    if (wid == PT_W_LOAD) {
      // ---- loads: one lane ----
      if (lane == 0) {
        int T = 0;                                          // tiles of K and V on their way
        u32 whole = 0, look = 0, kind = 0;                  // turns of each stage's vf and vx, and whether vx was the last
        bool ok = true;
        for (int t = 0; ok && item_at(t) && ring[t % PT_RING].h >= 0; ++t) {
          const PtItem& it = ring[t % PT_RING];
          const int n = it.n, h = it.h, base = it.base, w0 = it.w0, w1 = it.w1;
          for (int j = 0; ok && j < n; ++j) {
            if (j == n - 1) mbar_arrive(&bars.near[t % PT_RING]);
            const int st = T % ST;
            const u32 free_turn = ((T / ST) & 1) ^ 1;
            ok = T < ST || pt_wait(&bars.ke[st], free_turn, &gone, p);
            if (!ok) break;
            mbar_expect_tx(&bars.kf[st], C::TB);
            for (int x = 0; x < C::SLABS; ++x)
              tma_load3(k_a + st * C::TB + x * PT_N * 128, &kmap, &bars.kf[st], x * 64, h, base + place(n, j) * PT_N);
            const bool odd_tile = place(n, j) < w0 || place(n, j) >= w1;
            u64* bar = odd_tile ? &bars.vx[st] : &bars.vf[st];
            ok = T < ST || pt_wait(&bars.ve[st], free_turn, &gone, p);
            if (ok) {
              mbar_expect_tx(bar, C::TB);
              for (int x = 0; x < C::SLABS; ++x)
                tma_load3(v_a + st * C::TB + x * PT_N * 128, &vmap, bar, x * 64, h, base + place(n, j) * PT_N);
              if (odd_tile) look ^= 1u << st;
              else whole ^= 1u << st;
              kind = (kind & ~(1u << st)) | (odd_tile ? 1u << st : 0u);
            }
            ++T;
          }
          if (ok) mbar_arrive(&bars.ite[t % PT_RING]);
        }
        // no copy is in flight when the CTA ends, also where it gave up: the last ones have landed
        for (int x = max(0, T - ST); x < T; ++x) {
          const int st = x % ST;
          mbar_wait(&bars.kf[st], (x / ST) & 1, 1u << 16);
          mbar_wait(kind >> st & 1 ? &bars.vx[st] : &bars.vf[st], ((kind >> st & 1 ? look : whole) >> st & 1) ^ 1, 1u << 16);
        }
      }
      __syncwarp();
    } else if (wid < PT_W_MMA + 2) {
      // ---- products: a warp a row tile, of which one thread waits and issues.  The scores of the next tile, be it the
      // next item's first, follow the product with V ----
      if (elect_one()) {
        const int X = wid - PT_W_MMA;
        const u32 dq = static_cast<u32>(tc_desc(q_a + X * C::QB, 16)), dk = static_cast<u32>(tc_desc(k_a, 16)),
                  dv = static_cast<u32>(tc_desc(v_a, PT_N * 128)), ts = tm_s + X * PT_N, to = tm_o + X * DP;
        u32 go_turn = X ? 0 : 1;                            // the first row tile's turn comes first
        u32 p_turn = 0, o_turn = 1, q_turn = 0;             // of the row tile's barriers
        u32 whole = 0, look = 0;                            // and of each stage's vf and vc
        auto wait = [&](u64* bar, u32 parity) { return pt_wait(bar, parity, &gone, p); };
        int at = 0, t = 0, j = 0, n = 0, j0 = 0, j1 = 0, y1 = 0, w0 = 0, w1 = 0;
        u32 turns = 0;                                      // whether the row tiles take turns over this item
        // Item t, as the row tile sees it; whether there is one.
        auto take = [&] {
          if (!item_at(t)) return false;
          const PtItem& i = ring[t % PT_RING];
          n = i.n, j0 = i.j0[X], j1 = i.j1[X], y1 = i.y1[X], w0 = i.w0, w1 = i.w1, j = 0;
          turns = !SPLIT && n >= PT_TURNS ? 1u : 0u;
          return i.h >= 0;
        };
        bool go = take();
        int steps = 0;                                      // of the tile whose weights come next; 0: not this row tile's
        bool first = false, last = false;
        // (the loop's first half has nothing to do yet)
        for (bool begin = true; go; begin = false) {
          if (!begin) {
            const int st = at % ST;
            const bool clear = place(n, j) >= w0 && place(n, j) < w1;
            if (!wait(clear ? &bars.vf[st] : &bars.vc[st], (clear ? whole : look) >> st & 1)) break;
            if (clear) whole ^= 1u << st;
            else look ^= 1u << st;
            if (steps > 0) {
              if (first) {                                  // the item before has been read
                if (!wait(&bars.of[X], o_turn)) break;
                o_turn ^= 1;
              }
              const u32 d = dv + st * (C::TB >> 4);
              u32 acc = first ? 0 : 1;
              bool ok = true;
  #pragma unroll
              for (int half = 1; half >= 0; --half) {
                ok = wait(&bars.p[X][half], p_turn) && (half == 1 || !turns || wait(&bars.go[X], go_turn));
                if (!ok) break;
                tc_fence_after();
                const u32 w = ts + half * (PT_N / 2), v = d + half * (PT_N / 2 * 128 >> 4);
                if (steps >= (half + 1) * (PT_N / 32)) {
  #pragma unroll
                  for (int k = 0; k < PT_N / 32; ++k) tc_mma_ts_at(to, w + k * 8, v + k * (2048 >> 4), tc_idesc(DP, true), k > 0 ? 1u : acc);
                } else {
  #pragma unroll 1
                  for (int k = 0; k < steps - half * (PT_N / 32); ++k)
                    tc_mma_ts_at(to, w + k * 8, v + k * (2048 >> 4), tc_idesc(DP, true), k > 0 ? 1u : acc);
                }
                if (steps > half * (PT_N / 32)) acc = 1;
              }
              if (!ok) break;
              go_turn ^= turns;
              p_turn ^= 1;
              tc_commit(&bars.ve[st]);                      // V may be loaded again
              if (last) tc_commit(&bars.o[X]);
            } else {
              mbar_arrive(&bars.ve[st]);
              if (turns && !wait(&bars.go[X], go_turn)) break;
              go_turn ^= turns;
            }
            ++at;
            if (++j == n) {
              if (turns) mbar_arrive(&bars.go[X ^ 1]);
              mbar_arrive(&bars.ite[t % PT_RING]);
              ++t;
              go = take();
              if (!go) break;
            }
          }
          const int st = at % ST;
          const bool on = j >= j0 && j < j1 && (!SPLIT || (j & 1) == X);
          steps = on ? steps_of(y1, place(n, j)) : 0;
          first = j == j0;
          last = j + STEP >= j1;
          if (!wait(&bars.kf[st], (at / ST) & 1)) break;
          if (steps > 0) {
            if (first) {
              if (!wait(&bars.q[X], q_turn)) break;
              q_turn ^= 1;
            }
            const u32 d = dk + st * (C::TB >> 4);
            if (steps == PT_N / 16) {
  #pragma unroll
              for (int k = 0; k < DP / 16; ++k) {
                const u32 in = (k >> 2) * (PT_M * 128 >> 4) + (k & 3) * 2;
                tc_mma_ss_at(ts, dq + in, d + in, tc_idesc(PT_N, false), k > 0);
              }
            } else {
              const u32 what = tc_idesc(steps * 16, false);
  #pragma unroll 1
              for (int k = 0; k < DP / 16; ++k) {
                const u32 in = (k >> 2) * (PT_M * 128 >> 4) + (k & 3) * 2;
                tc_mma_ss_at(ts, dq + in, d + in, what, k > 0);
              }
            }
            tc_commit(&bars.s[X]);
            tc_commit(&bars.ke[st]);                        // K, and after the item's last Q, may be loaded again
            if (last) tc_commit(&bars.qe[X]);
          } else {
            mbar_arrive(&bars.ke[st]);
          }
          if (!begin && j > 0 && turns) mbar_arrive(&bars.go[X ^ 1]);
        }
        // the products in flight read shared memory and TMEM: all are done before either goes, also where the CTA gave up
        tc_commit(&bars.end);
        mbar_wait(&bars.end, 0, 1u << 16);
      }
      __syncwarp();
    } else {
      // ---- items: the last tokens first, which see the most ----
      u32 q_turn = 0, q_some = 0;                           // of the row tiles' Q, bit X, and whether there was one
      int t = 0, c = 0, i, left;                            // this item, and how many from it on are claimed; 0: none is
      auto take = [&](int block) {
        i = block < a.many ? block * a.batch : a.many * a.batch + block - a.many;
        left = block < 0 ? 0 : (block < a.many ? a.batch : 1);
      };
      take(blockIdx.x);
      while (true) {
        const bool last = left == 0;
        // the slot's item before is done with
        if (t >= PT_RING && !__all_sync(FULL, pt_wait(&bars.ite[t % PT_RING], ((t / PT_RING) - 1) & 1, &gone, p))) break;
        PtItem& x = ring[t % PT_RING];
        const int tile = i / p.H, h = last ? -1 : i - tile * p.H, tok0 = (a.tiles - 1 - tile) * a.per;
        int y0[2] = {INT_MAX, INT_MAX}, y1[2] = {0, 0}, z0[2] = {0, 0}, z1[2] = {INT_MAX, INT_MAX};   // of x and y of the spans
        if (!last) {
          int b = request_before(p, cu, every, tok0, lane);
          int2 at = request_at(p, cu, every, b);
          const int end = min(a.per, p.N - tok0);
          for (int w = lane; w < 2 * PT_M; w += 32) {
            const int tok = tok0 + w;
            if (!__all_sync(FULL, (tok >= at.x && tok < at.y) || w >= end)) {
              // the group's tokens are of several requests: each lane goes on to its own
              if (w < end) b = request_after(every == 1 ? cu : p.cu, b, p.B - 1, tok);
              __syncwarp();
              at = request_at(p, cu, every, b);
            }
            const bool live = w < end && tok >= at.x && tok < at.y;
            const int2 sp = live ? make_int2(at.x, p.causal ? tok + 1 : at.y) : make_int2(0, 0);
  #pragma unroll
            for (int X = 0; X < 2; ++X)
              if (live && (w >= a.TT) == (X == 1)) {
                y0[X] = min(y0[X], sp.x);
                y1[X] = max(y1[X], sp.y);
                z0[X] = max(z0[X], sp.x);
                z1[X] = min(z1[X], sp.y);
              }
            span[t % PT_RING][w] = sp;
            if (w + 32 - lane >= a.per) break;
            b = __shfl_sync(FULL, b, 31);                   // (the last token's)
            at = make_int2(__shfl_sync(FULL, at.x, 31), __shfl_sync(FULL, at.y, 31));
          }
        }
  #pragma unroll
        for (int X = 0; X < 2; ++X) {
          y0[X] = __reduce_min_sync(FULL, y0[X]);
          y1[X] = __reduce_max_sync(FULL, y1[X]);
          z0[X] = __reduce_max_sync(FULL, z0[X]);
          z1[X] = __reduce_min_sync(FULL, z1[X]);
        }
        const int base = min(y0[0], y0[1]);
        if (SPLIT && y1[0] - base > PT_N) y0[1] = y0[0], y1[1] = y1[0], z0[1] = z0[0], z1[1] = z1[0];   // (the same rows)
        const bool some = max(y1[0], y1[1]) > 0;            // (else: tokens of no request)
        if ((some || last) && lane == 0) {
          x.h = h;
          x.tok = tok0;
          x.base = base;
          int n = 0, w0 = 0, w1 = INT_MAX;
  #pragma unroll
          for (int X = 0; X < 2; ++X) {
            const bool on = y1[X] > 0;
            x.y1[X] = on ? y1[X] - base : 0;
            x.j0[X] = on ? (SPLIT ? X : (y0[X] - base) / PT_N) : 0;
            x.j1[X] = on ? (y1[X] - base + PT_N - 1) / PT_N : 0;
            if (on) {
              n = max(n, (y1[X] - base + PT_N - 1) / PT_N);
              w0 = max(w0, (z0[X] - base + PT_N - 1) / PT_N);
              w1 = min(w1, (z1[X] - base) / PT_N);
            }
          }
          x.n = n;
          x.w0 = w0;
          x.w1 = w1;
          x.odd0 = INT_MAX;
          x.odd1 = -1;
        }
        __syncwarp();
        if (some || last) {
          if (lane == 0) mbar_arrive(&bars.itf[t % PT_RING]);
          ++t;
        }
        if (last) break;
        if (some) {
          // its Q, as soon as the item before does not read its own any more (here, so that K and V do not wait for that)
          bool ok = true;
#pragma unroll 1
          for (int X = 0; X < 2; ++X) {
            if ((X ? y1[1] : y1[0]) == 0) continue;
            ok = !(q_some >> X & 1) || __all_sync(FULL, pt_wait(&bars.qe[X], (q_turn >> X & 1) ^ 1, &gone, p));
            if (!ok) break;
            if (lane == 0) {
              mbar_expect_tx(&bars.q[X], C::SLABS * 128 * a.G * a.TT);
              for (int x = 0; x < C::SLABS; ++x)
                tma_load3(q_a + X * C::QB + x * PT_M * 128, &qmap, &bars.q[X], x * 64, h * a.G, tok0 + (SPLIT ? 0 : X * a.TT));
            }
            q_turn ^= 1u << X;
            q_some |= 1u << X;
          }
          if (!ok) break;
        }
        if (left > 1) {
          ++i;
          --left;
        } else {
          // the next is claimed when this one's last tile is about to be loaded: claimed as far ahead as the ring goes, items
          // stay with a CTA that is late with them (6001 tokens x 32 heads: 250 against 223 us, 9000 x 8: 180 against 129,
          // 16001 x 32: 1409 against 1393, 64 x 1000: 573 against 559; requests of a few tiles the same either way)
          if (some && !__all_sync(FULL, pt_wait(&bars.near[(t - 1) % PT_RING], (t - 1) / PT_RING & 1, &gone, p))) break;
          if (lane == 0) claim_block(&claim, &bars.claim);
          if (!__all_sync(FULL, pt_wait(&bars.claim, c & 1, &gone, p))) {
            mbar_wait(&bars.claim, c & 1, 1u << 16);   // (the answer is in flight)
            break;
          }
          take(claimed_block(&claim));
          ++c;
        }
      }
      // (no copy is in flight when the CTA ends, also where it gave up)
      for (int X = 0; X < 2; ++X)
        if (q_some >> X & 1) mbar_wait(&bars.q[X], (q_turn >> X & 1) ^ 1, 1u << 16);
    }
  }
  __syncthreads();
  tc_fence_after();
  if (wid == PT_W_MMA)
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
  return p.Hq / p.H <= PT_M && (at & 15) == 0 && stride_ok(p.q_tok, p.N) && stride_ok(p.q_head, p.Hq) &&
         stride_ok(p.k_tok, p.N) && stride_ok(p.k_head, p.H) && stride_ok(p.v_tok, p.N) && stride_ok(p.v_head, p.H) &&
         tensor_map_encode() != nullptr;
}

template <int DP, bool SPLIT>
static int launch_tc(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const PtArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};
  if (!smem_attr_once(prompt_tc_kernel<DP, SPLIT>, static_cast<int>(PtCfg<DP>::SMEM), attr_done)) return VBS_ECUDA;
  return launch_dependent(prompt_tc_kernel<DP, SPLIT>, dim3(static_cast<unsigned>(a.tiles * a.p.H - a.many * (a.batch - 1))), dim3(PT_NT),
                          PtCfg<DP>::SMEM, s, qm, km, vm, a);
}

int launch_prompt_tc(const PromptArgs& p, int num_sms, cudaStream_t s) {
  const int G = p.Hq / p.H, TT = PT_M / G;
  CUtensorMap qm, km, vm;
  if (!encode(&qm, p.q, p, p.Hq, p.q_tok, p.q_head, G, TT) || !encode(&km, p.k, p, p.H, p.k_tok, p.k_head, 1, PT_N) ||
      !encode(&vm, p.v, p, p.H, p.v_tok, p.v_head, 1, PT_N))
    return VBS_ECUDA;
  // Two row tiles an item, but one where head_dim leaves no room for two, or, its positions split, where the GPU has an SM
  // for each pair.  Split / not in us: 7000 tokens x 1 head x 128: 63 / 90; 4000 x 8: 43 / 65; 2000 x 4 heads over 1: 27 / 35;
  // 32 sentences up to 256 x 8 x 64: 20.5 / 22.5; and with more pairs than SMs, 2000 x 32 over 8: 47 / 39; 9000 x 8 over 1:
  // 143 / 125; 64 such sentences: 33 / 31 (K and V are loaded for each row tile, and each brings out two sums).
  const int64_t pairs = (static_cast<int64_t>(p.N) + 2 * TT - 1) / (2 * TT) * p.H;
  const bool split = p.D <= 128 && pairs <= num_sms;
  const int per = p.D > 128 || split ? TT : 2 * TT;
  const int64_t tiles = (static_cast<int64_t>(p.N) + per - 1) / per, items = tiles * p.H;
  if (items >= int64_t{1} << 31) return VBS_EINVAL;
  // the GPU answers some 15 claims a microsecond: many items are claimed several at a time, the last quarter one by one
  const int batch = static_cast<int>(std::max<int64_t>(1, items / (16 * num_sms)));
  const int many = batch > 1 ? static_cast<int>(items * 3 / 4 / batch) : 0;
  const PtArgs a{p, G, TT, per, static_cast<int>(tiles), batch, many,
                 (reinterpret_cast<uintptr_t>(p.o) & 15) == 0 && (p.o_tok | p.o_head) % 8 == 0};
  if (p.B >= PT_LOOK && launch_dependent(prompt_starts_kernel, dim3(std::min((p.B + 255) / 256, 8 * num_sms)), dim3(256), 0, s,
                                         p) != VBS_OK)
    return VBS_ECUDA;
  if (p.D <= 64) return split ? launch_tc<64, true>(qm, km, vm, a, s) : launch_tc<64, false>(qm, km, vm, a, s);
  if (p.D <= 128) return split ? launch_tc<128, true>(qm, km, vm, a, s) : launch_tc<128, false>(qm, km, vm, a, s);
  return launch_tc<256, false>(qm, km, vm, a, s);
}

}  // namespace vbs
