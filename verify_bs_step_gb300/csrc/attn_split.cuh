// Attention of a few query rows over many cached positions: the split kernel (sm_103a).
//
// A segment is one sentence's K/V head with up to 16 MT of the query rows that read it (the W beams x
// n_q tokens x q_heads / kv_heads rows that share it are numbered beam first).  Positions come in units
// of at most 16.  All segments' units stand in one line, sentence by sentence; every CTA of one
// resident wave takes an equal share of it, whatever the lengths (a segment counts SP_FIX units more than it
// has, at its start), and its four warps take every fourth unit.  A segment inside one share is written
// straight out; one that crosses shares leaves (m, l, o) partials, and a second, dependent launch joins them
// in order, so equal calls give equal bits.  (Joining in the CTA that arrives last was slower: a fence and an
// atomic a piece, and one CTA's loads in turn while the others are done.)  Short segments are not split at all.
//
// A warp holds 16 MT rows x head_dim of o in registers.  Units come through a ring of cp.async stages of
// its own (no barrier between warps), stored with a XOR of 16-byte chunks so that both reads below
// meet no bank twice:
//   scores   S = Q K^T by mma.m16n8k16: a lane takes 16 bytes of a position's row, and the order of dims
//            inside the contraction is whatever that gives (Q is laid out the same way);
//   values   O += P V by mma.m16n8k16: a lane takes 16 bytes of four positions, pairs of positions are put
//            side by side with byte permutes, and the order of the output dims is undone at the end.
// What bounds it is the K/V stream for one long row (250001 positions, 8 heads x 128 e4m3: 95 us with the plan and
// the join, 5.4 TB/s, 80 % of the measured copy), the segments' fixed cost (some 5 us of lookups, Q and sums
// each) for many short ones (64 sentences x 4 beams x 1064: 46 us, 39 of them this kernel at 4.1 TB/s), and latency at
// few warps where 32 rows share a K/V head (64 x 8 tokens x 4 heads over 1..4000 positions, int8: 97 us, 2.8 TB/s: 254
// registers leave two warps a scheduler; issue slots 43 % active, the tensor pipe 33 %, the first stall the fixed
// latency of an instruction).
// Measured and not kept: two units an iteration (fewer instructions, 8 warps instead of 12: 102 and 65 us), CTAs
// of one warp (91 us at 64 x 4 beams: four times the partials), a join in the CTA that arrives last (57).

#pragma once

#include <cfloat>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attn.h"
#include "codes.cuh"
#include "common.cuh"

namespace vbs {

constexpr int NW = 4;                    // warps a CTA
constexpr int SP_MIN = 4 * NW;           // units a CTA takes at least: every warp's ring once
// What a segment costs besides its units (Q, the first loads, the warps' sums), in units: a share with many short
// segments takes as long as one with a single long one (64 x 8 tokens over 1..4000 positions: 184 us with 8,
// 139 with 20, 117 with 48 before the lookups were overlapped; 98 with 24 since).
constexpr int SP_FIX = 24;

// What the kernel needs to know of the split.
struct SplitArgs {
  int B, W, H, D;
  int G;                          // query heads per K/V head
  int M;                          // query rows per K/V head: W * n_q * G
  int MC;                         // chunks of 16 MT of them
  float* part;                    // [grid][2][16 MT][DP + 2]: o, m, l of a segment's piece
  int2* pieces;                   // [B * H * MC]: the first and last CTA of a segment in pieces, (0, -1) of a whole one
  bool out8, q8;                  // outputs may be stored, queries loaded 8 bytes at a time
  bool whole;                     // a CTA a segment, none in pieces
};

__device__ __forceinline__ void cp_async16(u32 dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds16(u32 a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds8(u32 a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}

template <bool BF> __device__ __forceinline__ void mma16816(float (&c)[4], const uint4& a, u32 b0, u32 b1) {
  if (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ u32 pack_f16(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<u32*>(&h);
}
__device__ __forceinline__ u32 pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<u32*>(&h);
}

// What a unit's consumer needs of it.
struct __align__(16) UnitHead {
  int pos, n;                     // its first position, and how many it has
  u32 rows;                       // the beams that see it
  float ks;                       // K's scale
  float ve, vinv;                 // log2 of V's scale, and its reciprocal
  float pad[2];
};

// ---------------------------------------------------------------------------------------
// sources
// ---------------------------------------------------------------------------------------

// The 8-bit paged cache: a unit is up to 16 positions of one page of the plan's list.
template <int FMT> struct PagedSrc {
  static constexpr int EL = 1, FORMAT = FMT;
  static constexpr bool BF = false;
  Kv8Geom g;
  const int4* list;               // [B][cap] (page, first position, beams, positions)
  const int* n_pages;             // [B]
  const int* seen;                // [R]
  int cap, tpp;                   // list entries a sentence, units a page
  int64_t most() const { return static_cast<int64_t>(cap) * tpp; }
  struct Batch {                  // one unit per lane
    const char* k;                // its K rows; V's stand H runs further on
    UnitHead u;
  };
  __device__ int units(int b) const { return n_pages[b] * tpp; }
  __device__ int limit(int b, int w, int i, int W, int n_q) const { return seen[b * W + w] - n_q + 1 + i; }
  __device__ void fetch(Batch& t, int b, int h, int u, bool valid) const {
    t.k = g.pool;
    t.u = UnitHead{0, 0, 0u, 0.f, 0.f, 1.f, {0.f, 0.f}};
    if (!valid) return;
    const int e = u / tpp, off = (u - e * tpp) * 16;
    const int4 x = list[static_cast<int64_t>(b) * cap + e];
    t.u.pos = x.y + off;
    t.u.n = max(0, min(16, x.w - off));
    t.u.rows = static_cast<u32>(x.z);
    if (t.u.n > 0) {
      const int64_t run = g.run(x.x, 0, h);
      t.k = g.pool + (run * g.block + off) * g.D;
      t.u.ks = g.scales[run];
      // held to the scales' range: a page no append has written (scale 0) counts as zeros
      const int ve = max(KV8_E_LO, min(KV8_E_HI, (__float_as_int(g.scales[run + g.H]) >> 23) - 127));
      t.u.ve = static_cast<float>(ve);
      t.u.vinv = __int_as_float((127 - ve) << 23);
    }
  }
  // lane `k`'s unit: the loads of its K and V rows into a stage, and its head
  template <class L>
  __device__ __forceinline__ void issue(const Batch& t, int k, int lane, int, int, UnitHead* head,
                                        const L& load) const {
    const u64 at = shfl64(reinterpret_cast<u64>(t.k), k);
    const int n = __shfl_sync(FULL, t.u.n, k);
    if (lane == k) *head = t.u;
    const char* kp = reinterpret_cast<const char*>(at);
    load(kp, kp + static_cast<int64_t>(g.H) * g.block * g.D, g.D, g.D, n);
  }
};

// An encoder's states: a unit is up to 16 positions of a sentence.
struct EncSrc {
  static constexpr int EL = 2, FORMAT = 0;
  static constexpr bool BF = true;
  EncKV e;
  struct Batch { int u; };
  int64_t most() const { return (static_cast<int64_t>(e.S) + 15) / 16; }
  __device__ int len(int b) const {
    const int n = e.len[b];
    if (n >= 0 && n <= e.S) return n;
    set_status(e.status, VBS_EINVAL);
    return n < 0 ? 0 : e.S;
  }
  __device__ int units(int b) const { return max(1, static_cast<int>((static_cast<u32>(len(b)) + 15) >> 4)); }
  __device__ int limit(int b, int, int, int, int) const { return len(b); }
  // (a lane without a unit stands past every end: no positions)
  __device__ void fetch(Batch& t, int, int, int u, bool valid) const { t.u = valid ? u : 1 << 26; }
  template <class L>
  __device__ __forceinline__ void issue(const Batch& t, int k, int lane, int b, int h, UnitHead* head,
                                        const L& load) const {
    const int pos = __shfl_sync(FULL, t.u, k) * 16;
    const int n = max(0, min(16, len(b) - pos));
    if (lane == 0) *head = UnitHead{pos, n, 0xffffu, 1.f, 0.f, 1.f, {0.f, 0.f}};
    load(reinterpret_cast<const char*>(e.k + b * e.k_sent + h * e.k_head + (n > 0 ? pos * e.k_pos : 0)),
         reinterpret_cast<const char*>(e.v + b * e.v_sent + h * e.v_head + (n > 0 ? pos * e.v_pos : 0)),
         e.k_pos * 2, e.v_pos * 2, n);
  }
};

// ---------------------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------------------

template <int EL, int DP, int MT> struct SplitCfg {
  static constexpr int CHK = 16 / EL;                       // dims in 16 bytes
  static constexpr int KS = DP / 16;                        // contraction steps of the scores
  static constexpr int NT = DP / 8;                         // output tiles of 8 dims
  static constexpr int VCH = NT < CHK ? NT : CHK;           // dims of a position that a lane reads at once
  static constexpr int STAGE = 2 * 16 * DP * EL;            // bytes of K and V of one unit
  // one tile of rows over 8-bit codes of up to 64 dims: little to hold, so that a shorter ring (4 stages, not 8) and a
  // fourth CTA an SM pay (1024 sentences x 8 heads x 64..1024 positions: 94 to 76 us .. 195 to 183; 64 x 512: 14.9 to 13.3;
  // 16 sentences, which do not fill the GPU: 1..5 % slower)
  static constexpr bool SMALL = EL == 1 && DP == 64 && MT == 1;
  static constexpr int NS = SMALL ? 4 : STAGE <= 2048 ? 8 : STAGE <= 4096 ? 4 : (STAGE <= 8192 ? 3 : 2);
  static constexpr int O_LD = DP + 4;                       // floats of an o row in shared memory
  static constexpr int RING = NS * STAGE > MT * 16 * O_LD * 4 ? NS * STAGE : MT * 16 * O_LD * 4;
  static constexpr int QBYTES = MT * KS * 512;              // Q in fragment order
  static constexpr int PART = MT * 16 * (DP + 2);           // floats of a partial
  static constexpr size_t SMEM = NW * RING + QBYTES;
  // resident CTAs a SM, by shared memory and by o's registers (MT * DP / 2 of a thread's)
  static constexpr int CTAS = SMEM > 113 * 1024 ? 1 : (SMEM > 75 * 1024 || MT * DP > 128 ? 2 : SMALL ? 4 : 3);
};

// The order of output dims: column n of output tile j.
template <int VCH> __device__ __forceinline__ int out_dim(int n, int j) {
  return (j / VCH) * (8 * VCH) + n * VCH + j % VCH;
}

// The XOR of a position's 16-byte chunks: rows of 8 (or 16) chunks, or two positions to a line of 8.
__device__ __forceinline__ int k_swz(int tok, int nc) { return (nc & 7) == 0 ? (tok & 1) << 2 : 0; }
__device__ __forceinline__ int v_swz(int tok, int nc) { return (nc & 3) == 0 ? ((tok >> 1) & 3) << 1 : 0; }

// The factor on a row's sums: 0 without a position seen (no reference); infinite, for NaN, where all it sees score -inf.
__device__ __forceinline__ float row_norm(float sum, float top) { return top == -INFINITY ? 0.f : 1.f / sum; }

// Four dims of an output row.
__device__ __forceinline__ void store_out(uint16_t* out, const SplitArgs& sa, const float4& v) {
  const uint2 q = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  if (sa.out8) {
    *reinterpret_cast<uint2*>(out) = q;
  } else {
    out[0] = static_cast<uint16_t>(q.x);
    out[1] = static_cast<uint16_t>(q.x >> 16);
    out[2] = static_cast<uint16_t>(q.y);
    out[3] = static_cast<uint16_t>(q.y >> 16);
  }
}

// EXACT: head_dim is DP; ALIGNED: K and V rows may be copied 16 bytes at a time.
template <class Src, int DP, int MT, bool EXACT, bool ALIGNED>
__global__ void __launch_bounds__(32 * NW, (SplitCfg<Src::EL, DP, MT>::CTAS))
attn_split_kernel(const Src src, const QO io, const SplitArgs sa) {
  using C = SplitCfg<Src::EL, DP, MT>;
  constexpr int NT = 32 * NW;
  constexpr int EL = Src::EL, ROWS = 16 * MT;
  constexpr float GROW = Src::BF ? 8.f : 3.f;
  extern __shared__ __align__(128) unsigned char sp_smem[];
  __shared__ UnitHead heads[NW][C::NS];
  __shared__ float row_f[ROWS];                             // a row's factor on its dot products
  __shared__ int64_t row_q[ROWS], row_o[ROWS];              // its elements in q (-1: none) and out
  __shared__ int row_lim[ROWS], row_beam[ROWS];
  __shared__ float wm[NW][ROWS], wl[NW][ROWS];
  __shared__ int64_t s_sum[NW];
  __shared__ int s_b, s_n;
  __shared__ int64_t s_pos;

  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, c4 = lane & 3;
  const int D = EXACT ? DP : sa.D;
  const int nc = D / C::CHK;                                // 16-byte chunks of a row
  unsigned char* ring = sp_smem + wid * C::RING;
  const u32 ring_a = smem_u32(ring);
  uint16_t* qf = reinterpret_cast<uint16_t*>(sp_smem + NW * C::RING);
  const u32 qf_a = smem_u32(qf);
  const int HM = sa.H * sa.MC;

  // a dependent launch (of the plan, or of what made q): set up before, reads nothing before its end
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's share of the line ----
  int b = 0;
  int n = 1;                                                // sentence b's units
  int64_t at = 0, end, per = 1;                             // position within sentence b's units (all heads)
  if (sa.whole) {
    b = blockIdx.x / HM;
    n = src.units(b);
    end = n + SP_FIX;
    at = (blockIdx.x - b * HM) * end;
  } else {
    const int k = (sa.B + NT - 1) / NT;               // a thread's sentences: [tid * k, tid * k + k)
    int64_t mine = 0;
    int own = 0;                                            // the last one's units
    for (int i = tid * k; i < min(sa.B, tid * k + k); ++i) {
      own = src.units(i);
      mine += own + SP_FIX;
    }
    int64_t inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(FULL, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) s_sum[wid] = inc;
    __syncthreads();
    int64_t before = inc - mine, all = 0;
    for (int w = 0; w < NW; ++w) {
      if (w < wid) before += s_sum[w];
      all += s_sum[w];
    }
    const int64_t total = all * HM;
    per = max(static_cast<int64_t>(SP_MIN + SP_FIX), (total + gridDim.x - 1) / gridDim.x);
    const int64_t from = per * blockIdx.x;
    end = min(total, from + per);
    if (from >= total) return;
    if (from >= before * HM && from < (before + mine) * HM) {
      int64_t p = from - before * HM;
      int i = tid * k;
      if (k > 1)
        for (; i < sa.B - 1; ++i) {
          own = src.units(i);
          const int64_t n = static_cast<int64_t>(own + SP_FIX) * HM;
          if (p < n) break;
          p -= n;
        }
      s_b = i;
      s_n = k > 1 ? src.units(i) : own;
      s_pos = p;
    }
    __syncthreads();
    b = s_b;
    n = s_n;
    at = s_pos;
    end -= from;                                            // units left
  }
  int64_t line0 = per * blockIdx.x - at;                    // the line's position of sentence b's first unit

  while (end > 0 && b < sa.B) {
    const int nf = n + SP_FIX;
    const int hm = static_cast<int>(at / nf), h = hm / sa.MC, mc = hm - h * sa.MC;
    const int f0 = static_cast<int>(at - static_cast<int64_t>(hm) * nf);   // on the line; u0, u1: units
    const int f1 = static_cast<int>(min(static_cast<int64_t>(nf), f0 + end));
    const int u0 = max(0, f0 - SP_FIX), u1 = f1 - SP_FIX;
    const int n_next = b + 1 < sa.B ? src.units(b + 1) : 1;  // on its way while this segment is worked on
    auto advance = [&] {
      const int done = f1 - f0;
      end -= done;
      at += done;
      if (at == static_cast<int64_t>(nf) * HM) {
        line0 += at;
        at = 0;
        ++b;
        n = n_next;
      }
    };
    if (u1 <= u0) {                                         // the segment's units are all in the next share
      advance();
      continue;
    }
    const int rho0 = mc * ROWS;
    const int rows = min(ROWS, sa.M - rho0);

    const int mine = u1 - u0 > wid ? (u1 - u0 - wid + NW - 1) / NW : 0;
    typename Src::Batch batch;
    auto issue = [&](int k) {                               // the warp's k-th unit into its stage
      if (k < mine) {
        if ((k & 31) == 0) src.fetch(batch, b, h, u0 + wid + (k + lane) * NW, k + lane < mine);
        const int st = k % C::NS;
        const u32 base = ring_a + st * C::STAGE;
        src.issue(batch, k & 31, lane, b, h, &heads[wid][st],
                  [&](const char* kp, const char* vp, int64_t kld, int64_t vld, int cnt) {
          if (EXACT && EL == 1 && cnt == 16) {              // a whole unit of contiguous rows: constant offsets
            const char *ks = kp + lane * 16, *vs = vp + lane * 16;
#pragma unroll
            for (int i = 0; i < DP / C::CHK / 2; ++i) {
              const int L = i * 32 + lane, tok = L / nc;
              cp_async16(base + (L ^ k_swz(tok, nc)) * 16, ks + i * 512, true);
              cp_async16(base + C::STAGE / 2 + (L ^ v_swz(tok, nc)) * 16, vs + i * 512, true);
            }
            return;
          }
#pragma unroll
          for (int i = 0; i < (DP / C::CHK + 1) / 2; ++i) {
            const int L = i * 32 + lane;
            const int tok = L / nc, ch = L - tok * nc;
            if (EXACT || tok < 16) {
              const bool ok = tok < cnt;
              const char* ks = kp + (ok ? tok * kld + ch * 16 : 0);
              const char* vs = vp + (ok ? tok * vld + ch * 16 : 0);
              const u32 kd = base + (L ^ k_swz(tok, nc)) * 16;
              const u32 vd = base + C::STAGE / 2 + (L ^ v_swz(tok, nc)) * 16;
              if (ALIGNED) {
                cp_async16(kd, ks, ok);
                cp_async16(vd, vs, ok);
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const uint16_t x = ok ? reinterpret_cast<const uint16_t*>(ks)[e] : uint16_t{0};
                  const uint16_t y = ok ? reinterpret_cast<const uint16_t*>(vs)[e] : uint16_t{0};
                  asm volatile("st.shared.u16 [%0], %1;" ::"r"(kd + e * 2), "h"(x) : "memory");
                  asm volatile("st.shared.u16 [%0], %1;" ::"r"(vd + e * 2), "h"(y) : "memory");
                }
              }
            }
          }
        });
      }
      cp_commit();
    };
    // ---- where the segment's rows stand and what they see, divided out once ----
    if (tid < ROWS) {
      const int rho = rho0 + tid, gq = rho % sa.G, iw = rho / sa.G, i = iw % io.n_q, w = iw / io.n_q;
      const bool live = tid < rows;
      const int64_t row = static_cast<int64_t>(b) * sa.W + w, head = h * sa.G + gq;
      row_q[tid] = live ? row * io.q_row + i * io.q_tok + head * io.q_head : -1;
      row_o[tid] = row * io.o_row + i * io.o_tok + head * io.o_head;
      row_lim[tid] = live ? src.limit(b, w, i, sa.W, io.n_q) : 1 << 30;
      row_beam[tid] = live ? w : 31;                        // padding rows see everything, and are not written
    }
    __syncthreads();

    // ---- Q in fragment order: a warp a row, four dims a lane, the loads of four rows at once; the first four
    // rows are on their way while the first units' addresses are looked up ----
    constexpr int QV = (DP + 127) / 128;
    uint2 x[4][QV];
    auto load_q = [&](int r0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t off = row_q[r0 + k * NW + wid];
#pragma unroll
        for (int v = 0; v < QV; ++v) {
          const int d = v * 128 + lane * 4;
          x[k][v] = make_uint2(0, 0);
          if (off >= 0 && d < D) {
            const uint16_t* q = io.q + off + d;
            if (sa.q8) x[k][v] = *reinterpret_cast<const uint2*>(q);
            else x[k][v] = make_uint2(q[0] | static_cast<u32>(q[1]) << 16, q[2] | static_cast<u32>(q[3]) << 16);
          }
        }
      }
    };
    load_q(0);
#pragma unroll
    for (int k = 0; k < C::NS - 1; ++k) issue(k);

#pragma unroll
    for (int r0 = 0; r0 < ROWS; r0 += 4 * NW) {
      if (r0 > 0) load_q(r0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + k * NW + wid;
        float up = 1.f;                                     // the row's power of two: its largest element to [1, 2)
        if (!Src::BF) {
          u32 top = 0;
#pragma unroll
          for (int v = 0; v < QV; ++v)
            top = max(max(top, max(x[k][v].x & 0x7fffu, x[k][v].x >> 16 & 0x7fffu)),
                      max(x[k][v].y & 0x7fffu, x[k][v].y >> 16 & 0x7fffu));
#pragma unroll
          for (int e = 16; e > 0; e >>= 1) top = max(top, __shfl_xor_sync(FULL, top, e));
          const int ex = static_cast<int>(top >> 7);        // biased exponent
          up = __int_as_float(max(1, min(254, 254 - ex)) << 23);
        }
        if (lane == 0) row_f[r] = io.scale * LOG2E_F / up;
#pragma unroll
        for (int v = 0; v < QV; ++v) {
          const int d = v * 128 + lane * 4, ch = d / C::CHK;
          if (d >= DP) continue;
          const int ks = (ch >> 2) * (C::CHK / 4) + d % C::CHK / 4;
          const u32 to = (((r >> 4) * C::KS + ks) * 32 + (r & 7) * 4 + (ch & 3)) * 4 + ((r >> 3) & 1);
          u32* qw = reinterpret_cast<u32*>(qf);
          const uint2 y = x[k][v];
          qw[to] = Src::BF ? y.x : pack_f16(bf16_lo(y.x) * up, bf16_hi(y.x) * up);
          qw[to + 2] = Src::BF ? y.y : pack_f16(bf16_lo(y.y) * up, bf16_hi(y.y) * up);
        }
      }
    }
    __syncthreads();

    float o[MT][C::NT][4], m[MT][2], l[MT][2], f[MT][2];
    int lim[MT][2], beam[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = mt * 16 + x * 8 + g;
        m[mt][x] = -INFINITY;
        l[mt][x] = 0.f;
        f[mt][x] = row_f[r];
        lim[mt][x] = row_lim[r];
        beam[mt][x] = row_beam[r];
#pragma unroll
        for (int j = 0; j < C::NT; ++j) o[mt][j][x * 2] = o[mt][j][x * 2 + 1] = 0.f;
      }

    for (int k = 0; k < mine; ++k) {
      cp_wait<C::NS - 2>();
      __syncwarp();
      issue(k + C::NS - 1);
      const int st = k % C::NS;
      const u32 ka = ring_a + st * C::STAGE, va = ka + C::STAGE / 2;
      const UnitHead u = heads[wid][st];

      // ---- scores of 16 positions: two tiles of 8 ----
      float s[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int t = 0; t < 2; ++t) s[mt][t][0] = s[mt][t][1] = s[mt][t][2] = s[mt][t][3] = 0.f;
#pragma unroll
      for (int grp = 0; grp < DP / C::CHK / 4; ++grp) {
        uint4 kw[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int tok = t * 8 + g, ch = grp * 4 + c4;
          kw[t] = EXACT || ch < nc ? lds16(ka + ((tok * nc + ch) ^ k_swz(tok, nc)) * 16) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int q4 = 0; q4 < C::CHK / 4; ++q4) {
          const int ks = grp * (C::CHK / 4) + q4;
          u32 b0[2], b1[2];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const u32 words[4] = {kw[t].x, kw[t].y, kw[t].z, kw[t].w};
            if (EL == 1) {
              codes4<Src::FORMAT>(words[q4], b0[t], b1[t]);
            } else {
              b0[t] = words[(q4 * 2) & 3];
              b1[t] = words[(q4 * 2 + 1) & 3];
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 a = lds16(qf_a + ((mt * C::KS + ks) * 32 + lane) * 16);
            mma16816<Src::BF>(s[mt][0], a, b0[0], b1[0]);
            mma16816<Src::BF>(s[mt][1], a, b0[1], b1[1]);
          }
        }
      }

      // ---- softmax: weights relative to the running maximum of s + log2(V's scale) ----
      uint4 p[MT], p2[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        int left[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) left[x] = (u.rows >> beam[mt][x]) & 1u || beam[mt][x] == 31 ? min(lim[mt][x] - u.pos, u.n) : 0;
        const bool full = __all_sync(FULL, left[0] >= 16 && left[1] >= 16);
        float mx[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float fk = f[mt][x] * u.ks;
          mx[x] = -INFINITY;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float& z = s[mt][t][x * 2 + y];
              z = fmaf(z, fk, u.ve);
              if (!full && t * 8 + c4 * 2 + y >= left[x]) z = -INFINITY;
              mx[x] = fmaxf(mx[x], z);
            }
          mx[x] = fmaxf(mx[x], __shfl_xor_sync(FULL, mx[x], 1));
          mx[x] = fmaxf(mx[x], __shfl_xor_sync(FULL, mx[x], 2));
        }
        // the reference moves once a maximum has outgrown it by 2^GROW
        if (__any_sync(FULL, mx[0] > m[mt][0] + GROW || mx[1] > m[mt][1] + GROW)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mx[x] = fmaxf(mx[x], m[mt][x]);
            const float corr = m[mt][x] == -INFINITY ? 0.f : ex2(m[mt][x] - mx[x]);
            l[mt][x] *= corr;
#pragma unroll
            for (int j = 0; j < C::NT; ++j) {
              o[mt][j][x * 2] *= corr;
              o[mt][j][x * 2 + 1] *= corr;
            }
            m[mt][x] = mx[x];
          }
        }
        float w[2][4];                                      // [row][position]
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // fp16 weights reach up to 2^15, so that small ones keep their bits
          const float ref = (m[mt][x] == -INFINITY ? 0.f : m[mt][x]) - (Src::BF ? 0.f : 15.f - GROW);
          float sum = 0.f;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              w[x][t * 2 + y] = ex2(s[mt][t][x * 2 + y] - ref);
              sum += w[x][t * 2 + y];
            }
          l[mt][x] = Src::BF ? l[mt][x] + sum : fmaf(sum, u.vinv, l[mt][x]);
        }
        if (Src::BF) {
          // two bf16 parts of each weight: the products carry 16 bits of it
          float r[2][4];
          p[mt] = make_uint4(pack_bf16(w[0][0], w[0][1]), pack_bf16(w[1][0], w[1][1]), pack_bf16(w[0][2], w[0][3]),
                             pack_bf16(w[1][2], w[1][3]));
          const u32 hi[2][2] = {{p[mt].x, p[mt].z}, {p[mt].y, p[mt].w}};
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              r[x][t * 2] = w[x][t * 2] - bf16_lo(hi[x][t]);
              r[x][t * 2 + 1] = w[x][t * 2 + 1] - bf16_hi(hi[x][t]);
            }
          p2[mt] = make_uint4(pack_bf16(r[0][0], r[0][1]), pack_bf16(r[1][0], r[1][1]), pack_bf16(r[0][2], r[0][3]),
                              pack_bf16(r[1][2], r[1][3]));
        } else {
          p[mt] = make_uint4(pack_f16(w[0][0], w[0][1]), pack_f16(w[1][0], w[1][1]), pack_f16(w[0][2], w[0][3]),
                             pack_f16(w[1][2], w[1][3]));
        }
      }

      // ---- o += P V ----
      const int toks[4] = {c4 * 2, c4 * 2 + 1, c4 * 2 + 8, c4 * 2 + 9};
#pragma unroll
      for (int vc = 0; vc < C::NT / C::VCH; ++vc) {
        u32 vw[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int dim = out_dim<C::VCH>(g, vc * C::VCH), ch = dim / C::CHK;
          const u32 a = va + ((toks[t] * nc + ch) ^ v_swz(toks[t], nc)) * 16;
          if (EXACT || dim < D) {
            if (C::VCH * EL == 16) {
              const uint4 q = lds16(a);
              vw[t][0] = q.x; vw[t][1] = q.y; vw[t][2] = q.z; vw[t][3] = q.w;
            } else {
              const uint2 q = lds8(a + (dim % C::CHK) * EL);
              vw[t][0] = q.x; vw[t][1] = q.y; vw[t][2] = vw[t][3] = 0;
            }
          } else {
            vw[t][0] = vw[t][1] = vw[t][2] = vw[t][3] = 0;
          }
        }
#pragma unroll
        for (int wd = 0; wd < C::VCH * EL / 4; ++wd) {
          if (EL == 1) {
            u32 b0[4], b1[4];                               // four dims, positions 0,1 and 2,3 of the lane
            codes4<Src::FORMAT>(__byte_perm(vw[0][wd], vw[1][wd], 0x5140), b0[0], b0[1]);
            codes4<Src::FORMAT>(__byte_perm(vw[0][wd], vw[1][wd], 0x7362), b0[2], b0[3]);
            codes4<Src::FORMAT>(__byte_perm(vw[2][wd], vw[3][wd], 0x5140), b1[0], b1[1]);
            codes4<Src::FORMAT>(__byte_perm(vw[2][wd], vw[3][wd], 0x7362), b1[2], b1[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma16816<false>(o[mt][vc * C::VCH + wd * 4 + i], p[mt], b0[i], b1[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const u32 b0 = __byte_perm(vw[0][wd], vw[1][wd], i ? 0x7632 : 0x5410);
              const u32 b1 = __byte_perm(vw[2][wd], vw[3][wd], i ? 0x7632 : 0x5410);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma16816<true>(o[mt][vc * C::VCH + wd * 2 + i], p[mt], b0, b1);
                mma16816<true>(o[mt][vc * C::VCH + wd * 2 + i], p2[mt], b0, b1);
              }
            }
          }
        }
      }
    }

    // ---- join the warps ----
    cp_wait<0>();
    __syncwarp();                                           // the ring is free: o goes there
    float* mo = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = mt * 16 + x * 8 + g;
        float ls = l[mt][x];
        ls += __shfl_xor_sync(FULL, ls, 1);
        ls += __shfl_xor_sync(FULL, ls, 2);
        if (c4 == 0) {
          wm[wid][r] = mine ? m[mt][x] : -INFINITY;
          wl[wid][r] = mine ? ls : 0.f;
        }
#pragma unroll
        for (int j = 0; j < C::NT; j += 4)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            *reinterpret_cast<float4*>(mo + r * C::O_LD + out_dim<C::VCH>(c4 * 2 + y, j)) =
                make_float4(o[mt][j][x * 2 + y], o[mt][j + 1][x * 2 + y], o[mt][j + 2][x * 2 + y], o[mt][j + 3][x * 2 + y]);
      }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == n;
    const int64_t line = line0 + static_cast<int64_t>(hm) * nf;  // the segment's place in the line
    float* part = sa.part + (static_cast<int64_t>(blockIdx.x) * 2 + (u0 > 0 ? 0 : 1)) * C::PART;
    if (tid < ROWS) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = fmaxf(top, wm[w][tid]);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float x = wm[w][tid] == -INFINITY ? 0.f : ex2(wm[w][tid] - top);
        sum += wl[w][tid] * x;                              // (a NaN stays one)
        wm[w][tid] = x;
      }
      // a row that sees positions, all of which score -inf, is told from one that sees none (softmax is 0 / 0 there)
      if (top == -INFINITY && row_lim[tid] > 0) top = -FLT_MAX;
      if (whole) {
        const float inv = row_norm(sum, top);
#pragma unroll
        for (int w = 0; w < NW; ++w) wm[w][tid] *= inv;
      } else {
        part[ROWS * DP + tid] = top;
        part[ROWS * DP + ROWS + tid] = sum;
      }
    }
    __syncthreads();
    for (int idx = tid; idx < rows * (DP / 4); idx += NT) {
      const int r = idx / (DP / 4), d = idx % (DP / 4) * 4;
      if (!EXACT && d >= D) continue;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float x = wm[w][r];
        if (x != 0.f) {
          const float4 v = *reinterpret_cast<const float4*>(sp_smem + w * C::RING + (r * C::O_LD + d) * 4);
          a.x += v.x * x; a.y += v.y * x; a.z += v.z * x; a.w += v.w * x;
        }
      }
      if (whole) store_out(io.o + row_o[r] + d, sa, a);
      else *reinterpret_cast<float4*>(part + r * DP + d) = a;
    }

    // the CTA with a segment's first unit says where its pieces are
    if (u0 == 0 && tid == 0 && !sa.whole)
      sa.pieces[static_cast<int64_t>(b) * HM + hm] =
          whole ? make_int2(0, -1) : make_int2(static_cast<int>((line + SP_FIX) / per), static_cast<int>((line + nf - 1) / per));
    __syncthreads();                                        // the ring and the row statistics are free again
    advance();
  }
}

// ---------------------------------------------------------------------------------------
// the join of segments in pieces
// ---------------------------------------------------------------------------------------

constexpr int JN_WARPS = 4, JN_FEW = 4;

// CTA (segment, c): rows 4 c .. 4 c + 3 of its segment, a warp each; where the pieces are many, all warps take
// a row after the other and share its pieces.  A dependent launch: it is set up while the split kernel runs.
template <int DP, int ROWS>
__global__ void __launch_bounds__(32 * JN_WARPS) attn_join_kernel(const QO io, const SplitArgs sa) {
  constexpr int PART = ROWS * (DP + 2), V = DP / 128 > 0 ? DP / 128 : 1;   // float4s of a row that a lane holds
  __shared__ float4 so[JN_WARPS][DP / 4];
  __shared__ float sm[JN_WARPS], sl[JN_WARPS];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t seg = blockIdx.x;
  const int2 at = __ldcg(sa.pieces + seg);
  if (at.y < at.x) return;
  const int mc = static_cast<int>(seg % sa.MC);
  const int64_t bh = seg / sa.MC;
  const int h = static_cast<int>(bh % sa.H), b = static_cast<int>(bh / sa.H);
  const int rows = min(ROWS, sa.M - mc * ROWS), np = at.y - at.x + 1;
  auto piece = [&](int c) { return sa.part + (static_cast<int64_t>(at.x + c) * 2 + (c == 0 ? 1 : 0)) * PART; };
  // one row's pieces c0, c0 + step, ... : their reference, sum and weighted sum
  auto gather = [&](int r, int c0, int step, float& top, float& sum, float4 (&a)[V]) {
    top = -INFINITY;
    for (int c = c0 + step * lane; c < np; c += step * 32) top = fmaxf(top, __ldcg(piece(c) + ROWS * DP + r));
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, k));
    sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 16
    for (int c = c0; c < np; c += step) {
      const float* pp = piece(c);
      const float mm = __ldcg(pp + ROWS * DP + r), ll = __ldcg(pp + ROWS * DP + ROWS + r);
      const float x = mm == -INFINITY ? 0.f : ex2(mm - top);
      sum += ll * x;                                        // (a NaN stays one)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (lane * 4 + v * 128 < DP) {
          const float4 q = __ldcg(reinterpret_cast<const float4*>(pp + r * DP + v * 128) + lane);
          a[v].x += q.x * x; a[v].y += q.y * x; a[v].z += q.z * x; a[v].w += q.w * x;
        }
    }
  };
  auto out_row = [&](int r) {
    const int rho = mc * ROWS + r, gq = rho % sa.G, iw = rho / sa.G;
    return io.o + (static_cast<int64_t>(b) * sa.W + iw / io.n_q) * io.o_row + iw % io.n_q * io.o_tok +
           static_cast<int64_t>(h * sa.G + gq) * io.o_head;
  };
  float4 a[V];
  float top, sum;
  if (np <= 64 * JN_WARPS) {
    const int r = blockIdx.y * JN_WARPS + wid;
    if (r >= rows) return;
    if (np <= JN_FEW) {                                     // few pieces: all loads at once
      float mm[JN_FEW], ll[JN_FEW];
      float4 q[JN_FEW][V];
#pragma unroll
      for (int c = 0; c < JN_FEW; ++c) {
        const float* pp = piece(min(c, np - 1));
        mm[c] = c < np ? __ldcg(pp + ROWS * DP + r) : -INFINITY;
        ll[c] = c < np ? __ldcg(pp + ROWS * DP + ROWS + r) : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
          q[c][v] = lane * 4 + v * 128 < DP ? __ldcg(reinterpret_cast<const float4*>(pp + r * DP + v * 128) + lane)
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      top = mm[0];
#pragma unroll
      for (int c = 1; c < JN_FEW; ++c) top = fmaxf(top, mm[c]);
      sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) a[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < JN_FEW; ++c) {
        const float x = mm[c] == -INFINITY ? 0.f : ex2(mm[c] - top);
        sum += ll[c] * x;                                   // (a NaN stays one)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          a[v].x += q[c][v].x * x; a[v].y += q[c][v].y * x; a[v].z += q[c][v].z * x; a[v].w += q[c][v].w * x;
        }
      }
    } else {
      gather(r, 0, 1, top, sum, a);
    }
    const float inv = row_norm(sum, top);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int d = lane * 4 + v * 128;
      if (d < sa.D) store_out(out_row(r) + d, sa, make_float4(a[v].x * inv, a[v].y * inv, a[v].z * inv, a[v].w * inv));
    }
    return;
  }
  for (int r = blockIdx.y * JN_WARPS; r < min(rows, (static_cast<int>(blockIdx.y) + 1) * JN_WARPS); ++r) {
    gather(r, wid, JN_WARPS, top, sum, a);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane * 4 + v * 128 < DP) so[wid][lane + v * 32] = a[v];
    if (lane == 0) {
      sm[wid] = top;
      sl[wid] = sum;
    }
    __syncthreads();
    float all = sm[0];
#pragma unroll
    for (int w = 1; w < JN_WARPS; ++w) all = fmaxf(all, sm[w]);
    float total = 0.f, f[JN_WARPS];
#pragma unroll
    for (int w = 0; w < JN_WARPS; ++w) {
      f[w] = sm[w] == -INFINITY ? 0.f : ex2(sm[w] - all);
      total += sl[w] * f[w];
    }
    const float inv = row_norm(total, all);
    for (int d = threadIdx.x * 4; d < sa.D; d += 32 * JN_WARPS * 4) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < JN_WARPS; ++w) {
        const float4 q = so[w][d / 4];
        const float x = f[w] * inv;
        o.x += q.x * x; o.y += q.y * x; o.z += q.z * x; o.w += q.w * x;
      }
      store_out(out_row(r) + d, sa, o);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------------------

// A launch that may be set up while its predecessor in the stream finishes; the kernel waits for it
// (griddepcontrol.wait) before its first access to memory.
template <typename... KArgs, typename... Args>
int launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...) == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

// Rows of a segment: two mma tiles where more than 16 rows share a K/V head (K/V are unpacked once for
// both); one at head_dim > 128, whose o does not fit the registers twice.
inline int split_mt(int M, int D) { return M > 16 && D <= 128 ? 2 : 1; }
inline int split_chunks(int M, int D) { return (M + 16 * split_mt(M, D) - 1) / (16 * split_mt(M, D)); }
inline int split_dp(int D) { return D <= 64 ? 64 : (D <= 128 ? 128 : 256); }
// floats of the partials of any grid: two pieces a CTA, up to 4 CTAs an SM of up to 32 rows
inline int64_t split_part_floats(int D, int num_sms) {
  return static_cast<int64_t>(num_sms) * 4 * 2 * 32 * (split_dp(D) + 2);
}

template <class Src, int DP, int MT, bool EXACT, bool ALIGNED>
int launch_split_as(const Src& src, const QO& io, const SplitArgs& sa, int num_sms, cudaStream_t s) {
  using C = SplitCfg<Src::EL, DP, MT>;
  static_assert(C::CTAS * MT * 16 <= 4 * 32, "split_part_floats");
  static std::atomic<unsigned long long> attr_done{0};
  auto* kernel = attn_split_kernel<Src, DP, MT, EXACT, ALIGNED>;
  if (!smem_attr_once(kernel, static_cast<int>(C::SMEM), attr_done)) return VBS_ECUDA;
  const int64_t segments = static_cast<int64_t>(sa.B) * sa.H * sa.MC;
  if (src.most() <= SP_WHOLE && segments < (int64_t{1} << 31)) {
    SplitArgs one = sa;
    one.whole = true;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(segments)), dim3(32 * NW), C::SMEM, s, src, io, one);
  }
  if (launch_dependent(kernel, dim3(num_sms * C::CTAS), dim3(32 * NW), C::SMEM, s, src, io, sa) != VBS_OK) return VBS_ECUDA;
  const dim3 grid(static_cast<unsigned>(segments), (std::min(sa.M, 16 * MT) + JN_WARPS - 1) / JN_WARPS);
  return launch_dependent(attn_join_kernel<DP, 16 * MT>, grid, dim3(32 * JN_WARPS), 0, s, io, sa);
}

template <class Src, int DP, int MT, bool ALIGNED>
int launch_split_dp(const Src& src, const QO& io, const SplitArgs& sa, int num_sms, cudaStream_t s) {
  if constexpr (ALIGNED) {
    if (sa.D == DP) return launch_split_as<Src, DP, MT, true, true>(src, io, sa, num_sms, s);
  }
  return launch_split_as<Src, DP, MT, false, ALIGNED>(src, io, sa, num_sms, s);
}

template <class Src, bool ALIGNED>
int launch_split(const Src& src, const QO& io, const SplitArgs& sa, int num_sms, cudaStream_t s) {
  const int mt = split_mt(sa.M, sa.D);
  if (sa.D <= 64)
    return mt == 2 ? launch_split_dp<Src, 64, 2, ALIGNED>(src, io, sa, num_sms, s)
                   : launch_split_dp<Src, 64, 1, ALIGNED>(src, io, sa, num_sms, s);
  if (sa.D <= 128)
    return mt == 2 ? launch_split_dp<Src, 128, 2, ALIGNED>(src, io, sa, num_sms, s)
                   : launch_split_dp<Src, 128, 1, ALIGNED>(src, io, sa, num_sms, s);
  return launch_split_dp<Src, 256, 1, ALIGNED>(src, io, sa, num_sms, s);
}

inline SplitArgs split_args(const QO& io, int B, int W, int H, int D, float* part, int2* pieces) {
  SplitArgs sa{B, W, H, D, io.Hq / H, W * io.n_q * (io.Hq / H), 0, part, pieces, false, false, false};
  sa.MC = split_chunks(sa.M, D);
  sa.out8 = (reinterpret_cast<uintptr_t>(io.o) & 7) == 0 && (io.o_row | io.o_tok | io.o_head) % 4 == 0;
  sa.q8 = (reinterpret_cast<uintptr_t>(io.q) & 7) == 0 && (io.q_row | io.q_tok | io.q_head) % 4 == 0;
  return sa;
}

}  // namespace vbs
