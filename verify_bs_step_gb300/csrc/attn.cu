// The plan of a step's attention over the 8-bit paged cache (sm_103a).
//
// The plan turns the block tables into each sentence's list of distinct pages: a page that several
// beams share stands in it once, with the beams that see it, so that attention reads it once.  It is a
// pass over R x pages table entries, made once a step and shared by the layers; latency bounds it (lengths, block
// counts, a column's entries together, the list: 64 sentences x 4 beams x 67 pages take 7 us alone).

#include "attn.h"
#include "attn_split.cuh"
#include "common.cuh"

namespace vbs {

constexpr int PLAN_NT = 256;

// A row's cached positions, held to what its table covers.
__device__ __forceinline__ int held_len(const PagedArgs& a, const int32_t* ctx, int r) {
  const int n = ctx[r];
  const int64_t most = static_cast<int64_t>(a.nblk[r]) * a.block;
  if (n < 0 || n > most) set_status(a.status, VBS_EINVAL);
  return n < 0 ? 0 : static_cast<int>(n < most ? n : most);
}

// A CTA a sentence; a thread looks at one table column of its W rows at a time.
__global__ void __launch_bounds__(PLAN_NT) kv8_plan_kernel(const PagedArgs a, const int32_t* ctx, const Kv8Plan p) {
  __shared__ int seen[WMAX];
  __shared__ int sums[PLAN_NT / 32];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, W = a.W;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid < W) {
    seen[tid] = held_len(a, ctx, b * W + tid);
    p.seen[b * W + tid] = seen[tid];
  }
  __syncthreads();
  int most = 0;
  for (int w = 0; w < W; ++w) most = max(most, seen[w]);
  const int cols = static_cast<int>((static_cast<u32>(most) + a.block - 1) / a.block);
  const int32_t* tab = a.table + static_cast<int64_t>(b) * W * a.MB;
  int4* list = p.list + static_cast<int64_t>(b) * a.S;
  int carry = 0;
  for (int j0 = 0; j0 < cols; j0 += PLAN_NT) {
    const int j = j0 + tid;
    int id[WMAX];
    u32 lead = 0;                                   // the beams that name a page first
#pragma unroll
    for (int w = 0; w < WMAX; ++w)                  // the column's entries, all on their way at once
      id[w] = w < W && j < cols && j * a.block < seen[w] ? tab[static_cast<int64_t>(w) * a.MB + j] : -1;
#pragma unroll
    for (int w = 0; w < WMAX; ++w) {
      if (id[w] < 0) continue;
      if (id[w] < b * a.S || id[w] >= (b + 1) * a.S) {     // not a page of this sentence
        set_status(a.status, VBS_EINVAL);
        id[w] = -1;
        continue;
      }
      bool first = true;
#pragma unroll
      for (int x = 0; x < w; ++x) first = first && id[x] != id[w];
      if (first) lead |= 1u << w;
    }
    const int n = __popc(lead);
    int at = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(FULL, at, d);
      if (lane >= d) at += y;
    }
    if (lane == 31) sums[wid] = at;
    __syncthreads();
    int all = 0;
    at += carry - n;
    for (int w = 0; w < PLAN_NT / 32; ++w) {
      if (w < wid) at += sums[w];
      all += sums[w];
    }
#pragma unroll
    for (int w = 0; w < WMAX; ++w) {
      if (!(lead >> w & 1u)) continue;
      u32 rows = 0;
      int to = 0;
#pragma unroll
      for (int x = w; x < WMAX; ++x)
        if (id[x] == id[w]) {
          rows |= 1u << x;
          to = max(to, seen[x]);
        }
      if (at < a.S) list[at] = make_int4(id[w], j * a.block, static_cast<int>(rows), min(a.block, to - j * a.block));
      else set_status(a.status, VBS_EINVAL);        // a page in two columns: not a table of this library
      ++at;
    }
    carry += all;
    __syncthreads();
  }
  if (tid == 0) {
    // a sentence with nothing to see has one page of no positions: its rows get their zeros from it
    if (carry == 0) list[0] = make_int4(0, 0, 0, 0);
    p.n_pages[b] = max(1, min(carry, a.S));
  }
}

// One row a sentence: the list is the table's row; CTA (b, c) copies every c-th chunk of it.
__global__ void __launch_bounds__(PLAN_NT)
kv8_plan_rows_kernel(const PagedArgs a, const int32_t* ctx, const Kv8Plan p) {
  const int b = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int seen = held_len(a, ctx, b);
  const int cols = static_cast<int>((static_cast<u32>(seen) + a.block - 1) / a.block);
  int4* list = p.list + static_cast<int64_t>(b) * a.S;
  for (int j = blockIdx.y * PLAN_NT + threadIdx.x; j < min(cols, a.S); j += gridDim.y * PLAN_NT) {
    const int id = a.table[static_cast<int64_t>(b) * a.MB + j];
    const bool ok = id >= b * a.S && id < (b + 1) * a.S;
    if (!ok) set_status(a.status, VBS_EINVAL);
    list[j] = make_int4(ok ? id : 0, j * a.block, ok ? 1 : 0, ok ? min(a.block, seen - j * a.block) : 0);
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    if (cols == 0) list[0] = make_int4(0, 0, 0, 0);
    p.n_pages[b] = max(1, min(cols, a.S));
    p.seen[b] = seen;
  }
}

int launch_kv8_plan(const PagedArgs& a, const int32_t* ctx, const Kv8Plan& p, cudaStream_t s) {
  if (a.W == 1) {
    const int chunks = std::min((std::min(a.MB, a.S) + PLAN_NT - 1) / PLAN_NT, 64);
    return launch_dependent(kv8_plan_rows_kernel, dim3(a.B, chunks), dim3(PLAN_NT), 0, s, a, ctx, p);
  }
  return launch_dependent(kv8_plan_kernel, dim3(a.B), dim3(PLAN_NT), 0, s, a, ctx, p);
}

int64_t attn_part_floats(int D, int num_sms) { return split_part_floats(D, num_sms); }

int64_t attn_segments(int B, int W, int H, int D, int Hq, int n_q) {
  return static_cast<int64_t>(B) * H * split_chunks(W * n_q * (Hq / H), D);
}

int launch_kv8_attention(const PagedArgs& a, const Kv8Geom& g, const QO& io, const Kv8Plan& p, float* part,
                         int2* pieces, int num_sms, cudaStream_t s) {
  return g.fmt == VBS_I8 ? launch_kv8_attention_i8(a, g, io, p, part, pieces, num_sms, s)
                         : launch_kv8_attention_e4m3(a, g, io, p, part, pieces, num_sms, s);
}

}  // namespace vbs
