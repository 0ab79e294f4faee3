// Attention of packed prompts to themselves, for rows that TMA cannot read and more than 128 heads a group (sm_103a).
//
// A CTA takes 16 query rows (tokens, the heads of a group side by side) of one K/V head over the positions that any of
// them sees, 32 at a time: K and V come to shared memory in fp32, a lane scores one position for its warp's four rows,
// and keeps D / 32 dims of their sums.  Scores, the running maximum and sum, and the sums are fp32, products plain
// fp32 arithmetic: it is the form for layouts out of the ordinary, and bound by that arithmetic
// (2000 tokens x 32 heads over 8 x 128: 2940 us, 11 TFLOP/s; the tiles take 34).

#include <cuda_bf16.h>

#include "common.cuh"
#include "prompt.h"

namespace vbs {

constexpr int PR_ROWS = 16, PR_N = 32, PR_NT = 128, PR_PER = PR_ROWS / (PR_NT / 32);

template <int DL>                                   // dims a lane
__global__ void __launch_bounds__(PR_NT) prompt_rows_kernel(const PromptArgs a, int GC, int TT, int tiles) {
  constexpr int D = 32 * DL, LD = D + 1;
  extern __shared__ float pr_smem[];
  float *ks = pr_smem, *vs = ks + PR_N * LD, *qs = vs + PR_N * LD;
  __shared__ int2 span[PR_ROWS];                    // positions [x, y) that a row sees; none: a row that is not there
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int G = a.Hq / a.H, chunks = (G + GC - 1) / GC;      // GC heads of a group at a time
  const int hc = blockIdx.x % (a.H * chunks), h = hc / chunks, g0 = hc % chunks * GC;
  const int tile = tiles - 1 - static_cast<int>(blockIdx.x / (a.H * chunks));   // long rows first
  if (blockIdx.x == 0)
    for (int b = tid; b < a.B; b += PR_NT)
      if (a.cu[b] < 0 || a.cu[b] > a.cu[b + 1] || a.cu[b + 1] > a.N) set_status(a.status, VBS_EINVAL);
  if (tid < PR_ROWS) {
    const int t = tile * TT + tid / GC;
    int2 r = make_int2(0, 0);
    if (tid < TT * GC && g0 + tid % GC < G && t < a.N) {
      r = request_of(a, t);
      if (r.y > 0 && a.causal) r.y = t + 1;
    }
    span[tid] = r;
  }
  __syncthreads();
  int p0 = a.N, p1 = 0;
  for (int r = 0; r < PR_ROWS; ++r)
    if (span[r].y > span[r].x) {
      p0 = min(p0, span[r].x);
      p1 = max(p1, span[r].y);
    }
  for (int i = tid; i < PR_ROWS * D; i += PR_NT) {
    const int r = i / D, d = i % D;
    const int64_t at = static_cast<int64_t>(tile * TT + r / GC) * a.q_tok + static_cast<int64_t>(h * G + g0 + r % GC) * a.q_head + d;
    qs[r * D + d] = span[r].y > span[r].x && d < a.D ? bf16_lo(a.q[at]) : 0.f;
  }
  const float sc = a.scale * LOG2E_F;
  float m[PR_PER], l[PR_PER], o[PR_PER][DL];
#pragma unroll
  for (int x = 0; x < PR_PER; ++x) {
    m[x] = -INFINITY;
    l[x] = 0.f;
#pragma unroll
    for (int i = 0; i < DL; ++i) o[x][i] = 0.f;
  }
  for (int p = p0; p < p1; p += PR_N) {
    __syncthreads();
    for (int i = tid; i < PR_N * D; i += PR_NT) {
      const int r = i / D, d = i % D;
      const bool there = p + r < p1 && d < a.D;
      ks[r * LD + d] = there ? bf16_lo(a.k[static_cast<int64_t>(p + r) * a.k_tok + h * a.k_head + d]) : 0.f;
      vs[r * LD + d] = there ? bf16_lo(a.v[static_cast<int64_t>(p + r) * a.v_tok + h * a.v_head + d]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < PR_PER; ++x) {
      const int r = wid * PR_PER + x;
      const int2 sp = span[r];
      const bool sees = p + lane >= sp.x && p + lane < sp.y;
      const u32 who = __ballot_sync(FULL, sees);
      if (who == 0) continue;
      float s = 0.f;
      for (int d = 0; d < a.D; ++d) s = fmaf(qs[r * D + d], ks[lane * LD + d], s);
      s = sees ? s * sc : -INFINITY;
      float top = s;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, k));
      top = fmaxf(top, m[x]);
      const float ref = top == -INFINITY ? 0.f : top;
      const float corr = m[x] == -INFINITY ? 0.f : ex2(m[x] - ref);
      const float w = ex2(s - ref);
      float sum = w;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(FULL, sum, k);
      m[x] = top;
      l[x] = l[x] * corr + sum;
#pragma unroll
      for (int i = 0; i < DL; ++i) o[x][i] *= corr;
      for (int y = 0; y < PR_N; ++y) {
        if (!(who >> y & 1u)) continue;             // (what a row does not see may hold anything)
        const float wy = __shfl_sync(FULL, w, y);
#pragma unroll
        for (int i = 0; i < DL; ++i) o[x][i] = fmaf(wy, vs[y * LD + i * 32 + lane], o[x][i]);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < PR_PER; ++x) {
    const int r = wid * PR_PER + x;
    if (span[r].y <= span[r].x) continue;
    uint16_t* out = a.o + static_cast<int64_t>(tile * TT + r / GC) * a.o_tok + static_cast<int64_t>(h * G + g0 + r % GC) * a.o_head;
    const float inv = 1.f / l[x];                   // (0 / 0 where every score is -inf: NaN)
#pragma unroll
    for (int i = 0; i < DL; ++i)
      if (i * 32 + lane < a.D) out[i * 32 + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(o[x][i] * inv));
  }
}

template <int DL> static int launch_rows(const PromptArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};
  constexpr int smem = (2 * PR_N * (32 * DL + 1) + PR_ROWS * 32 * DL) * 4;
  if (!smem_attr_once(prompt_rows_kernel<DL>, smem, attr_done)) return VBS_ECUDA;
  const int G = a.Hq / a.H, GC = std::min(G, PR_ROWS);
  const int TT = PR_ROWS / GC, tiles = (a.N + TT - 1) / TT;
  const int64_t grid = static_cast<int64_t>(tiles) * a.H * ((G + GC - 1) / GC);
  if (grid >= int64_t{1} << 31) return VBS_EINVAL;
  prompt_rows_kernel<DL><<<static_cast<unsigned>(grid), PR_NT, smem, s>>>(a, GC, TT, tiles);
  return cudaGetLastError() == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

int launch_prompt_rows(const PromptArgs& a, cudaStream_t s) {
  if (a.D <= 64) return launch_rows<2>(a, s);
  if (a.D <= 128) return launch_rows<4>(a, s);
  return launch_rows<8>(a, s);
}

}  // namespace vbs
