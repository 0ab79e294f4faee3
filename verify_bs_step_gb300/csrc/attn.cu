// Attention over the 8-bit paged cache and over an encoder's states (sm_103a).
//
//   o = sum_p softmax_p(scale q . k_p) v_p   over the positions p that a query sees
//
// with the running maximum m and sum l of a one-pass softmax, in fp32: a chunk of scores with
// maximum m' moves l and o to the new reference by 2^(m - max(m, m')).  A query that sees nothing
// gives zeros.
//
// One warp per (row, query token, query head): a lane scores one of 32 positions at a time, then the
// lanes share the head's dims for the weighted sum of the values.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "attn.h"
#include "common.cuh"

namespace vbs {

constexpr int AT_NT = 128;
constexpr int AT_DMAX = 256;

template <int FMT> struct Paged8 {
  PagedArgs a;
  Kv8Geom g;
  const int32_t* seen;            // [R] cached positions of each row
  int h;
  int row;
  __device__ int count(int r) const { return seen[r]; }
  __device__ float load(int kv, int p, int d) const {
    const int64_t page = a.table[static_cast<int64_t>(row) * a.MB + p / g.block];
    const int64_t run = g.run(page, kv, h);
    const uint8_t c = reinterpret_cast<const uint8_t*>(g.pool)[(run * g.block + p % g.block) * g.D + d];
    if (FMT == VBS_I8) return static_cast<float>(static_cast<int8_t>(c)) * g.scales[run];
    __nv_fp8_e4m3 f;
    f.__x = c;
    return static_cast<float>(f) * g.scales[run];
  }
};

struct EncRows {
  EncKV e;
  int h, row;
  __device__ int count(int r) const {
    const int n = e.len[r / e.W];
    if (n >= 0 && n <= e.S) return n;
    set_status(e.status, VBS_EINVAL);
    return n < 0 ? 0 : e.S;
  }
  __device__ float load(int kv, int p, int d) const {
    const int64_t b = row / e.W;
    const uint16_t x = kv ? e.v[b * e.v_sent + p * e.v_pos + h * e.v_head + d]
                          : e.k[b * e.k_sent + p * e.k_pos + h * e.k_head + d];
    return __uint_as_float(static_cast<u32>(x) << 16);
  }
};

template <class KV>
__global__ void __launch_bounds__(AT_NT) attn_warp_kernel(KV kv, const QO io, int64_t items, int H, int D, bool causal) {
  __shared__ float qs[AT_NT / 32][AT_DMAX];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (AT_NT / 32) + w;
  if (item >= items) return;
  const int hq = static_cast<int>(item % io.Hq);
  const int i = static_cast<int>(item / io.Hq % io.n_q);
  const int row = static_cast<int>(item / io.Hq / io.n_q);
  kv.h = hq / (io.Hq / H);
  kv.row = row;
  const uint16_t* q = io.q + row * io.q_row + i * io.q_tok + hq * io.q_head;
  for (int d = lane; d < D; d += 32) qs[w][d] = __uint_as_float(static_cast<u32>(q[d]) << 16) * io.scale * LOG2E_F;
  __syncwarp();
  const int T = kv.count(row) - (causal ? io.n_q - 1 - i : 0);
  float m = -INFINITY, l = 0.f, o[AT_DMAX / 32];
#pragma unroll
  for (int u = 0; u < AT_DMAX / 32; ++u) o[u] = 0.f;
  for (int p0 = 0; p0 < T; p0 += 32) {
    const int p = p0 + lane;
    float s = -INFINITY;
    if (p < T) {
      s = 0.f;
      for (int d = 0; d < D; ++d) s += qs[w][d] * kv.load(0, p, d);
    }
    float mx = s;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, k));
    const float mn = fmaxf(m, mx);
    const float corr = ex2(m - mn);
    const float pr = ex2(s - mn);
    float sum = pr;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(FULL, sum, k);
    l = l * corr + sum;
    m = mn;
#pragma unroll
    for (int u = 0; u < AT_DMAX / 32; ++u) o[u] *= corr;
    const int n = min(32, T - p0);
    for (int j = 0; j < n; ++j) {
      const float pj = __shfl_sync(FULL, pr, j);
#pragma unroll
      for (int u = 0; u < AT_DMAX / 32; ++u)
        if (u * 32 + lane < D) o[u] += pj * kv.load(1, p0 + j, u * 32 + lane);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
  uint16_t* out = io.o + row * io.o_row + i * io.o_tok + hq * io.o_head;
#pragma unroll
  for (int u = 0; u < AT_DMAX / 32; ++u)
    if (u * 32 + lane < D) out[u * 32 + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(o[u] * inv));
}

// Each row's cached positions, held to what its table covers.
__global__ void kv8_plan_kernel(const PagedArgs a, const int32_t* ctx, int32_t* seen, int R) {
  const int r = blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= R) return;
  const int n = ctx[r];
  const int64_t most = static_cast<int64_t>(a.nblk[r]) * a.block;
  if (n < 0 || n > most) set_status(a.status, VBS_EINVAL);
  seen[r] = n < 0 ? 0 : static_cast<int>(n < most ? n : most);
}

int launch_kv8_plan(const PagedArgs& a, const int32_t* ctx, int32_t* seen, cudaStream_t s) {
  const int R = a.B * a.W;
  kv8_plan_kernel<<<(R + 127) / 128, 128, 0, s>>>(a, ctx, seen, R);
  return cudaGetLastError() == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

int launch_kv8_attention(const PagedArgs& a, const Kv8Geom& g, const QO& io, const int32_t* seen, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(a.B) * a.W * io.n_q * io.Hq;
  const unsigned grid = static_cast<unsigned>((items + AT_NT / 32 - 1) / (AT_NT / 32));
  if (g.fmt == VBS_I8)
    attn_warp_kernel<<<grid, AT_NT, 0, s>>>(Paged8<VBS_I8>{a, g, seen, 0, 0}, io, items, g.H, g.D, true);
  else
    attn_warp_kernel<<<grid, AT_NT, 0, s>>>(Paged8<VBS_E4M3>{a, g, seen, 0, 0}, io, items, g.H, g.D, true);
  return cudaGetLastError() == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

int launch_xattn(const EncKV& e, const QO& io, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(e.B) * e.W * io.n_q * io.Hq;
  const unsigned grid = static_cast<unsigned>((items + AT_NT / 32 - 1) / (AT_NT / 32));
  attn_warp_kernel<<<grid, AT_NT, 0, s>>>(EncRows{e, 0, 0}, io, items, e.H, e.D, false);
  return cudaGetLastError() == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

}  // namespace vbs
