// Block tables and slot maps from request lengths, on the GPU (sm_103a).
//
// For request lengths len[b], sentence b gets n = ceil(len / block) blocks b*S, b*S + 1, ...
// named by all W rows' tables, reference counts W on them, and a free stack that hands out
// the rest in ascending order.  The flat token list of n requests is laid out one request after
// the other (cu = exclusive sums of the counts); the token at position p of request i lives in slot
// table[row][p / block] * block + p % block of a layer's pool.
//
// Both are stores with no reuse (16 bytes a token, 4 a table entry), so the time is the
// launch plus the bytes at the write bandwidth; the only dependence between requests is the
// sum of the counts before them: up to TAB_SCAN requests every CTA adds up the counts itself (n / 256
// loads a thread, from L2, in one launch); more take a scan kernel first.  8 requests take 4.3 us, 1024 with 2.1 million
// tokens 14.5 (2.4 TB/s of stores, the launch included); more CTAs a request cost more in sums than they gain (4: 18.6).

#include "common.cuh"
#include "kv_tables.h"

namespace vbs {

constexpr int TAB_NT = 256;
constexpr int TAB_SCAN = 4096;

// A request's length if the cache can hold it, else 0 (and the status says so).
__device__ __forceinline__ int valid_len(const PagedArgs& a, int len) {
  const int most = a.S < a.MB ? a.S : a.MB;
  if (len >= 0 && len <= static_cast<int64_t>(most) * a.block) return len;
  set_status(a.status, VBS_EINVAL);
  return 0;
}

__device__ __forceinline__ int valid_count(const PagedArgs& a, const SlotArgs& s, int i, bool build) {
  const int c = s.count[i];
  if (build) return valid_len(a, c);
  const int st = s.start ? s.start[i] : 0;
  if (c >= 0 && st >= 0 && static_cast<int64_t>(st) + c <= static_cast<int64_t>(a.MB) * a.block) return c;
  set_status(a.status, VBS_EINVAL);
  return 0;
}

// Exclusive sums of the counts into scan[0..n] (and cu): one CTA.
__global__ void __launch_bounds__(1024) kv_scan_kernel(const PagedArgs a, const SlotArgs s, bool build) {
  __shared__ int64_t warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  int64_t carry = 0;
  for (int i0 = 0; i0 < s.n; i0 += 1024) {
    const int i = i0 + tid;
    const int64_t v = i < s.n ? valid_count(a, s, i, build) : 0;
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(FULL, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) warp_sum[wid] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
      const int64_t t = warp_sum[w];
      if (w < wid) before += t;
      all += t;
    }
    const int64_t ex = carry + before + x - v;
    if (i < s.n) {
      const int e = static_cast<int>(ex < INT32_MAX ? ex : INT32_MAX);
      s.scan[i] = e;
      if (s.cu) s.cu[i] = e;
    }
    carry += all;
    __syncthreads();
  }
  if (tid == 0) {
    const int e = static_cast<int>(carry < INT32_MAX ? carry : INT32_MAX);
    s.scan[s.n] = e;
    if (s.cu) s.cu[s.n] = e;
    if (carry > s.cap && s.slots) set_status(a.status, VBS_EINVAL);
  }
}

// The sum of the counts before request i, and of all, added up by the whole CTA.
__device__ __forceinline__ void sums_of(const PagedArgs& a, const SlotArgs& s, int i, bool build, int64_t& before,
                                        int64_t& all) {
  __shared__ int64_t part[2][TAB_NT / 32];
  const int tid = threadIdx.x;
  int64_t lo = 0, hi = 0;
  for (int j = tid; j < s.n; j += TAB_NT) {
    const int c = valid_count(a, s, j, build);
    if (j < i) lo += c;
    else hi += c;
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    lo += __shfl_xor_sync(FULL, lo, m);
    hi += __shfl_xor_sync(FULL, hi, m);
  }
  if ((tid & 31) == 0) {
    part[0][tid >> 5] = lo;
    part[1][tid >> 5] = hi;
  }
  __syncthreads();
  before = all = 0;
  for (int w = 0; w < TAB_NT / 32; ++w) {
    before += part[0][w];
    all += part[1][w];
  }
  all += before;
}

// CTA (i, c): chunk c of request i's table rows and tokens; SCANNED: s.scan holds the sums.
template <bool SCANNED>
__global__ void __launch_bounds__(TAB_NT) kv_build_kernel(const PagedArgs a, const SlotArgs s, bool build) {
  const int i = blockIdx.x, tid = threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.y) * TAB_NT;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * TAB_NT + tid;
  const int count = valid_count(a, s, i, build);
  const int start = s.start ? s.start[i] : 0;
  int64_t first = 0, total = 0;
  if (SCANNED) {
    first = s.scan[i];
    total = s.scan[s.n];
  } else if (s.slots || s.cu) {
    sums_of(a, s, i, build, first, total);
    if (blockIdx.y == 0 && tid == 0) {
      if (s.cu) s.cu[i] = static_cast<int>(first < INT32_MAX ? first : INT32_MAX);
      if (i == s.n - 1) {
        if (s.cu) s.cu[s.n] = static_cast<int>(total < INT32_MAX ? total : INT32_MAX);
        if (total > s.cap && s.slots) set_status(a.status, VBS_EINVAL);
      }
    }
  }
  const int row = build || s.n == a.B ? i * a.W : i;
  const int32_t* tab = a.table + static_cast<int64_t>(row) * a.MB;
  if (build) {
    const int nb = static_cast<int>((static_cast<u32>(count) + a.block - 1) / a.block);
    for (int w = 0; w < a.W; ++w)
      for (int64_t c = t0; c < a.MB; c += step)
        a.table[(static_cast<int64_t>(row) + w) * a.MB + c] = c < nb ? i * a.S + static_cast<int>(c) : -1;
    for (int64_t j = t0; j < a.S; j += step) {
      a.refcnt[static_cast<int64_t>(i) * a.S + j] = j < nb ? a.W : 0;
      a.stack[static_cast<int64_t>(i) * a.S + j] = i * a.S + (a.S - 1 - static_cast<int>(j));
    }
    if (t0 < a.W) {
      a.nblk[row + t0] = nb;
      a.tasks[row + t0] = make_int4(0, 0, 0, 0);             // copies still pending refer to the tables before
    }
    if (t0 == 0) {
      a.top[i] = a.S - nb;
      a.base()[i] = count;
    }
  }
  if (!s.slots) return;
  const bool pow2 = (a.block & (a.block - 1)) == 0;         // the usual block: a shift for the division
  const int shift = __ffs(a.block) - 1;
  const int blocks = build ? 0 : a.nblk[row];
  for (int64_t k = t0; k < count; k += step) {
    const int64_t o = first + k;
    if (o >= s.cap) break;
    const int p = start + static_cast<int>(k);
    const int j = pow2 ? p >> shift : p / a.block;
    const int blk = build ? i * a.S + j : (j < blocks ? tab[j] : -1);
    if (blk < 0) set_status(a.status, VBS_EINVAL);          // a position that the table does not cover
    s.slots[o] = blk < 0 ? -1 : static_cast<int64_t>(blk) * a.block + (p - j * a.block);
    if (s.pos) s.pos[o] = p;
    if (s.row) s.row[o] = row;
  }
  // the entries past the last token, shared out over all CTAs
  const int64_t all = static_cast<int64_t>(gridDim.x) * step;
  for (int64_t o = total + i * step + t0; o < s.cap; o += all) {
    s.slots[o] = -1;
    if (s.pos) s.pos[o] = -1;
    if (s.row) s.row[o] = -1;
  }
}

int launch_kv_build(const PagedArgs& a, const SlotArgs& s, bool build, int num_sms, cudaStream_t stream) {
  // enough CTAs to fill the GPU when the requests are few and long
  const int64_t most = std::max<int64_t>(static_cast<int64_t>(a.MB) * a.block, static_cast<int64_t>(a.W) * a.MB);
  const int64_t want = (4 * static_cast<int64_t>(num_sms) + s.n - 1) / s.n;
  const int64_t chunks = std::max<int64_t>(1, std::min<int64_t>({want, (most + 2 * TAB_NT - 1) / (2 * TAB_NT), 65535}));
  const dim3 grid(s.n, static_cast<unsigned>(chunks));
  if (s.n > TAB_SCAN) {
    kv_scan_kernel<<<1, 1024, 0, stream>>>(a, s, build);
    kv_build_kernel<true><<<grid, TAB_NT, 0, stream>>>(a, s, build);
  } else {
    kv_build_kernel<false><<<grid, TAB_NT, 0, stream>>>(a, s, build);
  }
  return cudaGetLastError() == cudaSuccess ? VBS_OK : VBS_ECUDA;
}

}  // namespace vbs
