// Attention over a cache of float8 e4m3 codes: the split kernel's instances.

#include "attn_split.cuh"

namespace vbs {

int launch_kv8_attention_e4m3(const PagedArgs& a, const Kv8Geom& g, const QO& io, const Kv8Plan& p, float* part,
                         int2* pieces, int num_sms, cudaStream_t s) {
  const PagedSrc<VBS_E4M3> src{g, p.list, p.n_pages, p.seen, a.S, (g.block + 15) / 16};
  return launch_split<PagedSrc<VBS_E4M3>, true>(src, io, split_args(io, a.B, a.W, g.H, g.D, part, pieces), num_sms, s);
}

}  // namespace vbs
