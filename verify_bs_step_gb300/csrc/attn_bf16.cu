// Attention over a 16-bit paged cache: the split kernel's instances.

#include "attn_split.cuh"

namespace vbs {

int launch_kv16_attention(const PagedArgs& a, const Kv16Geom& g, const QO& io, const Kv8Plan& p, float* part,
                          int2* pieces, int num_sms, cudaStream_t s) {
  const Paged16Src src{g, p.list, p.n_pages, p.seen, a.S, (g.block + 15) / 16};
  return launch_split<Paged16Src, true>(src, io, split_args(io, a.B, a.W, g.H, g.D, part, pieces), num_sms, s);
}

}  // namespace vbs
