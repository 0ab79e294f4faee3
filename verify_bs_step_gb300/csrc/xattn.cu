// Cross attention to an encoder's states: the split kernel's instances for bf16 keys and values.

#include "attn_split.cuh"
#include "xattn_tc.h"

namespace vbs {

int launch_xattn(const EncKV& e, const QO& io, float* part, int2* pieces, int num_sms, cudaStream_t s, int* tiles) {
  *tiles = xattn_tc_takes(e, io, num_sms) ? 1 : 0;
  if (*tiles) return launch_xattn_tc(e, io, num_sms, s);
  const EncSrc src{e};
  const SplitArgs sa = split_args(io, e.B, e.W, e.H, e.D, part, pieces);
  const bool aligned = ((reinterpret_cast<uintptr_t>(e.k) | reinterpret_cast<uintptr_t>(e.v)) & 15) == 0 &&
                       (e.k_sent | e.k_pos | e.k_head | e.v_sent | e.v_pos | e.v_head) % 8 == 0;
  return aligned ? launch_split<EncSrc, true>(src, io, sa, num_sms, s) : launch_split<EncSrc, false>(src, io, sa, num_sms, s);
}

}  // namespace vbs
