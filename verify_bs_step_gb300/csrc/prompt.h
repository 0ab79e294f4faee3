// Attention of packed prompts to themselves: the launchers' interface.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "bs_internal.h"

namespace vbs {

// Packed requests (bf16): token t, head h, dim d of q at q[t * q_tok + h * q_head + d], k, v and out likewise; request b
// has the tokens cu[b] .. cu[b + 1] - 1.
struct PromptArgs {
  const uint16_t *q, *k, *v;
  uint16_t* o;
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, o_tok, o_head;
  const int32_t* cu;              // [B + 1]
  int N, B, Hq, H, D;
  bool causal;
  float scale;
  int* status;
};

// The last request that starts at or before token t: its first token and its end (0, 0: t is in none).
__device__ __forceinline__ int2 request_of(const PromptArgs& a, int t) {
  int lo = 0, hi = a.B + 1;       // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a.cu[m] <= t) lo = m;
    else hi = m;
  }
  if (lo == a.B || a.cu[lo] > t) return make_int2(0, 0);
  const int s = a.cu[lo], e = a.cu[lo + 1];
  return s >= 0 && e > t && e <= a.N ? make_int2(s, e) : make_int2(0, 0);
}

int launch_prompt_rows(const PromptArgs& a, cudaStream_t s);
// Whether the tiles take this call: up to 128 heads a group, and rows that TMA can read.
bool prompt_tc_takes(const PromptArgs& a);
int launch_prompt_tc(const PromptArgs& a, int num_sms, cudaStream_t s);

}  // namespace vbs
