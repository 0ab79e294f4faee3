// Attention over the 8-bit paged cache and over an encoder's states: the launchers' interface.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "bs_internal.h"
#include "kv8.h"

namespace vbs {

// Query rows and outputs (bf16): element (row, token, head, d) at p[row * row_s + token * tok + head * head_s + d].
struct QO {
  const uint16_t* q;
  uint16_t* o;
  int64_t q_row, q_tok, q_head, o_row, o_tok, o_head;
  int n_q, Hq;
  float scale;
};

// The encoder's keys and values (bf16): element (sentence, position, head, d) at p[b * sent + s * pos + h * head + d].
struct EncKV {
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_sent, k_pos, k_head, v_sent, v_pos, v_head;
  const int32_t* len;             // [B] positions of each sentence, at most S
  int S, B, W, H, D;
  int* status;
};

int launch_kv8_plan(const PagedArgs& a, const int32_t* ctx, int32_t* seen, cudaStream_t s);
int launch_kv8_attention(const PagedArgs& a, const Kv8Geom& g, const QO& io, const int32_t* seen, cudaStream_t s);
int launch_xattn(const EncKV& kv, const QO& io, cudaStream_t s);

}  // namespace vbs
