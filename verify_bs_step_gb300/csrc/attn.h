// Attention over the 8-bit paged cache and over an encoder's states: the launchers' interface.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "bs_internal.h"
#include "kv8.h"
#include "rope.h"

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

// A step over the paged cache, from the block tables: each sentence's distinct pages
// (page, first position, the beams that see it, positions), their number, and the rows' lengths.
struct Kv8Plan {
  int4* list;                     // [B][S]
  int* n_pages;                   // [B]
  int* seen;                      // [R]
};

int launch_kv8_plan(const PagedArgs& a, const int32_t* ctx, const Kv8Plan& p, cudaStream_t s);

// Where no sentence can have more units of 16 positions than this (the cache's or the encoder's size says so), a CTA
// of the split kernel takes a whole segment, and the second launch is left out: up to 2 times as fast over 8 to 16384
// segments of head_dim 64 to 256 and 4 to 128 rows (8 segments x 16 units: 9 to 7 us; 512 x 16: 15 to 13; 64 x 48: 14 to
// 11; at worst 512 x 48 of head_dim 128: 31 to 33, and 16384 x 4: 206 to 223); with 64 units few segments lose (8 x 64:
// 14.5 to 15.6), with 128 most.
constexpr int SP_WHOLE = 48;

// Workspace of the split: attn_part_floats floats of partials, and attn_segments entries of where each segment's are.
int64_t attn_part_floats(int D, int num_sms);
int64_t attn_segments(int B, int W, int H, int D, int Hq, int n_q);
int launch_kv8_attention(const PagedArgs& a, const Kv8Geom& g, const QO& io, const Kv8Plan& p, float* part,
                         int2* pieces, int num_sms, cudaStream_t s);
int launch_kv8_attention_i8(const PagedArgs& a, const Kv8Geom& g, const QO& io, const Kv8Plan& p, float* part,
                            int2* pieces, int num_sms, cudaStream_t s);
int launch_kv8_attention_e4m3(const PagedArgs& a, const Kv8Geom& g, const QO& io, const Kv8Plan& p, float* part,
                              int2* pieces, int num_sms, cudaStream_t s);
int launch_kv16_attention(const PagedArgs& a, const Kv16Geom& g, const QO& io, const Kv8Plan& p, float* part,
                          int2* pieces, int num_sms, cudaStream_t s);
// *tiles: whether the tcgen05 tiles took the call
int launch_xattn(const EncKV& kv, const QO& io, float* part, int2* pieces, int num_sms, cudaStream_t s, int* tiles);

}  // namespace vbs
