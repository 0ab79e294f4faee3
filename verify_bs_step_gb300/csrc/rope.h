// Rotary positions, and the write into the 16-bit paged cache: the launcher's interface.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "bs_internal.h"

namespace vbs {

constexpr int ROPE_MAX_D = 256;

// Turns a position makes, per pair of rotated dims, as fractions of 2^64; what the rotated values are scaled by.
struct RopeGeom {
  const unsigned long long* turns;   // [rot / 2], NULL: nothing is rotated
  int rot, layout;
  float amp;
};

// Rows of `heads` heads: element (token, head, d) at p[token * tok + head * head_s + d]; p NULL: none.
struct RopeRows {
  const void* in;
  void* out;                         // NULL: not written
  int64_t in_tok, in_head, out_tok, out_head;
  int heads;
};

// A 16-bit cache's layer: pool [NB][L][2][H][block][D]; pool NULL: none.
struct Kv16Geom {
  uint16_t* pool;
  int64_t NB;
  int L, H, block, D, layer;
  int* status;
};

struct RopeArgs {
  int64_t n;
  const int32_t* pos;                // a negative one: the token is skipped; NULL with nothing rotated
  const int64_t* slots;              // of the cache, -1: not written there
  RopeGeom r;
  RopeRows q, k, v;                  // v goes to the cache alone
  Kv16Geom kv;
  int D, dtype;
};

int launch_rope(const RopeArgs& a, int num_sms, cudaStream_t s);

}  // namespace vbs
