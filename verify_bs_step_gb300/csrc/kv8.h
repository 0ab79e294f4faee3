// The 8-bit paged cache: what its kernels take, and the launchers' interface.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "bs_internal.h"

namespace vbs {

constexpr int KV8_E_LO = -60, KV8_E_HI = 60;      // the range of the scales' exponents

// The cache as the kernels see it: pool [NB][L][2][H][block][D] of one byte each, scales [NB][L][2][H].
struct Kv8Geom {
  char* pool;
  float* scales;
  int fmt;                        // VBS_I8 or VBS_E4M3
  int64_t NB;
  int L, H, block, D;
  int layer;
  int* status;
  // the (layer, k/v, head) run of page p
  __host__ __device__ int64_t run(int64_t p, int kv, int h) const {
    return ((p * L + layer) * 2 + kv) * H + h;
  }
};

// New rows: element (token, head, d) at base[token * tok + head * head_stride + d].
struct Kv8Src {
  const void* k;
  const void* v;
  int64_t k_tok, k_head, v_tok, v_head;
  int dtype;                      // VBS_F32 or VBS_BF16
};

int launch_kv8_append(const Kv8Geom& g, const Kv8Src& src, int64_t n, const int64_t* slots, int num_sms,
                      cudaStream_t s);
// values of the slots as bf16 [n][H][D] each (zeros for slot -1)
int launch_kv8_read(const Kv8Geom& g, int64_t n, const int64_t* slots, void* k_out, void* v_out, int num_sms,
                    cudaStream_t s);

}  // namespace vbs
