// Host-side helpers and context types shared by the C ABI's translation units.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "bs_internal.h"
#include "kv_tables.h"

#define VBS_EXPORT extern "C" __attribute__((visibility("default")))

namespace vbs {

inline int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return n;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// One device allocation carved into 256-byte aligned pieces.
struct Carver {
  size_t off = 0;
  char* base = nullptr;
  template <class T> T* take(size_t n) {
    off = (off + 255) & ~static_cast<size_t>(255);
    T* p = reinterpret_cast<T*>(base ? base + off : nullptr);
    off += n * sizeof(T);
    return p;
  }
};

}  // namespace vbs

struct vbs_pkv {
  vbs::PagedArgs a;
  cudaStream_t stream;
  int32_t* identity;
  int R;
  int elem_bytes;
  float* scales;         // of an 8-bit cache (kv8_init), else NULL: copy-on-write carries a page's scales along
  void* dev_block;
  char* state;           // table .. base: one contiguous range of the allocation
  char* saved;           // its copy (kv_paged_save / kv_paged_restore)
  size_t state_bytes;
  bool copy_pending;     // bs_step_paged recorded copies that kv_paged_copy has not run
  int32_t* scan;         // [R + 1] exclusive sums of a slot map's counts
  int64_t tables;        // how often the tables may have changed: an attention plan holds for the tables it was made from
};
