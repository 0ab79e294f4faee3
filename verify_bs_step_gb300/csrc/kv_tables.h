// Block tables and slot maps from request lengths: the launchers' interface.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "bs_internal.h"

namespace vbs {

// The flat list of `n` requests' tokens: request i covers positions [start[i], start[i] + count[i])
// (start NULL: 0) of row i, or of the first row of sentence i when n is the number of sentences.
struct SlotArgs {
  int n;
  const int32_t* start;
  const int32_t* count;
  int64_t cap;                    // entries of slots / pos / row; unused ones become -1
  int64_t* slots;
  int32_t* pos;                   // may be NULL
  int32_t* row;                   // may be NULL
  int32_t* cu;                    // [n + 1] exclusive sums; may be NULL
  int32_t* scan;                  // [n + 1] workspace
};

// With `build` the tables, counts and free stacks are laid down for the counts first (n = B).
int launch_kv_build(const PagedArgs& a, const SlotArgs& s, bool build, int num_sms, cudaStream_t stream);

}  // namespace vbs
