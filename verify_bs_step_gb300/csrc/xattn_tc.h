// Cross attention of many query rows on tcgen05 tiles: the launcher's interface.
#pragma once

#include "attn.h"

namespace vbs {

// Whether the tiles take this call: enough rows, and K and V that TMA can read.
bool xattn_tc_takes(const EncKV& e, const QO& io, int num_sms);
int launch_xattn_tc(const EncKV& e, const QO& io, int num_sms, cudaStream_t s);

}  // namespace vbs
