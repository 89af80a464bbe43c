// Kernel kinds for the optional event timing, those of moe_internal.h and the
// decoder-block operators' after them. (A header of its own: committed traffic
// figures of the decode kernels hold as long as moe_internal.h is unchanged.)
#pragma once

#include "moe_internal.h"

namespace moe {

enum BlockKernelKind : int { K_NORM = K_NUM_KINDS, K_LOGPROBS, K_LINEAR_STEP, K_LINEAR_CHUNK, K_ALL_KINDS };

}  // namespace moe
