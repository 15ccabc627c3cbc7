// debug_hooks.h -- a test hook of the expert operators, exported only by the debug
// build of the library (-DMOE_DEBUG_HOOKS, libmoe_permute_debug.so).
#pragma once

#include "moe_experts.h"

// The same in the source of the 8-bit operators, whose kernels have variables of their own.
namespace moe {
namespace experts {
bool set_quant_wait(int slices, unsigned long long wait_ns);
}  // namespace experts
}  // namespace moe

extern "C" {

// From the next launch on, a wait inside the expert products (of 16 and 8 bits) gives up after
// `wait_ns` nanoseconds without progress, and, with slices > 0, each block's
// producer stops after that many slices of its contractions, so that the waits for
// the next one run out: the kernel raises MOE_FLAG_BARRIER_TIMEOUT and returns, its
// outputs undefined.  The copies that were issued do arrive, and what lets them
// land keeps its 2 s.  (0, 2000000000) restores the production behaviour.
// wait_ns should be some milliseconds at least.  Process-wide and synchronous (it
// copies to device symbols); not to be changed while launches are in flight.
// Returns MOE_OK, MOE_ERR_INVALID_ARG (slices < 0, wait_ns 0) or MOE_ERR_CUDA.
MOE_API int moe_debug_set_expert_wait(int slices, unsigned long long wait_ns);

}  // extern "C"
