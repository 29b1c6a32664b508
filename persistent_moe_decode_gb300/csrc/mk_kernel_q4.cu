// The persistent step kernel's instances over the 4-bit KV cache: the same
// source with Q4 set, a translation unit of its own so that both halves of the
// instances compile at the same time.
#define MK_STEP_Q4_UNIT
#define MK_STEP_Q4 true
#include "mk_kernel.cu"
