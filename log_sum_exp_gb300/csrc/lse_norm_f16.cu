// The end of a block, rows of f16.
#include "lse_norm.cuh"
LSE_DEFINE_NORM(lse::kF16, f16)
