// The end of a block, rows of bf16.
#include "lse_norm.cuh"
LSE_DEFINE_NORM(lse::kBF16, bf16)
