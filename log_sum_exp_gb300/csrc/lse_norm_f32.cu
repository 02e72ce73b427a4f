// The end of a block, rows of f32.
#include "lse_norm.cuh"
LSE_DEFINE_NORM(lse::kF32, f32)
