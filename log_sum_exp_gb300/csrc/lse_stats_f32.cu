// Token statistics of f32 logits.
#include "lse_stats.cuh"
LSE_DEFINE_TOKEN_STATS(lse::kF32, f32)
