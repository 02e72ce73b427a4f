// Token statistics of f16 logits.
#include "lse_stats.cuh"
LSE_DEFINE_TOKEN_STATS(lse::kF16, f16)
