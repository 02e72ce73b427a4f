// Token statistics of bf16 logits.
#include "lse_stats.cuh"
LSE_DEFINE_TOKEN_STATS(lse::kBF16, bf16)
