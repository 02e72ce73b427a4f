// Products of bf16 tokens with matrices held in 4 bits.
#include "lse_linear4.cuh"
namespace lse { cudaError_t launch_linear4_bf16(const LinearArgs& a, int sms, cudaStream_t s) { return launch_linear_tokens<kBF16>(a, sms, s); } }
