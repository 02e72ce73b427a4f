// Products of f16 tokens with matrices held in 4 bits.
#include "lse_linear4.cuh"
namespace lse { cudaError_t launch_linear4_f16(const LinearArgs& a, int sms, cudaStream_t s) { return launch_linear_tokens<kF16>(a, sms, s); } }
