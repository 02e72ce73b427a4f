// Products of f32 tokens with matrices held in 4 bits.
#include "lse_linear4.cuh"
namespace lse { cudaError_t launch_linear4_f32(const LinearArgs& a, int sms, cudaStream_t s) { return launch_linear_tokens<kF32>(a, sms, s); } }
