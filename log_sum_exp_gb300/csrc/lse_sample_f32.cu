// Drawing tokens from f32 logits.
#include "lse_sample.cuh"
namespace lse { cudaError_t launch_sample_f32(const SampleArgs& a, int sms, cudaStream_t s) { return launch_sample<kF32>(a, sms, s); } }
