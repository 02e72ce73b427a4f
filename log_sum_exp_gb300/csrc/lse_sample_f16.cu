// Drawing tokens from f16 logits.
#include "lse_sample.cuh"
namespace lse { cudaError_t launch_sample_f16(const SampleArgs& a, int sms, cudaStream_t s) { return launch_sample<kF16>(a, sms, s); } }
