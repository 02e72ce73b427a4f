// Drawing tokens from bf16 logits.
#include "lse_sample.cuh"
namespace lse { cudaError_t launch_sample_bf16(const SampleArgs& a, int sms, cudaStream_t s) { return launch_sample<kBF16>(a, sms, s); } }
