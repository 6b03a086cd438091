// The prompts' kernels with weights of 16 bits: a file of their own, so that the two sets
// compile side by side.
#include "attn_prefill.cuh"

namespace fp8moe {

cudaError_t ready_prefill16(int d, PrefillFit *fit) { return ready_terms<2>(d, fit); }
cudaError_t launch_prefill16(const PrefillArgs &a, int d, int sms, cudaStream_t s) { return launch_terms<2>(a, d, sms, s); }

}  // namespace fp8moe
