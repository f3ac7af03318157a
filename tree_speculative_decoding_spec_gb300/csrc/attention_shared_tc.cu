// Tensor-core items of the shared-prefix and scored tree attention: bf16 runs on the CUDA-core
// items until these exist.
#include "attention_shared.cuh"

namespace spec {
namespace shr {

bool attn_shared_tc_supported(int) { return false; }
spec_status attn_shared_tc_run(const Params&, int, cudaStream_t) { return SPEC_OK; }

}  // namespace shr
}  // namespace spec
