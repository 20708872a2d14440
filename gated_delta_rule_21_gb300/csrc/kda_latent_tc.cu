#include "kda_latent.cuh"
namespace kda {
namespace latent {
bool prompt_tc_ok(const Prompt &) { return false; }
cudaError_t launch_prompt_tc(const Prompt &, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t launch_prompt_bwd_tc(const Prompt &, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace latent
}  // namespace kda
