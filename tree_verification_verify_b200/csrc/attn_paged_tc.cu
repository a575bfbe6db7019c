#include "attn_paged.cuh"
namespace tv {
bool attn_paged_tc_supported(const tv_attn_paged_args*) { return false; }
cudaError_t launch_attn_paged_tc(const PagedAttnParams&, int, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace tv
