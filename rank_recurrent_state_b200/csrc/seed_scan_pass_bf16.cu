// seed_scan_pass_bf16.cu -- the chunked pass of the dense scan for __nv_bfloat16 activations
// (kernel in seed_scan_pass.cuh; one file per type, so that they compile in parallel).
#include "seed_scan_pass.cuh"

namespace seed {

template int launch_scan_pass_as<__nv_bfloat16>(const ScanParams& p, int form, cudaStream_t st);

}  // namespace seed
