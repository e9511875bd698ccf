// seed_scan_pass_f16.cu -- the chunked kernels of the dense scan for __half activations
// (seed_scan_prep.cuh, seed_scan_pass.cuh, seed_scan_back.cuh; one file per type, so that they compile in
// parallel).
#include "seed_scan_back.cuh"
#include "seed_scan_prep.cuh"

namespace seed {

template int launch_scan_prep_as<__half>(const ScanParams& p, int form, cudaStream_t st);
template int launch_scan_pass_as<__half>(const ScanParams& p, int form, cudaStream_t st);
template int launch_scan_back_as<__half>(const ScanParams& p, int form, cudaStream_t st);

}  // namespace seed
