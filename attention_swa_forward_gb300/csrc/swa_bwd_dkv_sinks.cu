// swa_bwd_dkv_sinks.cu — swa_bwd_dkv.cuh with sinks.
#include "swa_bwd_dkv.cuh"

namespace swa {

template cudaError_t launch_backward_dkv<true, kSmallTable>(
    const BwdArgs&, const SeqTable<kSmallTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
    cudaStream_t);
template cudaError_t launch_backward_dkv<true, kLargeTable>(
    const BwdArgs&, const SeqTable<kLargeTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
    cudaStream_t);

}  // namespace swa
