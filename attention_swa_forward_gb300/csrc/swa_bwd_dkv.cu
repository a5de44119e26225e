// swa_bwd_dkv.cu — swa_bwd_dkv.cuh without sinks.
#include "swa_bwd_dkv.cuh"

namespace swa {

template cudaError_t launch_backward_dkv<false, kSmallTable>(
    const BwdArgs&, const SeqTable<kSmallTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
    cudaStream_t);
template cudaError_t launch_backward_dkv<false, kLargeTable>(
    const BwdArgs&, const SeqTable<kLargeTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
    cudaStream_t);

}  // namespace swa
