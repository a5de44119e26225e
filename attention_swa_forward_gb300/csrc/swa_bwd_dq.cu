// swa_bwd_dq.cu — swa_bwd_dq.cuh without sinks.
#include "swa_bwd_dq.cuh"

namespace swa {

template cudaError_t launch_backward_dq<false, kSmallTable>(
    const BwdArgs&, const SeqTable<kSmallTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
    cudaStream_t);
template cudaError_t launch_backward_dq<false, kLargeTable>(
    const BwdArgs&, const SeqTable<kLargeTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
    cudaStream_t);

}  // namespace swa
