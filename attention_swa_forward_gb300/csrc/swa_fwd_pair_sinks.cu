// swa_fwd_pair_sinks.cu — swa_fwd_pair.cuh with sinks.
#include "swa_fwd_pair.cuh"

namespace swa {

template cudaError_t launch_forward_pair<true, kSmallTable>(
    const FwdArgs&, const SeqTable<kSmallTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
template cudaError_t launch_forward_pair<true, kLargeTable>(
    const FwdArgs&, const SeqTable<kLargeTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);

}  // namespace swa
