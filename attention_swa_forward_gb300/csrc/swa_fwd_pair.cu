// swa_fwd_pair.cu — swa_fwd_pair.cuh without sinks.
#include "swa_fwd_pair.cuh"

namespace swa {

template cudaError_t launch_forward_pair<false, kSmallTable>(
    const FwdArgs&, const SeqTable<kSmallTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
template cudaError_t launch_forward_pair<false, kLargeTable>(
    const FwdArgs&, const SeqTable<kLargeTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);

}  // namespace swa
