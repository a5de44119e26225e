// swa_fwd.cu — swa_fwd.cuh without sinks.
#include "swa_fwd.cuh"

namespace swa {

template cudaError_t launch_forward<false, kSmallTable>(
    const FwdArgs&, const SeqTable<kSmallTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
template cudaError_t launch_forward<false, kLargeTable>(
    const FwdArgs&, const SeqTable<kLargeTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);

}  // namespace swa
