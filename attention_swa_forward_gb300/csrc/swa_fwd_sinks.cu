// swa_fwd_sinks.cu — swa_fwd.cuh with sinks.
#include "swa_fwd.cuh"

namespace swa {

template cudaError_t launch_forward<true, kSmallTable>(
    const FwdArgs&, const SeqTable<kSmallTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
template cudaError_t launch_forward<true, kLargeTable>(
    const FwdArgs&, const SeqTable<kLargeTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);

}  // namespace swa
