// swa_bwd_dq_sinks.cu — swa_bwd_dq.cuh with sinks.
//
// The key tiles of a query tile as in swa_fwd_sinks.cu.  BNSD 1x16x32768x128, 4
// key/value heads, window 4096, 4 sinks: 996 us (tensor pipe 71 % active).
#include "swa_bwd_dq.cuh"

namespace swa {

template cudaError_t launch_backward_dq<true, kSmallTable>(
    const BwdArgs&, const SeqTable<kSmallTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
    cudaStream_t);
template cudaError_t launch_backward_dq<true, kLargeTable>(
    const BwdArgs&, const SeqTable<kLargeTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
    cudaStream_t);

}  // namespace swa
