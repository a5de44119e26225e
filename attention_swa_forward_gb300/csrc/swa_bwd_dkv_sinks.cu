// swa_bwd_dkv_sinks.cu — swa_bwd_dkv.cuh with sinks.
//
// A key tile with sinks walks every query tile behind it.  Where that is more than
// any other CTA has, it is cut into pieces (swa_api.cpp), whose fp32 sums
// swa_bwd_join.cu adds in their order: no atomics, the same bits from run to run.
// BNSD 1x16x32768x128, 4 key/value heads, window 4096, 4 sinks: 1533 us (tensor
// pipe 64 % active) and 10 us for the join.
#include "swa_bwd_dkv.cuh"

namespace swa {

template cudaError_t launch_backward_dkv<true, kSmallTable>(
    const BwdArgs&, const SeqTable<kSmallTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
    cudaStream_t);
template cudaError_t launch_backward_dkv<true, kLargeTable>(
    const BwdArgs&, const SeqTable<kLargeTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
    cudaStream_t);

}  // namespace swa
