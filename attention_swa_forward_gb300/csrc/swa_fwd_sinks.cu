// swa_fwd_sinks.cu — swa_fwd.cuh with sinks.
//
// A query tile's list of key tiles begins with those that hold sinks; where they
// touch the window's run the two are one.  A key is visible if its column is in
// the window or below the sinks, one more compare on tiles that are not visible as
// a whole.  Bound as without sinks, by the hand-offs between the softmax and the
// tensor pipe: BNSD 1x16x32768x128, 4 key/value heads, window 4096, 4 sinks, 885 us
// (tensor pipe 53 % active), and the step 3.52 ms, 3.33 without sinks.  A kernel of
// its own, because the tests on sinks in the plain one cost a step without any 1.5 %
// (1x32x32768x128 under 4096: 6.76 ms instead of 6.67).
#include "swa_fwd.cuh"

namespace swa {

template cudaError_t launch_forward<true, kSmallTable>(
    const FwdArgs&, const SeqTable<kSmallTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
template cudaError_t launch_forward<true, kLargeTable>(
    const FwdArgs&, const SeqTable<kLargeTable>&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);

}  // namespace swa
