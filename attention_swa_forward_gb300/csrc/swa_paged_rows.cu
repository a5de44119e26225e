// swa_paged_rows.cu — attention of a few query rows under the window, 16-bit cache (swa_paged_rows.cuh).
#include "swa_paged_rows.cuh"

namespace swa {

template cudaError_t launch_paged_rows<PagedKind::kPlain, kPagedSmallTable>(const PagedArgs&,
                                                                         const PagedTable<kPagedSmallTable>&,
                                                                         cudaStream_t);
template cudaError_t launch_paged_rows<PagedKind::kPlain, kPagedLargeTable>(const PagedArgs&,
                                                                         const PagedTable<kPagedLargeTable>&,
                                                                         cudaStream_t);

}  // namespace swa
