// swa_paged_rows_masks.cu — attention of a few query rows with sinks or a tree, 16-bit cache (swa_paged_rows.cuh).
#include "swa_paged_rows.cuh"

namespace swa {

template cudaError_t launch_paged_rows<PagedKind::kMasks, kPagedSmallTable>(const PagedArgs&,
                                                                         const PagedTable<kPagedSmallTable>&,
                                                                         cudaStream_t);
template cudaError_t launch_paged_rows<PagedKind::kMasks, kPagedLargeTable>(const PagedArgs&,
                                                                         const PagedTable<kPagedLargeTable>&,
                                                                         cudaStream_t);

}  // namespace swa
