// swa_paged_rows_e4m3.cu — attention of a few query rows over the 8-bit cache (swa_paged_rows.cuh).
#include "swa_paged_rows.cuh"

namespace swa {

template cudaError_t launch_paged_rows<PagedKind::kE4m3, kPagedSmallTable>(const PagedArgs&,
                                                                         const PagedTable<kPagedSmallTable>&,
                                                                         cudaStream_t);
template cudaError_t launch_paged_rows<PagedKind::kE4m3, kPagedLargeTable>(const PagedArgs&,
                                                                         const PagedTable<kPagedLargeTable>&,
                                                                         cudaStream_t);

}  // namespace swa
