// swa_paged_tile.cu — attention of a chunk under the window, 16-bit cache (swa_paged_tile.cuh).
#include "swa_paged_tile.cuh"

namespace swa {

template cudaError_t launch_paged_tile<PagedKind::kPlain, kPagedSmallTable>(const PagedArgs&,
                                                                         const PagedTable<kPagedSmallTable>&,
                                                                         const CUtensorMap&, const CUtensorMap&,
                                                                         const CUtensorMap&, cudaStream_t);
template cudaError_t launch_paged_tile<PagedKind::kPlain, kPagedLargeTable>(const PagedArgs&,
                                                                         const PagedTable<kPagedLargeTable>&,
                                                                         const CUtensorMap&, const CUtensorMap&,
                                                                         const CUtensorMap&, cudaStream_t);

}  // namespace swa
