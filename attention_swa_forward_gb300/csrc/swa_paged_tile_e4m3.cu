// swa_paged_tile_e4m3.cu — attention of a chunk over the 8-bit cache (swa_paged_tile.cuh).
#include "swa_paged_tile.cuh"

namespace swa {

template cudaError_t launch_paged_tile<PagedKind::kE4m3, kPagedSmallTable>(const PagedArgs&,
                                                                         const PagedTable<kPagedSmallTable>&,
                                                                         const CUtensorMap&, const CUtensorMap&,
                                                                         const CUtensorMap&, cudaStream_t);
template cudaError_t launch_paged_tile<PagedKind::kE4m3, kPagedLargeTable>(const PagedArgs&,
                                                                         const PagedTable<kPagedLargeTable>&,
                                                                         const CUtensorMap&, const CUtensorMap&,
                                                                         const CUtensorMap&, cudaStream_t);

}  // namespace swa
