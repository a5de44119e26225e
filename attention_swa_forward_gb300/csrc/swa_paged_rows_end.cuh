// swa_paged_rows_end.cuh — what the few-row kernels share: the product
// instruction, and the join of a CTA's four warps and of a cluster's CTAs.
#pragma once
#include "swa_paged.h"
#include "swa_device.cuh"
#include "swa_paged_mask.cuh"

#include <type_traits>
#include <utility>

namespace swa {
namespace {

constexpr int kRowsWarps = kRowsStep / 16;
constexpr int kRowsThreads = kRowsWarps * 32;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // rescale only when the maximum grows by more than 2^8

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The CTAs of a cluster: barrier over all their threads (every thread arrives
// and waits; orders shared-memory accesses across the cluster), this CTA's
// rank, and reads of a peer's shared memory.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_peer2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// Shared memory of the end, in floats: the warps' O, [warp][row][DP + 4], and
// behind it the CTA's own joined rows and their maxima and sums, for the cluster.
template <int DP>
struct RowsEnd {
  static constexpr int kOPitch = DP + 4;
  static constexpr int kJoinAt = kRowsWarps * kRowsTile * kOPitch;
  static constexpr int kMlAt = kJoinAt + kRowsTile * DP;
  static constexpr int kBytes = 4 * (kMlAt + 2 * kRowsTile);
};

// Page status, and the item's rows from the warps' O (in `so`), maxima and sums
// (ml): to the results, to the workspace, or through the cluster.
template <int DP, bool F16, bool CL>
__device__ __forceinline__ void rows_end(const PagedBase& a, const PagedItem& w, int split, int64_t item, int tok0,
                                         int n_rows, bool direct, int bad, float* so, float (*ml)[kRowsTile][2]) {
  using Layout = RowsEnd<DP>;
  const PagedGeom& g = a.g;
  const int any_len = __syncthreads_or(bad == kPageErrLength), any_entry = __syncthreads_or(bad == kPageErrEntry);
  if (threadIdx.x == 0)
    a.page_err[item * a.splits + split] = any_len ? kPageErrLength : (any_entry ? kPageErrEntry : 0);

  // four columns of row r, from their maximum, sum and unnormalised values
  auto finish = [&](int r, int col, float M, float L, const float (&acc)[4]) {
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
    const int i = row_token(r, a.gs_magic), h = w.vh * a.gs + (r - i * a.gs);
    const int64_t row = static_cast<int64_t>(w.q_start + tok0 + i) * g.N + h;
    if (col < g.D && in_bounds(row * g.D + col, 4, a.n_out, a.err))
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * g.D + col) =
          make_uint2(pack2<F16>(acc[0] * inv, acc[1] * inv), pack2<F16>(acc[2] * inv, acc[3] * inv));
    if (col == 0 && in_bounds(row, 1, a.n_stats, a.err)) {
      if (a.smax) a.smax[row] = M == -INFINITY ? -INFINITY : M * kLn2;
      if (a.ssum) a.ssum[row] = L;
    }
  };
  // join the four warps: thread = 4 columns of a row
  constexpr int kCols4 = DP / 4;
  for (int x = threadIdx.x; x < n_rows * kCols4; x += kRowsThreads) {
    const int r = x / kCols4, col = (x % kCols4) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int v = 0; v < kRowsWarps; ++v) M = fmaxf(M, ml[v][r][0]);
    const float ms = M == -INFINITY ? 0.f : M;
    float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kRowsWarps; ++v) {
      const float f = ex2_approx(ml[v][r][0] - ms);
      L += ml[v][r][1] * f;
      const float4 ov = *reinterpret_cast<const float4*>(so + (v * kRowsTile + r) * Layout::kOPitch + col);
      acc[0] += ov.x * f;
      acc[1] += ov.y * f;
      acc[2] += ov.z * f;
      acc[3] += ov.w * f;
    }
    if (CL) {
      *reinterpret_cast<float4*>(so + Layout::kJoinAt + r * DP + col) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (col == 0) *reinterpret_cast<float2*>(so + Layout::kMlAt + 2 * r) = make_float2(M, L);
    } else if (!direct) {
      const int64_t pr = (item * a.splits + split) * a.rows_pad + r;
      *reinterpret_cast<float4*>(a.part_o + pr * DP + col) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (col == 0) a.part_ml[pr] = make_float2(M, L);
    } else {
      finish(r, col, M, L, acc);
    }
  }
  if constexpr (CL) {
    // row r of the item is finished by the CTA of rank r mod splits
    cluster_sync();
    const uint32_t rank = cluster_rank(), mine = smem_u32(so + Layout::kJoinAt), mine_ml = smem_u32(so + Layout::kMlAt);
    for (int x = threadIdx.x;; x += kRowsThreads) {
      const int r = static_cast<int>(rank) + x / kCols4 * a.splits, col = (x % kCols4) * 4;
      if (r >= n_rows) break;
      float M = -INFINITY;
#pragma unroll 8
      for (int v = 0; v < a.splits; ++v) M = fmaxf(M, ld_peer2(peer_smem(mine_ml + 8 * r, v)).x);
      const float ms = M == -INFINITY ? 0.f : M;
      float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int v = 0; v < a.splits; ++v) {
        const float2 ml = ld_peer2(peer_smem(mine_ml + 8 * r, v));
        const float4 ov = ld_peer4(peer_smem(mine + 4 * (r * DP + col), v));
        const float f = ex2_approx(ml.x - ms);
        L += ml.y * f;
        acc[0] += ov.x * f;
        acc[1] += ov.y * f;
        acc[2] += ov.z * f;
        acc[3] += ov.w * f;
      }
      finish(r, col, M, L, acc);
    }
    cluster_sync();  // a CTA's shared memory stays until its peers have read it
  }
}

// The launch; CL: the splits of an item (grid.y) are a cluster.
template <bool CL, typename... Params, typename... Args>
cudaError_t launch_rows_grid(void (*kernel)(Params...), dim3 grid, size_t smem, cudaStream_t stream, Args&&... args) {
  if constexpr (!CL) {
    return launch_pdl(kernel, grid, dim3(kRowsThreads), smem, stream, std::forward<Args>(args)...);
  } else {
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = grid.y;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  }
}

}  // namespace
}  // namespace swa
