// swa_paged_unpack.cu — the keys of an 8-bit cache that the row tiles of a call
// see, as 16-bit pages in the workspace, with a block table of their own
// (swa_paged_tile.cuh then runs on those).
//
// Each 128-key tile of the chunk's list (the sinks' tiles, then the window's) is
// a page of 128 slots, [N_kv][128][D]; values are exact, rows that no query of
// the chunk sees and those of a page that is not to be followed are zeros.  A CTA
// takes a page and a head.  Bound by HBM and L2: it reads a byte per value and
// writes two, which the attention then reads once per row tile.  A chunk of 1024
// tokens behind 15360 keys, 32 / 8 heads of 128: 226 us in all, 205 over a 16-bit
// cache.
//
// (Converting in the attention kernel, by four more warps, took that chunk 536 us
// at best.  A tile's 128 x 256 values take 3000 instructions, which share the
// schedulers and the instruction cache with the softmax, and every row tile
// converts them again.)
#include "swa_paged.h"
#include "swa_device.cuh"
#include "swa_paged_mask.cuh"

namespace swa {
namespace {

constexpr int kThreads = 256;

template <bool F16, int CAP>
__global__ void __launch_bounds__(kThreads)
    swa_paged_unpack_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedTable<CAP> tab,
                            const __grid_constant__ UnpackArgs u) {
  __shared__ int64_t s_k[8], s_v[8], s_e[8];  // of the tile's groups of 16 keys (head 0); < 0: zeros
  __shared__ int s_bad;
  const PagedGeom& g = a.g;
  const int tid = threadIdx.x, hk = blockIdx.y;
  griddep_wait();
  griddep_launch_dependents();
  if (a.clear_err && blockIdx.x == 0 && hk == 0 && tid == 0) *a.err = 0;
  if (tid == 0) s_bad = 0;
  int lo = 0, hi = tab.count - 1;  // the page's sequence: item_begin counts pages here
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.d[mid].item_begin <= static_cast<int>(blockIdx.x)) lo = mid; else hi = mid - 1;
  }
  const PagedDesc& d = tab.d[lo];
  const int unit = static_cast<int>(blockIdx.x) - d.item_begin;
  const int raw = in_bounds(d.b, 1, g.n_lens, a.err) ? g.kv_lens[d.b] : 0;
  const int kv_len = raw < 0 || raw > g.kv_limit ? 0 : raw;  // (the attention reports a bad one)
  const PagedKeys keys = paged_keys<true>(a, kv_len, d.q_len, 0, d.q_len);
  const PagedUnits units = paged_units<true>(keys, 7);
  int32_t* status = a.page_err + u.status_base + blockIdx.x;
  if (unit >= units.total) {
    if (hk == 0 && tid == 0) *status = 0;
    return;
  }
  const int j0 = units.at(unit) * kPagedTileStep;
  auto seen = [&](int j) { return (j >= keys.lo || j < keys.sinks) && j <= keys.hi; };
  __syncthreads();
  if (tid < 8) {
    const int j = j0 + tid * 16;
    int64_t k = -1, v = -1, e = 0;
    if (j < keys.sinks || (j <= keys.hi && j + 15 >= keys.lo)) {  // some key of it is seen
      const int entry = j / g.page_size, slot = j - entry * g.page_size;
      const int64_t at = d.b * g.table_stride + entry;
      const int page = in_bounds(at, 1, g.n_table, a.err) ? g.table[at] : -1;
      if (page >= 0 && page < g.num_pages) {
        k = page * g.k_page + slot * g.k_slot;
        v = page * g.v_page + slot * g.v_slot;
        e = page * a.ex.page + slot;
      } else {
        s_bad = kPageErrEntry;
      }
    }
    s_k[tid] = k;
    s_v[tid] = v;
    s_e[tid] = e;
  }
  __syncthreads();
  if (hk == 0 && tid == 0) {
    *status = s_bad;
    // (inside the scratch by the host's count of pages)
    u.table[d.b * u.table_stride + j0 / kPagedTileStep] = blockIdx.x;
  }

  // a thread: 16 codes of a row, of K and V, four rows in flight
  const int c = (tid & (u.lanes - 1)) * 16, step = kThreads >> u.lane_shift;
  if (c >= g.D) return;
  const int64_t head = static_cast<int64_t>(blockIdx.x) * g.N_kv + hk;
  uint16_t* dst[2] = {static_cast<uint16_t*>(u.k) + head * kPagedTileStep * g.D + c,
                      static_cast<uint16_t*>(u.v) + head * kPagedTileStep * g.D + c};
  constexpr int kBatch = 2;
  for (int r0 = tid >> u.lane_shift; r0 < kPagedTileStep; r0 += kBatch * step) {
    uint4 in[kBatch][2];
    int e[kBatch][2];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int r = r0 + y * step;
      const bool ok = r < kPagedTileStep && s_k[(r >> 4) & 7] >= 0 && seen(j0 + r);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        in[y][x] = make_uint4(0u, 0u, 0u, 0u);
        e[y][x] = 0;
        if (!ok) continue;
        const int64_t at = (x ? s_v : s_k)[r >> 4] + (r & 15) * (x ? g.v_slot : g.k_slot) +
                           hk * (x ? g.v_head : g.k_head) + c;
        const int64_t extent = x ? g.n_v : g.n_k;
        const uint8_t* p = static_cast<const uint8_t*>(x ? a.v_pages : a.k_pages) + at;
        if (a.ex.wide) {
          if (in_bounds(at, 16, extent, a.err)) in[y][x] = __ldcs(reinterpret_cast<const uint4*>(p));
        } else {  // rows start on 8 bytes, and the last 16 codes may be 8
          if (in_bounds(at, 8, extent, a.err)) *reinterpret_cast<uint2*>(&in[y][x].x) = __ldcs(reinterpret_cast<const uint2*>(p));
          if (c + 8 < g.D && in_bounds(at + 8, 8, extent, a.err))
            *reinterpret_cast<uint2*>(&in[y][x].z) = __ldcs(reinterpret_cast<const uint2*>(p + 8));
        }
        const int64_t ex = s_e[r >> 4] + (r & 15) + static_cast<int64_t>(hk) * g.page_size;
        if (in_bounds(ex, 1, a.ex.n, a.err)) e[y][x] = (x ? a.ex.v : a.ex.k)[ex];
      }
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int r = r0 + y * step;
      if (r >= kPagedTileStep) continue;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t f = exp_factor<F16>(e[y][x]) * 0x10001u;
        const uint2 a0 = values4<F16>(in[y][x].x, f), a1 = values4<F16>(in[y][x].y, f);
        const uint2 a2 = values4<F16>(in[y][x].z, f), a3 = values4<F16>(in[y][x].w, f);
        uint16_t* p = dst[x] + r * g.D;
        *reinterpret_cast<uint4*>(p) = make_uint4(a0.x, a0.y, a1.x, a1.y);
        if (c + 8 < g.D) *reinterpret_cast<uint4*>(p + 8) = make_uint4(a2.x, a2.y, a3.x, a3.y);
      }
    }
  }
}

}  // namespace

template <int CAP>
cudaError_t launch_paged_unpack(const PagedArgs& a, const PagedTable<CAP>& tab, const UnpackArgs& u, int pages,
                                cudaStream_t stream) {
  if (pages == 0) return cudaSuccess;
  const dim3 grid(pages, a.g.N_kv);
  return a.f16 ? launch_pdl(swa_paged_unpack_kernel<true, CAP>, grid, dim3(kThreads), 0, stream, a, tab, u)
               : launch_pdl(swa_paged_unpack_kernel<false, CAP>, grid, dim3(kThreads), 0, stream, a, tab, u);
}
template cudaError_t launch_paged_unpack<kPagedSmallTable>(const PagedArgs&, const PagedTable<kPagedSmallTable>&,
                                                           const UnpackArgs&, int, cudaStream_t);
template cudaError_t launch_paged_unpack<kPagedLargeTable>(const PagedArgs&, const PagedTable<kPagedLargeTable>&,
                                                           const UnpackArgs&, int, cudaStream_t);

}  // namespace swa
