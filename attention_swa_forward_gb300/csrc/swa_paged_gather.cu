// swa_paged_gather.cu — the keys and values of a chunk read back from the paged
// cache (include/swa.h, swa_paged_gather): the copy that swa_paged_append made,
// in the other direction.
//
// A row of an 8-bit cache is code 2^e, exact in the 16-bit types
// (swa_paged_mask.cuh).  A CTA takes up to 16 tokens, all heads of K and V; its
// first threads look up their pages, then each thread moves 16 bytes of a row at a
// time, four rows in flight.  Bound by HBM: every code is read once and every value
// written once.  131072 tokens of 8 + 8 heads of 128, 807 MB: 125 us, 0.95 of the
// copy rate; 19205 tokens of 96, 74 MB: 18.2, 0.60 (with up to 32 tokens per CTA 127
// and 24).
#include "swa_paged.h"
#include "swa_device.cuh"
#include "swa_paged_mask.cuh"

namespace swa {
namespace {

template <bool F16, bool Q8, int CAP>
__global__ void __launch_bounds__(kGatherThreads)
    swa_paged_gather_kernel(const __grid_constant__ GatherArgs a, const __grid_constant__ PagedTable<CAP> tab) {
  __shared__ int64_t s_src[kGatherMostTok][2], s_ex[kGatherMostTok];  // of (token, head 0); < 0: a row of zeros
  const PagedGeom& g = a.pg;
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  if (a.clear_err && blockIdx.x == 0 && tid == 0) *a.err = 0;
  const int64_t t0 = a.tok_begin + static_cast<int64_t>(blockIdx.x) * a.tok;
  const int n_tok = static_cast<int>(a.rows - t0 < a.tok ? a.rows - t0 : a.tok);
  if (tid < n_tok) {
    const int t = static_cast<int>(t0) + tid;
    int b, i, q_len;  // the token's sequence and place in its chunk
    if (tab.d[0].b < 0) {
      q_len = tab.d[0].q_len;
      b = t / q_len;
      i = t - b * q_len;
    } else {
      int lo = 0, hi = tab.count - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.d[mid].q_start <= t) lo = mid; else hi = mid - 1;
      }
      b = tab.d[lo].b;
      q_len = tab.d[lo].q_len;
      i = t - tab.d[lo].q_start;
    }
    int bad = 0;
    int len = in_bounds(b, 1, g.n_lens, a.err) ? g.kv_lens[b] : 0;
    if (len < 0 || len > g.kv_limit) {
      bad = kPageErrLength;
      len = 0;
    }
    const int pos = len - q_len + i;
    int64_t k = -1, v = -1, ex = 0;
    if (pos >= 0) {
      const int entry = pos / g.page_size, slot = pos - entry * g.page_size;
      const int64_t e = b * g.table_stride + entry;
      const int page = in_bounds(e, 1, g.n_table, a.err) ? g.table[e] : -1;
      if (page >= 0 && page < g.num_pages) {
        k = page * g.k_page + slot * g.k_slot;
        v = page * g.v_page + slot * g.v_slot;
        ex = page * a.ex.page + slot;
      } else {
        bad = kPageErrEntry;
      }
    }
    s_src[tid][0] = k;
    s_src[tid][1] = v;
    s_ex[tid] = ex;
    a.page_err[t] = bad;
  }
  __syncthreads();

  constexpr int kCodes = Q8 ? 16 : 8;  // elements that a thread moves at a time
  constexpr int kBatch = 4;
  const int c = (tid & (a.lanes - 1)) * kCodes, row_lanes = kGatherThreads >> a.lane_shift;
  const int n_rows = n_tok * 2 * g.N_kv;
  // row r: token r / (2 N_kv), then K's heads, then V's
  struct Place {
    int x;
    int64_t src, ex, dst;
  };
  auto locate = [&](int r, Place& w) {
    const int t = r / (2 * g.N_kv), y = r - t * 2 * g.N_kv;
    w.x = y >= g.N_kv ? 1 : 0;
    const int h = y - w.x * g.N_kv;
    const int64_t at = s_src[t][w.x];
    w.src = at < 0 ? -1 : at + h * (w.x ? g.v_head : g.k_head) + c;
    w.ex = s_ex[t] + static_cast<int64_t>(h) * g.page_size;
    w.dst = (t0 + t) * a.dst_r[w.x] + h * a.dst_h[w.x] + c;
  };
  if (c >= g.D) return;
  for (int r0 = tid >> a.lane_shift; r0 < n_rows; r0 += kBatch * row_lanes) {
    uint4 in[kBatch];
    int e[kBatch];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      in[y] = make_uint4(0u, 0u, 0u, 0u);
      e[y] = 0;
      Place w;
      if (r0 + y * row_lanes >= n_rows) continue;
      locate(r0 + y * row_lanes, w);
      if (w.src < 0) continue;
      const int64_t extent = w.x ? g.n_v : g.n_k;
      if constexpr (Q8) {
        const uint8_t* p = static_cast<const uint8_t*>(a.src[w.x]) + w.src;
        if (a.ex.wide) {
          if (in_bounds(w.src, 16, extent, a.err)) in[y] = __ldcs(reinterpret_cast<const uint4*>(p));
        } else {  // rows start on 8 bytes, and the last 16 codes may be 8
          if (in_bounds(w.src, 8, extent, a.err)) *reinterpret_cast<uint2*>(&in[y].x) = __ldcs(reinterpret_cast<const uint2*>(p));
          if (c + 8 < g.D && in_bounds(w.src + 8, 8, extent, a.err))
            *reinterpret_cast<uint2*>(&in[y].z) = __ldcs(reinterpret_cast<const uint2*>(p + 8));
        }
        if (in_bounds(w.ex, 1, a.ex.n, a.err)) e[y] = (w.x ? a.ex.v : a.ex.k)[w.ex];
      } else if (in_bounds(w.src, 8, extent, a.err)) {
        in[y] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.src[w.x]) + w.src));
      }
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      if (r0 + y * row_lanes >= n_rows) continue;
      Place w;
      locate(r0 + y * row_lanes, w);
      uint16_t* p = static_cast<uint16_t*>(a.dst[w.x]) + w.dst;
      if constexpr (Q8) {
        const uint32_t f = exp_factor<F16>(e[y]) * 0x10001u;
        const uint2 a0 = values4<F16>(in[y].x, f), a1 = values4<F16>(in[y].y, f);
        const uint2 a2 = values4<F16>(in[y].z, f), a3 = values4<F16>(in[y].w, f);
        const uint4 lo = make_uint4(a0.x, a0.y, a1.x, a1.y), hi = make_uint4(a2.x, a2.y, a3.x, a3.y);
        if (in_bounds(w.dst, 8, a.n_dst[w.x], a.err)) __stcs(reinterpret_cast<uint4*>(p), lo);
        if (c + 8 < g.D && in_bounds(w.dst + 8, 8, a.n_dst[w.x], a.err)) __stcs(reinterpret_cast<uint4*>(p + 8), hi);
      } else {
        if (in_bounds(w.dst, 8, a.n_dst[w.x], a.err)) __stcs(reinterpret_cast<uint4*>(p), in[y]);
      }
    }
  }
}

}  // namespace

template <int CAP>
cudaError_t launch_gather(const GatherArgs& a, const PagedTable<CAP>& tab, bool f16, int n_ctas, cudaStream_t stream) {
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(n_ctas), dim3(kGatherThreads), 0, stream, a, tab); };
  if (a.ex.k) return f16 ? go(swa_paged_gather_kernel<true, true, CAP>) : go(swa_paged_gather_kernel<false, true, CAP>);
  return go(swa_paged_gather_kernel<false, false, CAP>);  // (copies bits)
}
template cudaError_t launch_gather<kPagedSmallTable>(const GatherArgs&, const PagedTable<kPagedSmallTable>&, bool, int,
                                                     cudaStream_t);
template cudaError_t launch_gather<kPagedLargeTable>(const GatherArgs&, const PagedTable<kPagedLargeTable>&, bool, int,
                                                     cudaStream_t);

}  // namespace swa
