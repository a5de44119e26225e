// swa_paged_join.cu — the pass that joins the results of keys split over
// several CTAs (swa_paged_rows.cuh, swa_paged_tile.cuh).
#include "swa_paged.h"
#include "swa_device.cuh"

namespace swa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// Join the splits of a row tile: WPR warps per row over its splits (each reads
// a partial row with one load per lane), then over their sums in shared
// memory; one warp up to 8 splits, eight past that.  Reads the active partial
// rows once, a few microseconds behind the kernel that wrote them, launched so
// that its prologue overlaps that tail.  (One warp per row took 30 us for the
// 152 splits that one 131072-token sequence had.)
// Where a warp per row gives every SM half a CTA, up to 32 splits are joined by it in
// the eight warps' order, with the same bits (FOLD).  61 tokens of 32 / 8 heads over
// 32768 keys, 2048 rows of 9 splits: 38.4 us instead of 43.2; 32 tokens, 1024 rows of 19: 36.3
// instead of 37.0; over 16384 keys 20.5 instead of 21.4.
constexpr int kJoinWarps = 8;
constexpr int kFoldMost = 32;
template <int DP, bool F16, int WPR, bool FOLD, int CAP>
__global__ void __launch_bounds__(kJoinWarps * 32)
    swa_paged_join_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedTable<CAP> tab,
                          const int step_keys) {
  constexpr int kPer = DP / 32;  // columns of a lane: 4 or 2
  __shared__ float s_acc[WPR][DP], s_l[WPR], s_m[WPR];
  const PagedGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedItem w = resolve_paged(tab, a.groups, a.whole + static_cast<int>(blockIdx.x));
  const int r = blockIdx.y * (kJoinWarps / WPR) + warp / WPR, part = warp % WPR;
  const int tok0 = w.tile * a.tok;
  const int n_tok = min(a.tok, w.q_len - tok0);
  // (the lengths come from grids before the one that wrote the partial rows:
  // there is nothing to wait for, and L2 has them)
  int kv_len = in_bounds(w.b, 1, g.n_lens, a.err) ? __ldcg(g.kv_lens + w.b) : 0;
  if (kv_len < 0 || kv_len > g.kv_limit) kv_len = 0;
  int st0, st1, active;
  const PagedKeys keys = paged_keys<true>(a, kv_len, w.q_len, tok0, n_tok);
  const int steps = step_keys == kRowsStep ? (paged_units<true>(keys, 4).total + kRowsStep / 16 - 1) / (kRowsStep / 16)
                                           : paged_units<true>(keys, 7).total;
  paged_split(steps, a.par, a.cap, a.least, 0, &st0, &st1, &active);
  griddep_wait();
  griddep_launch_dependents();
  if (r >= n_tok * a.gs) return;  // (with WPR > 1 a CTA is one row: all of it returns)
  static_assert(WPR == 1 || WPR == kJoinWarps, "a CTA is one row or one row per warp");
  if (active <= 1) return;  // written by the CTA that had the keys
  const int64_t item = a.item_base + static_cast<int64_t>(blockIdx.x);  // among the split ones
  const int64_t p0 = item * a.splits * a.rows_pad + r;
  float M = -INFINITY, L = 0.f, acc[kPer];
#pragma unroll
  for (int y = 0; y < kPer; ++y) acc[y] = 0.f;
  if constexpr (FOLD) {
    // split x belongs to part x mod 8: lane x has its maximum, sum and factor
    constexpr int kParts = kJoinWarps;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < active) ml = a.part_ml[p0 + static_cast<int64_t>(lane) * a.rows_pad];
    float m = fmaxf(ml.x, __shfl_xor_sync(0xFFFFFFFFu, ml.x, 8));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));  // of the lane's part
    M = m;
#pragma unroll
    for (int x = 4; x >= 1; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, x));
    const float f = ex2_approx(ml.x - (m == -INFINITY ? 0.f : m));
    const float fp = ex2_approx(m - (M == -INFINITY ? 0.f : M));
    float sum[kParts][kPer], l = 0.f;
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
      for (int y = 0; y < kPer; ++y) sum[p][y] = 0.f;
#pragma unroll 1
    for (int x0 = 0; x0 < active; x0 += kParts) {
      float v[kParts][kPer];
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        const float* src = a.part_o + (p0 + static_cast<int64_t>(x0 + p) * a.rows_pad) * DP + lane * kPer;
        if constexpr (kPer == 4)
          *reinterpret_cast<float4*>(v[p]) = x0 + p < active ? *reinterpret_cast<const float4*>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
        else
          *reinterpret_cast<float2*>(v[p]) = x0 + p < active ? *reinterpret_cast<const float2*>(src) : make_float2(0.f, 0.f);
      }
      // (lanes past the last split hold a sum and a factor of 0)
      l = fmaf(__shfl_sync(0xFFFFFFFFu, ml.y, x0 + lane % kParts), __shfl_sync(0xFFFFFFFFu, f, x0 + lane % kParts), l);
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        const float fx = __shfl_sync(0xFFFFFFFFu, f, x0 + p);
#pragma unroll
        for (int y = 0; y < kPer; ++y) sum[p][y] = fmaf(v[p][y], fx, sum[p][y]);
      }
    }
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const float fx = __shfl_sync(0xFFFFFFFFu, fp, p);
      L = fmaf(__shfl_sync(0xFFFFFFFFu, l, p), fx, L);
#pragma unroll
      for (int y = 0; y < kPer; ++y) acc[y] = fmaf(sum[p][y], fx, acc[y]);
    }
  } else {
    // each warp: its splits' maximum, then their sum relative to it
    for (int x = part + WPR * lane; x < active; x += 32 * WPR)
      M = fmaxf(M, a.part_ml[p0 + static_cast<int64_t>(x) * a.rows_pad].x);
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, x));
    const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll 4
    for (int x = part; x < active; x += WPR) {
      const int64_t p = p0 + static_cast<int64_t>(x) * a.rows_pad;
      const float2 ml = a.part_ml[p];
      const float f = ex2_approx(ml.x - ms);
      L += ml.y * f;
      if constexpr (kPer == 4) {
        const float4 v = *reinterpret_cast<const float4*>(a.part_o + p * DP + lane * 4);
        acc[0] += v.x * f;
        acc[1] += v.y * f;
        acc[2] += v.z * f;
        acc[3] += v.w * f;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(a.part_o + p * DP + lane * 2);
        acc[0] += v.x * f;
        acc[1] += v.y * f;
      }
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int y = 0; y < kPer; ++y) s_acc[warp][lane * kPer + y] = acc[y];
    if (lane == 0) {
      s_l[warp] = L;
      s_m[warp] = M;
    }
    __syncthreads();
    if (warp != 0) return;
    M = s_m[0];
#pragma unroll
    for (int x = 1; x < kJoinWarps; ++x) M = fmaxf(M, s_m[x]);
    const float mt = M == -INFINITY ? 0.f : M;
    L = 0.f;
#pragma unroll
    for (int y = 0; y < kPer; ++y) acc[y] = 0.f;
#pragma unroll
    for (int x = 0; x < kJoinWarps; ++x) {
      const float f = ex2_approx(s_m[x] - mt);
      L += s_l[x] * f;
#pragma unroll
      for (int y = 0; y < kPer; ++y) acc[y] += s_acc[x][lane * kPer + y] * f;
    }
  }
  const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
  const int i = row_token(r, a.gs_magic), h = w.vh * a.gs + (r - i * a.gs);
  const int64_t row = static_cast<int64_t>(w.q_start + tok0 + i) * g.N + h;
  const int col = lane * kPer;
  if (col < g.D && in_bounds(row * g.D + col, kPer, a.n_out, a.err)) {
    uint32_t* d = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * g.D + col);
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(d) =
          make_uint2(pack2<F16>(acc[0] * inv, acc[1] * inv), pack2<F16>(acc[2] * inv, acc[3] * inv));
    else
      *d = pack2<F16>(acc[0] * inv, acc[1] * inv);
  }
  if (lane == 0 && in_bounds(row, 1, a.n_stats, a.err)) {
    if (a.smax) a.smax[row] = M == -INFINITY ? -INFINITY : M * kLn2;
    if (a.ssum) a.ssum[row] = L;
  }
}

template <int DP, bool F16, int CAP>
cudaError_t launch_join_t(const PagedArgs& a, const PagedTable<CAP>& tab, int step_keys, cudaStream_t stream) {
  const int rows = a.tok * a.gs, items = tab.n_items - a.whole;
  auto go = [&](auto kernel, int per_cta) {
    return launch_pdl(kernel, dim3(items, (rows + per_cta - 1) / per_cta), dim3(kJoinWarps * 32), 0, stream, a, tab, step_keys);
  };
  if (a.splits <= kJoinWarps) return go(swa_paged_join_kernel<DP, F16, 1, false, CAP>, kJoinWarps);
  if (a.splits <= kFoldMost && static_cast<int64_t>(rows) * items >= kSms * 4)
    return go(swa_paged_join_kernel<DP, F16, 1, true, CAP>, kJoinWarps);
  return go(swa_paged_join_kernel<DP, F16, kJoinWarps, false, CAP>, 1);
}

}  // namespace

template <int CAP>
cudaError_t launch_paged_join(const PagedArgs& a, const PagedTable<CAP>& tab, int step_keys, cudaStream_t stream) {
  if (tab.n_items == 0) return cudaSuccess;
  if (a.g.D <= 64)
    return a.f16 ? launch_join_t<64, true>(a, tab, step_keys, stream)
                 : launch_join_t<64, false>(a, tab, step_keys, stream);
  return a.f16 ? launch_join_t<128, true>(a, tab, step_keys, stream)
               : launch_join_t<128, false>(a, tab, step_keys, stream);
}

template cudaError_t launch_paged_join<kPagedSmallTable>(const PagedArgs&, const PagedTable<kPagedSmallTable>&, int,
                                                         cudaStream_t);
template cudaError_t launch_paged_join<kPagedLargeTable>(const PagedArgs&, const PagedTable<kPagedLargeTable>&, int,
                                                         cudaStream_t);

}  // namespace swa
