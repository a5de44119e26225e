// swa_bwd_join.cu — the sum of the pieces that a key tile with sinks is cut into
// (swa_bwd_dkv.cuh).
#include "swa_device.cuh"

namespace swa {
namespace {

// dK and dV of the key tiles whose steps were cut into pieces: the pieces'
// fp32 rows, summed in their order.  The CTA of piece x takes every pieces-th
// row from x on; a few MB, read once, behind a pass of milliseconds.
constexpr int kJoinThreads = 256;
template <int D, bool F16, int CAP>
__global__ void __launch_bounds__(kJoinThreads)
    swa_bwd_join_kernel(const BwdArgs a, const __grid_constant__ SeqTable<CAP> tab) {
  griddep_wait();
  griddep_launch_dependents();
  const Geometry& g = a.g;
  const Item w = resolve_item(tab, g, static_cast<int>(blockIdx.x), g.N_kv);
  int q_t0, n_q;
  query_tiles_of_key_tile(g, w.s, w.tile, &q_t0, &n_q);
  const int n_it = g.group * n_q, per = steps_per_piece(n_it, w.pieces);
  const int live = n_it > 0 ? (n_it + per - 1) / per : 0;  // pieces with steps
  const float* part = a.part + (a.part_base + blockIdx.x - w.piece) * 2 * kTileN * D;
  constexpr int kChunks = D / 8;
  const int n_rows = min(kTileN, w.s.kv_len - w.tile * kTileN);
  const int mine = n_rows > w.piece ? (n_rows - w.piece + w.pieces - 1) / w.pieces : 0;  // rows of this CTA
  const int h = blockIdx.y;  // dV, dK
  for (int x = threadIdx.x; x < mine * kChunks; x += kJoinThreads) {
    const int c = x % kChunks, r = w.piece + x / kChunks * w.pieces;
    if (c * 8 >= g.D) continue;
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int p = 0; p < live; ++p) {
      const float4* src = reinterpret_cast<const float4*>(part + ((p * 2 + h) * kTileN + r) * D + c * 8);
      const float4 u = src[0], v = src[1];
      o[0] += u.x; o[1] += u.y; o[2] += u.z; o[3] += u.w;
      o[4] += v.x; o[5] += v.y; o[6] += v.z; o[7] += v.w;
    }
    const int64_t e = kv_elem(g, w.s, w.b, w.n, w.tile * kTileN + r) + c * 8;
    if (in_bounds(e, 8, g.n_kv_elems, a.err)) store8<F16>(h == 0 ? a.dv : a.dk, e, o, g.out_f32);
  }
}

}  // namespace

template <int CAP>
cudaError_t launch_backward_join(const BwdArgs& a, const SeqTable<CAP>& tab, int n_pieces, cudaStream_t stream) {
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(n_pieces, 2), dim3(kJoinThreads), 0, stream, a, tab); };
  if (a.g.D <= 64) return a.g.f16 ? go(swa_bwd_join_kernel<64, true, CAP>) : go(swa_bwd_join_kernel<64, false, CAP>);
  return a.g.f16 ? go(swa_bwd_join_kernel<128, true, CAP>) : go(swa_bwd_join_kernel<128, false, CAP>);
}

template cudaError_t launch_backward_join<kSmallTable>(const BwdArgs&, const SeqTable<kSmallTable>&, int, cudaStream_t);
template cudaError_t launch_backward_join<kLargeTable>(const BwdArgs&, const SeqTable<kLargeTable>&, int, cudaStream_t);

}  // namespace swa
