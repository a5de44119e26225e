// swa_paged_rows.cuh — attention over the paged cache for a few query rows per
// sequence and key/value head (single tokens, short speculative chunks, small
// trees of drafted tokens).
//
// Per row (include/swa.h): O = sum_j softmax_j(scale q.k_j) v_j over visible
// keys, softmax_max, softmax_sum; online softmax in fp32 (log2 units).
//
// Bound by HBM: each key and value is read once for the 16 rows of a tile (the
// tokens x query heads that share the key/value head).  A CTA of 4 warps takes
// a run of 64-key steps; each warp owns 16 keys of every step and runs by
// itself: its own 3-stage rings of cp.async copies of K and V (16-byte chunks
// XOR-swizzled against bank conflicts), its own maximum and sum, S = Q K^T and
// O += P V by mma.sync m16n8k16.  With at most 16 rows a 128-row tcgen05 tile
// would be seven eighths padding and its barrier hand-offs would set the
// latency, while the legacy tensor path has several times the rate that HBM
// can feed here.  What a warp does per 16 keys bounds a CTA's rate: with all
// fragments of a group loaded before the first product, a stage refilled as
// soon as they are in registers, and no per-row tests inside the visible run,
// a CTA draws 46 GB/s (32 before).  Measured: 256 sequences x 1024-key windows
// 137 us (the copy rate's own time), 64 x 4096 145 us (0.96 of it), 24
// sequences of up to 8192 keys, 16 heads of 64, 80 us (0.89), one sequence of
// 131072 keys 83 us (0.95).  The warps' results are joined in shared memory at
// the end.
//
// The probabilities are rounded to the element type for the second product, as
// in the dense forward: half a step (2^-8 in bf16, 2^-11 in fp16) of each, which
// leaves the output 1.4 times as far from exact as its own rounding does
// (relative 2.3e-3 and 1.7e-3 in bf16).  With what the rounding leaves out in a
// second product it was at its own rounding, 3 to 5 % slower (64 x 4096 keys
// 150.5 us for 144.1, 131072 keys 85.9 for 82.2): not kept.
//
// A 16-key group lies in one page (page sizes are multiples of 16).  Keys no
// row of the tile sees are never read: their chunks are zero-filled, so a NaN
// in an unused slot cannot reach the products.
//
// Sinks: the 16-key groups that hold them come before those of the window, in
// one list.  A tree: the groups of the chunk itself test a bit per row and key.
//
// The 8-bit cache has a kernel of its own (swa_paged_rows_e4m3.cu).
#pragma once
#include "swa_paged_rows_end.cuh"

namespace swa {
namespace {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <int DP>
struct RowsSmem {
  static constexpr int kRowsStages = 3;
  static constexpr int kRowBytes = DP * 2;
  static constexpr int kGroupBytes = 16 * kRowBytes;  // 16 keys of K or V
  alignas(128) uint8_t ring[kRowsWarps][kRowsStages][2][kGroupBytes];
  float ml[kRowsWarps][kRowsTile][2];
  // the warps' O and what the cluster reads reuse the ring
  static constexpr int kRingBytes = kRowsWarps * kRowsStages * 2 * kGroupBytes;
  static_assert(RowsEnd<DP>::kBytes <= kRingBytes, "join space");
};

// CL: the splits of an item are the CTAs of one cluster, which join their rows
// through each other's shared memory; otherwise partial rows go to the
// workspace and swa_paged_join_kernel joins them.
template <PagedKind KIND, int DP, bool F16, bool CL, int CAP>
__global__ void __launch_bounds__(kRowsThreads, 2)
    swa_paged_rows_kernel(const __grid_constant__ ArgsOf<KIND != PagedKind::kPlain> a,
                          const __grid_constant__ PagedTable<CAP> tab) {
  constexpr bool X = KIND != PagedKind::kPlain;
  using Smem = RowsSmem<DP>;
  constexpr int kRowsStages = Smem::kRowsStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  constexpr int kChunks = Smem::kRowBytes / 16;  // 16-byte chunks of a key row
  const PagedGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Behind the tile kernel of the same call (overlap), whose CTAs signalled
  // after their own wait, every earlier grid has completed: this one may run
  // beside that kernel, and its first CTA waits for it at the end.  Its other
  // CTAs do not wait for a grid, which would make what earlier grids wrote
  // visible to them: the fence does, so that no line which their SM's L1 holds
  // from a call before is taken for q, a length or a block table entry (K and V
  // are read from L2).  Reading all of those from L2 instead cost the calls
  // without overlap, whose warps share them in L1: 131072 keys 86.1 us for
  // 83.4, one token 6.7 for 6.3.
  if (a.overlap) __threadfence();
  else griddep_wait();
  griddep_launch_dependents();
  const PagedItem w = resolve_paged(tab, a.groups, static_cast<int>(blockIdx.x));
  const int split = blockIdx.y;
  if (a.clear_err && blockIdx.x == 0 && split == 0 && threadIdx.x == 0) *a.err = 0;
  const int64_t item = a.item_base + static_cast<int64_t>(blockIdx.x);
  const int tok0 = w.tile * a.tok;
  const int n_tok = min(a.tok, w.q_len - tok0), n_rows = n_tok * a.gs;
  const int kv_raw = in_bounds(w.b, 1, g.n_lens, a.err) ? g.kv_lens[w.b] : 0;  // in flight behind the loads of Q

  // Q as A fragments: rows lane / 4 and lane / 4 + 8
  const int nk = (g.D + 15) >> 4;
  uint32_t qf[DP / 16][4];
  int row_tok[2];  // tokens of the thread's two rows
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = (lane >> 2) + 8 * x;
    const bool valid = r < n_rows;
    const int i = valid ? row_token(r, a.gs_magic) : 0;
    row_tok[x] = i;
    const int h = w.vh * a.gs + (r - i * a.gs);
    const int64_t e = static_cast<int64_t>(w.q_start + tok0 + i) * a.q_row + h * a.q_head;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + e;
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int c = kk * 16 + y * 8 + (lane & 3) * 2;
        qf[kk][x + 2 * y] = valid && c < g.D && in_bounds(e + c, 2, a.n_q, a.err)
                                ? *reinterpret_cast<const uint32_t*>(q + c)
                                : 0u;
      }
  }

  int bad = 0;
  int kv_len = kv_raw;
  if (kv_len < 0 || kv_len > g.kv_limit) {
    bad = kPageErrLength;
    kv_len = 0;
  }
  const PagedKeys keys = paged_keys<X>(a, kv_len, w.q_len, tok0, n_tok);
  const int lo = keys.lo, hi = keys.hi;
  // steps of 64 keys = 4 groups of 16, from the group that holds the first
  const PagedUnits groups = paged_units<X>(keys, 4);
  const int steps = (groups.total + kRowsWarps - 1) / kRowsWarps;
  int st0, st1, active;
  paged_split(steps, a.par, a.cap, a.least, split, &st0, &st1, &active);
  const bool direct = active <= 1;  // no other CTA has keys of this item: write the result itself
  if (!CL && split > 0 && split >= active) {  // nothing to do (split 0 writes the result of an empty item)
    if (threadIdx.x == 0) a.page_err[item * a.splits + split] = 0;
    return;
  }

  int row_lo[2], row_hi[2];  // visible keys of the thread's two rows
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    row_lo[x] = 0;
    row_hi[x] = kv_len - 1;
    if (a.sparse_mode == 4) {
      const int p = token_position<X>(a, w, kv_len, tok0 + row_tok[x]);
      row_lo[x] = max(0, p - a.pre);
      row_hi[x] = min(kv_len - 1, p + a.next);
    }
    if (tree_of<X>(a)) row_hi[x] = kv_len - w.q_len - 1;  // the chunk's own keys go by the tree's bits
  }

  // keys every row of the tile sees: from the last token's first to the first token's last
  int all_lo = 0, all_hi = kv_len - 1;
  if (a.sparse_mode == 4) {
    const int p0 = kv_len - w.q_len + tok0;
    all_lo = max(0, p0 + n_tok - 1 - a.pre);
    all_hi = min(kv_len - 1, p0 + a.next);
  }
  if (tree_of<X>(a)) {  // the deepest token may be q_len - 1 deep
    if (a.sparse_mode == 4) all_lo = max(0, kv_len - 1 - a.pre);
    all_hi = kv_len - w.q_len - 1;
  }

  const int hk = w.vh * a.gs / a.group;
  const uint16_t* kb = static_cast<const uint16_t*>(a.k_pages) + hk * g.k_head;
  const uint16_t* vb = static_cast<const uint16_t*>(a.v_pages) + hk * g.v_head;
  const uint32_t ring = smem_u32(s.ring[warp]);
  const int n_it = st1 - st0;  // the warp's groups: number (st0 + it) * 4 + warp
  const int gw = st0 * kRowsWarps + warp;
  // first key of the warp's group `it`, past hi where there is none
  auto first_key = [&](int it) {
    const int x = gw + it * kRowsWarps;
    return (X ? groups.at(x) : groups.jump + x) * 16;
  };
  // is key j seen by some row of the tile
  auto some_see = [&](int j) { return (j >= lo || (X && j < keys.sinks)) && j <= hi; };

  // page number and first slot of the warp's next 32 groups, one per lane
  int my_page = 0, my_slot = 0;
  auto fetch_pages = [&](int it0) {
    const int j = first_key(it0 + lane);
    my_page = -1;
    my_slot = 0;
    if (it0 + lane < n_it && j <= hi) {
      const int entry = j / g.page_size;
      my_slot = j - entry * g.page_size;
      const int64_t e = w.b * g.table_stride + entry;
      const int page = in_bounds(e, 1, g.n_table, a.err) ? g.table[e] : -1;
      if (page >= 0 && page < g.num_pages) my_page = page;
      else bad = kPageErrEntry;
    }
  };
  const int row_in = lane / kChunks, chunk = lane % kChunks;  // the lane's part of 32 / kChunks rows
  const int live_chunks = 2 * nk;                             // chunks the products read
  // The copies of K (V) of the warp's group `it`.  A stage is free once its
  // fragments are in registers, so close to a ring of each is in flight; every call commits one group, empty past the end.  A group
  // whose 16 keys are all seen needs no per-row test.
  const int in_d = chunk * 8 < g.D;
  const uint32_t lane_dst = ring + row_in * Smem::kRowBytes;
  auto issue = [&](int it, bool is_v) {
    if ((it & 31) == 0 && !is_v) fetch_pages(it);
    const int page = __shfl_sync(0xFFFFFFFFu, my_page, it & 31), slot = __shfl_sync(0xFFFFFFFFu, my_slot, it & 31);
    if (it < n_it && chunk < live_chunks) {
      const int j0 = first_key(it);
      const uint32_t dst = lane_dst + ((it % kRowsStages) * 2 + (is_v ? 1 : 0)) * Smem::kGroupBytes;
      const uint16_t* base = is_v ? vb : kb;
      const int64_t step = is_v ? g.v_slot : g.k_slot;
      const int64_t e0 = page * (is_v ? g.v_page : g.k_page) + (slot + row_in) * step + chunk * 8;
      const bool whole = page >= 0 && (j0 >= lo || (X && j0 + 15 < keys.sinks)) && j0 + 15 <= hi;
      const int64_t head = hk * (is_v ? g.v_head : g.k_head), extent = is_v ? g.n_v : g.n_k;
      if (SWA_CHECKS == 0 && whole) {
        const uint16_t* src = in_d ? base + e0 : base;
        const int64_t hop = in_d ? step * (32 / kChunks) : 0;
#pragma unroll
        for (int x = 0; x < 16 * kChunks / 32; ++x) {
          const int r = x * (32 / kChunks) + row_in;
          cp_async16(dst + x * (32 / kChunks) * Smem::kRowBytes + ((chunk ^ (r & 7)) << 4), src, in_d);
          src += hop;
        }
      } else {
#pragma unroll
        for (int x = 0; x < 16 * kChunks / 32; ++x) {
          const int r = x * (32 / kChunks) + row_in;
          const int64_t e = e0 + x * (32 / kChunks) * step;
          const bool ok = in_d && page >= 0 && some_see(j0 + r) && in_bounds(head + e, 8, extent, a.err);
          cp_async16(dst + x * (32 / kChunks) * Smem::kRowBytes + ((chunk ^ (r & 7)) << 4), ok ? base + e : base, ok);
        }
      }
    }
    cp_async_commit();
  };

  float o[DP / 8][4];
#pragma unroll
  for (int x = 0; x < DP / 8; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y) o[x][y] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, m_true[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const float c = a.scale_log2;

#pragma unroll
  for (int it = 0; it < kRowsStages; ++it) {
    issue(it, false);
    issue(it, true);
  }
  const bool fold = c > 0.f;  // the scale folds into the exponent's multiply-add
  const int mat = lane >> 3, lr = lane & 7;
  const uint32_t k_row = ((mat >> 1) * 8 + lr) * Smem::kRowBytes, v_row = ((mat & 1) * 8 + lr) * Smem::kRowBytes;
  for (int it = 0; it < n_it; ++it) {
    cp_async_wait<2 * kRowsStages - 1>();  // K(it) is the oldest group in flight
    __syncwarp();
    const int j0 = first_key(it);
    const uint32_t kd = ring + (it % kRowsStages) * 2 * Smem::kGroupBytes, vd = kd + Smem::kGroupBytes;
    float sc[2][4];  // scores of keys 0-7 and 8-15
    {
      uint32_t b[DP / 16][4];
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
        if (kk < nk) ldsm_x4(b[kk], kd + k_row + (((kk * 2 + (mat & 1)) ^ lr) << 4));
      __syncwarp();
      issue(it + kRowsStages, false);  // K's stage is free
      // even and odd steps apart: two chains per accumulator instead of one of twice the length
      float s2[2][2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int z = 0; z < 4; ++z) s2[x][y][z] = 0.f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
        if (kk < nk) {
          mma16816<F16>(s2[kk & 1][0], qf[kk], b[kk][0], b[kk][1]);
          mma16816<F16>(s2[kk & 1][1], qf[kk], b[kk][2], b[kk][3]);
        }
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int z = 0; z < 4; ++z) sc[y][z] = s2[0][y][z] + s2[1][y][z];
    }
    cp_async_wait<2 * kRowsStages - 1>();  // V(it): its fragments load behind the softmax
    __syncwarp();
    uint32_t vf[DP / 16][4];
#pragma unroll
    for (int nb = 0; nb < DP / 16; ++nb)
      if (nb < nk) ldsm_x4_trans(vf[nb], vd + v_row + (((nb * 2 + (mat >> 1)) ^ lr) << 4));
    __syncwarp();
    issue(it + kRowsStages, true);  // V's stage is free
    // mask (groups at the ends of the visible run only), running maximum
    float mx[2] = {-INFINITY, -INFINITY};
    if (!fold || (j0 < all_lo && !(X && j0 + 15 < sinks_of<X>(a))) || j0 + 15 > all_hi) {
      uint32_t drafted[2] = {0u, 0u};  // bit t: key j0 + t is a token of the chunk that the row sees
      if constexpr (X) {
        const int c0 = j0 - (kv_len - w.q_len);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (a.tree && c0 > -16) drafted[x] = tree_bits(a, w, tok0 + row_tok[x], c0);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int x = y >> 1;
          const int j = j0 + t * 8 + (lane & 3) * 2 + (y & 1);
          bool vis = (j >= row_lo[x] || (X && j < sinks_of<X>(a))) && j <= row_hi[x];
          if (X) vis = vis || ((drafted[x] >> (j - j0)) & 1u) != 0;
          sc[t][y] = vis ? (fold ? sc[t][y] : sc[t][y] * c) : -INFINITY;
        }
    }
    const float cf = fold ? c : 1.f;
    bool grow = false;
    float mn[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      mx[x] = fmaxf(fmaxf(sc[0][2 * x], sc[0][2 * x + 1]), fmaxf(sc[1][2 * x], sc[1][2 * x + 1]));
      mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xFFFFFFFFu, mx[x], 1));
      mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xFFFFFFFFu, mx[x], 2));
      m_true[x] = mn[x] = fmaxf(m_true[x], mx[x] * cf);
      grow |= mn[x] > m[x] + kRescale;
    }
    if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float alpha = mn[x] > m[x] ? ex2_approx(m[x] - mn[x]) : 1.f;  // (also when m is -inf: 0)
        m[x] = mn[x];
        l[x] *= alpha;
#pragma unroll
        for (int t = 0; t < DP / 8; ++t) {
          o[t][2 * x] *= alpha;
          o[t][2 * x + 1] *= alpha;
        }
      }
    }
    uint32_t p[4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float ms = m[x] == -INFINITY ? 0.f : m[x];
      const float p0 = ex2_approx(fmaf(sc[0][2 * x], cf, -ms)), p1 = ex2_approx(fmaf(sc[0][2 * x + 1], cf, -ms));
      const float p2 = ex2_approx(fmaf(sc[1][2 * x], cf, -ms)), p3 = ex2_approx(fmaf(sc[1][2 * x + 1], cf, -ms));
      l[x] += (p0 + p1) + (p2 + p3);
      p[x] = pack2<F16>(p0, p1);      // keys 0-7
      p[2 + x] = pack2<F16>(p2, p3);  // keys 8-15
    }
#pragma unroll
    for (int nb = 0; nb < DP / 16; ++nb)
      if (nb < nk) {
        mma16816<F16>(o[2 * nb], p, vf[nb][0], vf[nb][1]);
        mma16816<F16>(o[2 * nb + 1], p, vf[nb][2], vf[nb][3]);
      }
  }
  cp_async_wait<0>();
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 1);
    l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 2);
  }
  bad = __reduce_max_sync(0xFFFFFFFFu, bad);
  __syncthreads();  // every warp is done with its ring
  float* so = reinterpret_cast<float*>(&s.ring[0][0][0][0]);
  // l is relative to m (which may lag behind the true maximum by 2^8); both go on
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = (lane >> 2) + 8 * x;
    if ((lane & 3) == 0) {
      // relative to the true maximum from here on
      const float f = m_true[x] == -INFINITY ? 0.f : ex2_approx(m[x] - m_true[x]);
      s.ml[warp][r][0] = m_true[x];
      s.ml[warp][r][1] = l[x] * f;
    }
    const float f = m_true[x] == -INFINITY ? 0.f : ex2_approx(m[x] - m_true[x]);
    float* row = so + (warp * kRowsTile + r) * RowsEnd<DP>::kOPitch;
#pragma unroll
    for (int t = 0; t < DP / 8; ++t)
      *reinterpret_cast<float2*>(row + t * 8 + (lane & 3) * 2) = make_float2(o[t][2 * x] * f, o[t][2 * x + 1] * f);
  }
  rows_end<DP, F16, CL>(a, w, split, item, tok0, n_rows, direct, bad, so, s.ml);
  if (a.overlap && blockIdx.x == 0 && blockIdx.y == 0) griddep_wait();  // (no early return: split 0 always runs)
}

template <PagedKind KIND, int DP, bool F16, bool CL, int CAP>
cudaError_t launch_rows_t(const ArgsOf<KIND != PagedKind::kPlain>& a, const PagedTable<CAP>& tab, cudaStream_t stream) {
  const size_t smem = sizeof(RowsSmem<DP>);
  auto kernel = swa_paged_rows_kernel<KIND, DP, F16, CL, CAP>;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit(kernel, smem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_rows_grid<CL>(kernel, dim3(tab.n_items, a.splits), smem, stream, a, tab);
}

}  // namespace

template <PagedKind KIND, int CAP>
cudaError_t launch_paged_rows(const PagedArgs& a, const PagedTable<CAP>& tab, cudaStream_t stream) {
  if (tab.n_items == 0) return cudaSuccess;
  if (a.cluster) {
    if (a.g.D <= 64)
      return a.f16 ? launch_rows_t<KIND, 64, true, true>(a, tab, stream)
                   : launch_rows_t<KIND, 64, false, true>(a, tab, stream);
    return a.f16 ? launch_rows_t<KIND, 128, true, true>(a, tab, stream)
                 : launch_rows_t<KIND, 128, false, true>(a, tab, stream);
  }
  if (a.g.D <= 64)
    return a.f16 ? launch_rows_t<KIND, 64, true, false>(a, tab, stream)
                 : launch_rows_t<KIND, 64, false, false>(a, tab, stream);
  return a.f16 ? launch_rows_t<KIND, 128, true, false>(a, tab, stream)
               : launch_rows_t<KIND, 128, false, false>(a, tab, stream);
}

}  // namespace swa
