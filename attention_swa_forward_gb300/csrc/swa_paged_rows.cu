// swa_paged_rows.cu — attention over the paged cache for a few query rows per
// sequence and key/value head (single tokens, short speculative chunks), and
// the pass that joins results of keys split over several CTAs.
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
#include "swa_paged.h"
#include "swa_device.cuh"

namespace swa {
namespace {

constexpr int kRowsWarps = kRowsStep / 16;
constexpr int kRowsThreads = kRowsWarps * 32;
constexpr int kRowsStages = 3;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // rescale only when the maximum grows by more than 2^8

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

template <int DP>
struct RowsSmem {
  static constexpr int kRowBytes = DP * 2;
  static constexpr int kGroupBytes = 16 * kRowBytes;  // 16 keys of K or V
  alignas(128) uint8_t ring[kRowsWarps][kRowsStages][2][kGroupBytes];
  float ml[kRowsWarps][kRowsTile][2];
  // the warps' O, [warp][row][DP + 4], reuses the ring, and behind it the
  // CTA's own joined rows and their maxima and sums, for the cluster
  static constexpr int kOPitch = DP + 4;
  static constexpr int kRingBytes = kRowsWarps * kRowsStages * 2 * kGroupBytes;
  static constexpr int kJoinAt = kRowsWarps * kRowsTile * kOPitch;  // floats
  static constexpr int kMlAt = kJoinAt + kRowsTile * DP;
  static_assert(4 * (kMlAt + 2 * kRowsTile) <= kRingBytes, "join space");
};

// CL: the splits of an item are the CTAs of one cluster, which join their rows
// through each other's shared memory; otherwise partial rows go to the
// workspace and swa_paged_join_kernel joins them.
template <int DP, bool F16, bool CL, int CAP>
__global__ void __launch_bounds__(kRowsThreads, 2)
    swa_paged_rows_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedTable<CAP> tab) {
  using Smem = RowsSmem<DP>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  constexpr int kChunks = DP / 8;  // 16-byte chunks of a key row
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
  int lo, hi;
  paged_key_range(a.sparse_mode, a.pre, a.next, kv_len, w.q_len, tok0, n_tok, &lo, &hi);
  // steps of 64 keys = 4 groups of 16, from the group that holds lo
  const int g0 = lo >> 4;
  const int steps = lo <= hi ? ((hi >> 4) - g0) / kRowsWarps + 1 : 0;
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
      const int p = kv_len - w.q_len + tok0 + row_tok[x];
      row_lo[x] = max(0, p - a.pre);
      row_hi[x] = min(kv_len - 1, p + a.next);
    }
  }

  // keys every row of the tile sees: from the last token's first to the first token's last
  int all_lo = 0, all_hi = kv_len - 1;
  if (a.sparse_mode == 4) {
    const int p0 = kv_len - w.q_len + tok0;
    all_lo = max(0, p0 + n_tok - 1 - a.pre);
    all_hi = min(kv_len - 1, p0 + a.next);
  }

  const int hk = w.vh * a.gs / a.group;
  const uint16_t* kb = static_cast<const uint16_t*>(a.k_pages) + hk * g.k_head;
  const uint16_t* vb = static_cast<const uint16_t*>(a.v_pages) + hk * g.v_head;
  const uint32_t ring = smem_u32(s.ring[warp]);
  const int n_it = st1 - st0;  // the warp's groups: g0 + (st0 + it) * 4 + warp
  const int gw = g0 + st0 * kRowsWarps + warp;

  // page number and first slot of the warp's next 32 groups, one per lane
  int my_page = 0, my_slot = 0;
  auto fetch_pages = [&](int it0) {
    const int j = (gw + (it0 + lane) * kRowsWarps) * 16;
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
      const int j0 = (gw + it * kRowsWarps) * 16;
      const uint32_t dst = lane_dst + ((it % kRowsStages) * 2 + (is_v ? 1 : 0)) * Smem::kGroupBytes;
      const uint16_t* base = is_v ? vb : kb;
      const int64_t step = is_v ? g.v_slot : g.k_slot;
      const int64_t e0 = page * (is_v ? g.v_page : g.k_page) + (slot + row_in) * step + chunk * 8;
      const bool whole = page >= 0 && j0 >= lo && j0 + 15 <= hi;
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
          const bool ok = in_d && page >= 0 && j0 + r >= lo && j0 + r <= hi && in_bounds(head + e, 8, extent, a.err);
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
    const int j0 = (gw + it * kRowsWarps) * 16;
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
    if (!fold || j0 < all_lo || j0 + 15 > all_hi) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int x = y >> 1;
          const int j = j0 + t * 8 + (lane & 3) * 2 + (y & 1);
          const bool vis = j >= row_lo[x] && j <= row_hi[x];
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
#pragma unroll
    for (int t = 0; t < DP / 8; ++t)
      *reinterpret_cast<float2*>(so + (warp * kRowsTile + r) * Smem::kOPitch + t * 8 + (lane & 3) * 2) =
          make_float2(o[t][2 * x] * f, o[t][2 * x + 1] * f);
  }
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
    for (int v = 0; v < kRowsWarps; ++v) M = fmaxf(M, s.ml[v][r][0]);
    const float ms = M == -INFINITY ? 0.f : M;
    float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kRowsWarps; ++v) {
      const float f = ex2_approx(s.ml[v][r][0] - ms);
      L += s.ml[v][r][1] * f;
      const float4 ov = *reinterpret_cast<const float4*>(so + (v * kRowsTile + r) * Smem::kOPitch + col);
      acc[0] += ov.x * f;
      acc[1] += ov.y * f;
      acc[2] += ov.z * f;
      acc[3] += ov.w * f;
    }
    if (CL) {
      *reinterpret_cast<float4*>(so + Smem::kJoinAt + r * DP + col) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (col == 0) *reinterpret_cast<float2*>(so + Smem::kMlAt + 2 * r) = make_float2(M, L);
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
    const uint32_t rank = cluster_rank(), mine = smem_u32(so + Smem::kJoinAt), mine_ml = smem_u32(so + Smem::kMlAt);
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
  if (a.overlap && blockIdx.x == 0 && blockIdx.y == 0) griddep_wait();  // (no early return: split 0 always runs)
}

// Join the splits of a row tile: WPR warps per row over its splits (each reads
// a partial row with one load per lane), then over their sums in shared
// memory; one warp up to 8 splits, eight past that.  Reads the active partial
// rows once, a few microseconds behind the kernel that wrote them, launched so
// that its prologue overlaps that tail.  (One warp per row took 30 us for the
// 152 splits that one 131072-token sequence had.)
constexpr int kJoinWarps = 8;
template <int DP, bool F16, int WPR, int CAP>
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
  int lo, hi, st0, st1, active;
  paged_key_range(a.sparse_mode, a.pre, a.next, kv_len, w.q_len, tok0, n_tok, &lo, &hi);
  const int first = step_keys == kRowsStep ? lo >> 4 << 4 : lo / step_keys * step_keys;
  const int steps = lo <= hi ? (hi - first) / step_keys + 1 : 0;
  paged_split(steps, a.par, a.cap, a.least, 0, &st0, &st1, &active);
  griddep_wait();
  griddep_launch_dependents();
  if (r >= n_tok * a.gs) return;  // (with WPR > 1 a CTA is one row: all of it returns)
  static_assert(WPR == 1 || WPR == kJoinWarps, "a CTA is one row or one row per warp");
  if (active <= 1) return;  // written by the CTA that had the keys
  const int64_t item = a.item_base + static_cast<int64_t>(blockIdx.x);  // among the split ones
  const int64_t p0 = item * a.splits * a.rows_pad + r;
  // each warp: its splits' maximum, then their sum relative to it
  float M = -INFINITY;
  for (int x = part + WPR * lane; x < active; x += 32 * WPR)
    M = fmaxf(M, a.part_ml[p0 + static_cast<int64_t>(x) * a.rows_pad].x);
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, x));
  const float ms = M == -INFINITY ? 0.f : M;
  float L = 0.f, acc[kPer];
#pragma unroll
  for (int y = 0; y < kPer; ++y) acc[y] = 0.f;
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

template <int DP, bool F16, bool CL, int CAP>
cudaError_t launch_rows_t(const PagedArgs& a, const PagedTable<CAP>& tab, cudaStream_t stream) {
  const size_t smem = sizeof(RowsSmem<DP>);
  auto kernel = swa_paged_rows_kernel<DP, F16, CL, CAP>;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit(kernel, smem, smem_set);
  if (e != cudaSuccess) return e;
  const dim3 grid(tab.n_items, a.splits), block(kRowsThreads);
  if constexpr (!CL) {
    return launch_pdl(kernel, grid, block, smem, stream, a, tab);
  } else {
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = static_cast<unsigned>(a.splits);
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, tab);
  }
}

template <int DP, bool F16, int CAP>
cudaError_t launch_join_t(const PagedArgs& a, const PagedTable<CAP>& tab, int step_keys, cudaStream_t stream) {
  const int rows = a.tok * a.gs;
  if (a.splits <= 8)
    return launch_pdl(swa_paged_join_kernel<DP, F16, 1, CAP>, dim3(tab.n_items - a.whole, (rows + kJoinWarps - 1) / kJoinWarps),
                      dim3(kJoinWarps * 32), 0, stream, a, tab, step_keys);
  return launch_pdl(swa_paged_join_kernel<DP, F16, kJoinWarps, CAP>, dim3(tab.n_items - a.whole, rows), dim3(kJoinWarps * 32), 0,
                    stream, a, tab, step_keys);
}

}  // namespace

template <int CAP>
cudaError_t launch_paged_rows(const PagedArgs& a, const PagedTable<CAP>& tab, cudaStream_t stream) {
  if (tab.n_items == 0) return cudaSuccess;
  if (a.cluster) {
    if (a.g.D <= 64)
      return a.f16 ? launch_rows_t<64, true, true>(a, tab, stream) : launch_rows_t<64, false, true>(a, tab, stream);
    return a.f16 ? launch_rows_t<128, true, true>(a, tab, stream) : launch_rows_t<128, false, true>(a, tab, stream);
  }
  if (a.g.D <= 64)
    return a.f16 ? launch_rows_t<64, true, false>(a, tab, stream) : launch_rows_t<64, false, false>(a, tab, stream);
  return a.f16 ? launch_rows_t<128, true, false>(a, tab, stream) : launch_rows_t<128, false, false>(a, tab, stream);
}
template <int CAP>
cudaError_t launch_paged_join(const PagedArgs& a, const PagedTable<CAP>& tab, int step_keys, cudaStream_t stream) {
  if (tab.n_items == 0) return cudaSuccess;
  if (a.g.D <= 64)
    return a.f16 ? launch_join_t<64, true>(a, tab, step_keys, stream)
                 : launch_join_t<64, false>(a, tab, step_keys, stream);
  return a.f16 ? launch_join_t<128, true>(a, tab, step_keys, stream)
               : launch_join_t<128, false>(a, tab, step_keys, stream);
}

template cudaError_t launch_paged_rows<kPagedSmallTable>(const PagedArgs&, const PagedTable<kPagedSmallTable>&,
                                                         cudaStream_t);
template cudaError_t launch_paged_rows<kPagedLargeTable>(const PagedArgs&, const PagedTable<kPagedLargeTable>&,
                                                         cudaStream_t);
template cudaError_t launch_paged_join<kPagedSmallTable>(const PagedArgs&, const PagedTable<kPagedSmallTable>&, int,
                                                         cudaStream_t);
template cudaError_t launch_paged_join<kPagedLargeTable>(const PagedArgs&, const PagedTable<kPagedLargeTable>&, int,
                                                         cudaStream_t);

}  // namespace swa
