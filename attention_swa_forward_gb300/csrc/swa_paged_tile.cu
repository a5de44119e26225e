// swa_paged_tile.cu — attention of a chunk over the paged cache on the 5th-gen
// tensor cores: row tiles of 128 (tokens x the query heads that share a
// key/value head), key tiles of 128.
//
// Per row (include/swa.h): O = sum_j softmax_j(scale q.k_j) v_j over visible
// keys, softmax_max, softmax_sum; online softmax in fp32 (log2 units), P
// rounded to the element type for the second product.
//
// Bound by the tensor pipe and its hand-offs to the softmax, like the dense
// forward, whose roles it keeps (swa_fwd.cu): one thread per row in warps 0-3,
// S = Q K^T into one of two TMEM tiles by the thread of warp 5, O += P V by the
// thread of warp 6 with P taken from TMEM.  What is different:
//  * Packing the G heads of a key/value head into the rows (128 / G tokens per
//    tile) reads a key tile once for all of them, fills tiles of short chunks,
//    and cuts the masked part of the tiles at the window's edges by G.
//  * Warps 4 and 7 gather the K and the V tiles from pages: each lane issues one
//    TMA box (up to 128 slots x 64 columns) at the page its own block table
//    entry names, loaded two tiles ahead.  An entry that is not to be followed
//    becomes the coordinate past the last page, which TMA fills with zeros.
//    (One warp for both, waiting for its table entries one tile ahead, took
//    ~3500 cycles per tile and held everything up: 765 us against 426 of the
//    dense forward on a causal 8192-token prompt.)
//  * Q rows are gathered by the softmax warps (any strides; rows past the tile
//    are zero).
//  * A key tile at either end of the chunk's keys may hold slots that no query
//    sees (stale or never written, possibly NaN): warp 6 zeroes those rows of
//    V in shared memory, since 0 * NaN would reach O.
// TMEM columns as in swa_fwd.cu: S0 [0,128), S1 [128,256), O [256,256+D),
// P0 [384,448), P1 [448,512).
#include "swa_paged.h"
#include "swa_device.cuh"

namespace swa {
namespace {

constexpr int kStages = 3;
constexpr int kThreads = 256;

template <int D>
struct TileSmem {
  static constexpr int kTileBytes = kPagedTileRows * D * 2;
  alignas(1024) uint8_t q[kTileBytes];
  alignas(1024) uint8_t k[kStages][kTileBytes];
  alignas(1024) uint8_t v[kStages][kTileBytes];
  uint64_t q_full, k_full[kStages], v_full[kStages], k_empty[kStages], v_empty[kStages];
  uint64_t s_full[2], s_free[2], p_full[2], o_done[2], drain_s, drain_pv;
  uint64_t never;  // completed by nothing: the target of the stall test hook
  uint32_t tmem_base;
};
static_assert(sizeof(TileSmem<128>) + 1024 <= 232448, "shared memory budget");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256, kColP = 384;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // as in swa_fwd.cu

// Where one lane of a gathering warp finds its part of successive key tiles:
// box `box` (box_rows slots) of the tile, in atom column `atom`.
struct PageWalk {
  int entry, slot;    // block table column and first slot of the next tile's box
  int step_e, step_s;  // 128 slots on
  int j;              // its first key
  int lo, hi, box_rows, page_size, num_pages;
  const int32_t* row;  // the sequence's block table row
  int64_t left;        // entries of the table from `row` on (bounds-checked build)
  int32_t* err;

  __device__ __forceinline__ void start(const PagedArgs& a, int b, int j0, int box, int lo_, int hi_) {
    lo = lo_;
    hi = hi_;
    box_rows = a.box_rows;
    page_size = a.g.page_size;
    num_pages = a.g.num_pages;
    j = j0 + box * box_rows;
    entry = j / page_size;
    slot = j - entry * page_size;
    step_e = kPagedTileStep / page_size;
    step_s = kPagedTileStep - step_e * page_size;
    row = a.g.table + b * a.g.table_stride;
    left = a.g.n_table - b * a.g.table_stride;
    err = a.err;
  }
  // The raw entry of the next tile's box and its first slot (num_pages and -1
  // when no key of it is seen), and on to the tile after.  Nothing waits for
  // the load here.
  __device__ __forceinline__ void next(bool mine, int& raw, int& at) {
    raw = num_pages;
    at = -1;
    if (mine && j <= hi && j + box_rows > lo) {
      at = slot;
      raw = in_bounds(entry, 1, left, err) ? __ldg(row + entry) : -1;
    }
    j += kPagedTileStep;
    entry += step_e;
    slot += step_s;
    if (slot >= page_size) {
      slot -= page_size;
      ++entry;
    }
  }
};

template <int D, bool F16, int CAP>
__global__ void __launch_bounds__(kThreads, 1)
    swa_paged_tile_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedTable<CAP> tab,
                          const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  extern __shared__ uint8_t smem_raw[];
  TileSmem<D>& s = *reinterpret_cast<TileSmem<D>*>(align1024(smem_raw));
  constexpr int kTileBytes = TileSmem<D>::kTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  // the few-row kernel of the same call may fill the SMs that the last wave
  // leaves (it waits for this grid at its end); nothing else starts early
  if (a.signal) griddep_launch_dependents();
  if (a.clear_err && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.err = 0;
  const PagedGeom& g = a.g;
  const PagedItem w = resolve_paged(tab, a.groups, static_cast<int>(blockIdx.x));
  const int split = blockIdx.y;
  const int64_t slot_id = (a.item_base + static_cast<int64_t>(blockIdx.x)) * a.splits + split;
  int kv_len = in_bounds(w.b, 1, g.n_lens, a.err) ? g.kv_lens[w.b] : 0;
  const bool bad_len = kv_len < 0 || kv_len > g.kv_limit;
  if (bad_len) kv_len = 0;
  const int tok0 = w.tile * a.tok;
  const int n_tok = min(a.tok, w.q_len - tok0), n_rows = n_tok * a.gs;
  int lo, hi;
  paged_key_range(a.sparse_mode, a.pre, a.next, kv_len, w.q_len, tok0, n_tok, &lo, &hi);
  const int t_first = lo >> 7;
  const int steps = lo <= hi ? (hi >> 7) - t_first + 1 : 0;
  int st0, st1, active;
  paged_split(steps, a.par, a.cap, a.least, split, &st0, &st1, &active);
  const bool direct = active <= 1;  // no other CTA has keys of this item: write the result itself
  if (split > 0 && split >= active) {  // nothing to do (split 0 writes the result of an empty item)
    if (threadIdx.x == 0) a.page_err[slot_id] = 0;
    return;
  }
  const int kv_t0 = t_first + st0, n_kv = st1 - st0;
  const int hk = w.vh * a.gs / a.group;  // the key/value head of the tile's rows

  // Q, by the softmax warps: 32 rows each, 16 bytes a lane; rows past the tile
  // are zero.  Nothing here depends on the cache, so the loads go out first.
  if (warp < 4) {
    constexpr int kChunks = D / 8, kRowsPer = 32 / kChunks;  // 16 chunks: 2 rows a step; 8: 4 rows
    const int ch = lane % kChunks;
    uint4 v[32 / kRowsPer];
#pragma unroll
    for (int x = 0; x < 32 / kRowsPer; ++x) {
      const int rr = warp * 32 + x * kRowsPer + lane / kChunks;
      const int ii = row_token(rr, a.gs_magic);
      const int64_t e = static_cast<int64_t>(w.q_start + tok0 + ii) * a.q_row +
                        static_cast<int64_t>(w.vh * a.gs + rr - ii * a.gs) * a.q_head + ch * 8;
      v[x] = make_uint4(0u, 0u, 0u, 0u);
      if (rr < n_rows && ch * 8 < g.D && in_bounds(e, 8, a.n_q, a.err))
        v[x] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + e);
    }
#pragma unroll
    for (int x = 0; x < 32 / kRowsPer; ++x) st_chunk_sw128(s.q, warp * 32 + x * kRowsPer + lane / kChunks, ch, v[x]);
    fence_proxy_async_smem();
  }

  // The gathering warps: lane = (box, atom column).
  const int box = lane / (D / 64), atom = lane % (D / 64);
  const bool mine = box < kPagedTileStep / a.box_rows;
  int bad = bad_len ? kPageErrLength : 0;
  PageWalk walk;
  int raw0 = g.num_pages, at0 = -1, raw1 = g.num_pages, at1 = -1;  // entries of this tile and the next
  auto put = [&](uint8_t* tile, const CUtensorMap* map, const PageDims& pd, uint64_t* bar, int raw, int slot) {
    int page = raw;
    if (page < 0 || page > g.num_pages) {
      bad = max(bad, static_cast<int>(kPageErrEntry));
      page = g.num_pages;
    } else if (page == g.num_pages && slot >= 0) {
      bad = max(bad, static_cast<int>(kPageErrEntry));
    }
    slot = max(slot, 0);
    if (lane == 0) mbar_arrive_expect_tx(bar, kTileBytes);
    __syncwarp();
    if (mine) {
      const int c1 = pd.slot_at == 1 ? slot : (pd.head_at == 1 ? hk : page);
      const int c2 = pd.slot_at == 2 ? slot : (pd.head_at == 2 ? hk : page);
      const int c3 = pd.slot_at == 3 ? slot : (pd.head_at == 3 ? hk : page);
      tma_load_4d(tile + atom * kAtomBytes + box * a.box_rows * 128, map, bar, atom * 64, c1, c2, c3);
    }
  };
  if (warp == 4 || warp == 7) {
    walk.start(a, w.b, kv_t0 * kPagedTileStep, box, lo, hi);
    walk.next(mine && n_kv > 0, raw0, at0);
    walk.next(mine && n_kv > 1, raw1, at1);
  }
  if (warp == 4) {
    if (lane == 0) {
      mbar_init(&s.q_full, kPagedTileRows);
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&s.k_full[i], 1);
        mbar_init(&s.v_full[i], 1);
        mbar_init(&s.k_empty[i], 1);
        mbar_init(&s.v_empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s.s_full[i], 1);
        mbar_init(&s.s_free[i], kPagedTileRows);
        mbar_init(&s.p_full[i], kPagedTileRows);
      }
      mbar_init(&s.o_done[0], 1);
      mbar_init(&s.o_done[1], 1);
      mbar_init(&s.drain_s, 1);
      mbar_init(&s.drain_pv, 1);
      mbar_init(&s.never, 1);
      fence_mbar_init();
      tma_prefetch_desc(&mk);
      tma_prefetch_desc(&mv);
    }
    __syncwarp();
    // the first K tile before the CTA-wide barrier, so that its latency runs
    // while TMEM is allocated
    if (n_kv > 0) put(s.k[0], &mk, a.kd, &s.k_full[0], raw0, at0);
  }
  if (warp == 5) {
    tmem_alloc(&s.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s.tmem_base;

  if (warp == 4 || warp == 7) {
    // ------------------------------------------- producers: pages -> tiles --
    const bool is_k = warp == 4;
    uint64_t* full = is_k ? s.k_full : s.v_full;
    uint64_t* empty = is_k ? s.k_empty : s.v_empty;
    int issued = 0;
    for (int it = 0; it < n_kv; ++it) {
      const int st = it % kStages;
      if (!is_k || it > 0) {  // (K(0) is on its way)
        if (it >= kStages &&
            !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], (it / kStages - 1) & 1, a.err, kErrFwdLoad)))
          break;
        if (is_k) put(s.k[st], &mk, a.kd, &full[st], raw0, at0);
        else put(s.v[st], &mv, a.vd, &full[st], raw0, at0);
      }
      ++issued;
      raw0 = raw1;
      at0 = at1;
      walk.next(mine && it + 2 < n_kv, raw1, at1);
    }
    if (lane == 0) {  // every copy issued has landed before the CTA may exit
      for (int st = 0; st < kStages; ++st) {
        const int uses = (issued - st + kStages - 1) / kStages;
        if (uses > 0) mbar_wait_drain(&full[st], (uses - 1) & 1);
      }
    }
    bad = __reduce_max_sync(0xFFFFFFFFu, bad);
    if (is_k && lane == 0) a.page_err[slot_id] = bad;
  } else if (warp == 5) {
    // ------------------------------------------------ S = Q K^T issuer --
    if (lane == 0 && n_kv > 0) {
      constexpr uint32_t kIdS = idesc_f16_f32(kTileM, kTileN, false, false, F16);
      const uint32_t q_addr = smem_u32(s.q);
      const int nk = (g.D + 15) >> 4;
      bool ok = mbar_wait(&s.q_full, 0, a.err, kErrFwdMma);
      for (int it = 0; ok && it < n_kv; ++it) {
        const int st = it % kStages, sb = it & 1;
        if (it >= 2 && !mbar_wait(&s.s_free[sb], ((it >> 1) - 1) & 1, a.err, kErrFwdMma)) break;
        if (!mbar_wait(&s.k_full[st], (it / kStages) & 1, a.err, kErrFwdMma)) break;
        tc_fence_after_sync();
        const uint64_t dq_ = sdesc_sw128(q_addr, 16, 1024), dk_ = sdesc_sw128(smem_u32(s.k[st]), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if (kk >= nk) break;
          const uint32_t off = (kk >> 2) * kAtomBytes + (kk & 3) * 32;
          umma_bf16_ss(tmem + sb * kTileN, sdesc_advance(dq_, off), sdesc_advance(dk_, off), kIdS, kk > 0);
        }
        umma_commit(&s.s_full[sb]);
        umma_commit(&s.k_empty[st]);
      }
      umma_commit(&s.drain_s);
      mbar_wait_drain(&s.drain_s, 0);
    }
  } else if (warp == 6) {
    // ------------------------------------------------- O += P V issuer --
    if (n_kv > 0) {
      constexpr uint32_t kIdO = idesc_f16_f32(kTileM, D, false, true, F16);
      int seen_lo, seen_hi;
      paged_key_range(a.sparse_mode, a.pre, a.next, kv_len, w.q_len, 0, w.q_len, &seen_lo, &seen_hi);
      for (int it = 0; it < n_kv; ++it) {
        const int pb = it & 1, st = it % kStages;
        const int j0 = (kv_t0 + it) * kPagedTileStep;
        if (j0 < seen_lo || j0 + kPagedTileStep - 1 > seen_hi) {
          // rows of V that no query of the chunk sees
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&s.v_full[st], (it / kStages) & 1, a.err, kErrFwdMma))) break;
          const int head_rows = max(seen_lo - j0, 0), tail_at = min(seen_hi - j0 + 1, kPagedTileStep);
          const int dead = head_rows + kPagedTileStep - tail_at;
          for (int x = lane; x < dead * (D / 8); x += 32) {
            const int d = x / (D / 8), c = x % (D / 8);
            const int r = d < head_rows ? d : tail_at + (d - head_rows);
            *reinterpret_cast<uint4*>(s.v[st] + (c >> 3) * kAtomBytes + r * 128 + (c & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        bool ok = true;
        if (lane == 0) {
          ok = mbar_wait(&s.p_full[pb], (it >> 1) & 1, a.err, kErrFwdMma) &&
               mbar_wait(&s.v_full[st], (it / kStages) & 1, a.err, kErrFwdMma);
          if (ok) {
            tc_fence_after_sync();
            const uint64_t dv_ = sdesc_sw128(smem_u32(s.v[st]), kAtomBytes, 1024);
#pragma unroll
            for (int kk = 0; kk < kTileN / 16; ++kk)  // O += P V  (A = P in TMEM)
              umma_bf16_ts(tmem + kColO, tmem + kColP + pb * 64 + kk * 8, sdesc_advance(dv_, kk * 2048), kIdO,
                           (it > 0 || kk > 0) ? 1u : 0u);
            umma_commit(&s.o_done[pb]);
            umma_commit(&s.v_empty[st]);
          }
        }
        if (!__shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0)) break;
      }
      if (lane == 0) {
        umma_commit(&s.drain_pv);
        mbar_wait_drain(&s.drain_pv, 0);
      }
    }
  } else {
    // ------------------------------------------ softmax + epilogue (rows) --
    const int r = threadIdx.x;  // 0..127 == TMEM lane
    const int i = row_token(r, a.gs_magic);  // token of the tile
    const bool row_valid = r < n_rows;
    const int p_row = kv_len - w.q_len + tok0 + i;
    int wlo = 0, whi = kv_len - 1;
    if (a.sparse_mode == 4) {
      wlo = max(0, p_row - a.pre);
      whi = min(kv_len - 1, p_row + a.next);
    }
    if (!row_valid) {
      wlo = 1;
      whi = 0;
    }
    // keys every valid row sees: from the last token's first to the first token's last
    int all_lo = 0, all_hi = kv_len - 1;
    if (a.sparse_mode == 4) {
      const int p0 = kv_len - w.q_len + tok0;
      all_lo = max(0, p0 + n_tok - 1 - a.pre);
      all_hi = min(kv_len - 1, p0 + a.next);
    }
    mbar_arrive(&s.q_full);  // (Q was gathered before the CTA-wide barrier)
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const float c = a.scale_log2;
    float m_use = -INFINITY, m_true = -INFINITY, l = 0.f;
    bool ok = true;
    if (a.stall & kStallPaged)  // test hook: a wait that nothing completes
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s.never, 0, a.err, kErrFwdSoftmax));
    bool s_ready = false;  // S(it) known complete from a probe issued during the previous tile
    for (int it = 0; ok && it < n_kv; ++it) {
      const int sb = it & 1;
      if (!s_ready && !__all_sync(0xFFFFFFFFu, mbar_wait(&s.s_full[sb], (it >> 1) & 1, a.err, kErrFwdSoftmax))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      uint32_t xr[kTileN];
      {
        uint32_t(&x0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&xr[0]);
        uint32_t(&x1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&xr[32]);
        uint32_t(&x2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&xr[64]);
        uint32_t(&x3)[32] = *reinterpret_cast<uint32_t(*)[32]>(&xr[96]);
        const uint32_t base = tmem + lane_off + sb * kTileN;
        tmem_ld_32x32b_x32(base + 0, x0);
        tmem_ld_32x32b_x32(base + 32, x1);
        tmem_ld_32x32b_x32(base + 64, x2);
        tmem_ld_32x32b_x32(base + 96, x3);
        tmem_ld_wait(x0);
        tmem_ld_wait(x1);
        tmem_ld_wait(x2);
        tmem_ld_wait(x3);
      }
      tc_fence_before_sync();
      mbar_arrive(&s.s_free[sb]);
      const bool p_free = it < 2 || mbar_test(&s.o_done[sb], ((it >> 1) - 1) & 1);
      auto X = [&](int t) -> float { return __uint_as_float(xr[t]); };

      const int j0 = (kv_t0 + it) * kPagedTileStep;
      const bool fold = c > 0.f;
      const bool fast = fold && j0 >= all_lo && j0 + kPagedTileStep - 1 <= all_hi;
      float mx;
      {
        float m8[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) m8[u] = -INFINITY;
        if (fast) {
#pragma unroll
          for (int t = 0; t < kTileN; t += 2) m8[(t >> 1) & 7] = fmax3(m8[(t >> 1) & 7], X(t), X(t + 1));
        } else {
          const int lo_t = wlo - j0, hi_t = whi - j0;
#pragma unroll
          for (int t = 0; t < kTileN; ++t) {
            const bool vis = (t >= lo_t) & (t <= hi_t);
            const float v = vis ? (fold ? X(t) : X(t) * c) : -INFINITY;
            xr[t] = __float_as_uint(v);
            m8[t & 7] = fmaxf(m8[t & 7], v);
          }
        }
        mx = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], fmax3(m8[5], m8[6], m8[7])));
        if (fold) mx *= c;
      }
      const float m_new = fmaxf(m_true, mx);
      m_true = m_new;
      const bool need = m_new > m_use + kRescaleThreshold;
      const bool warp_need = __any_sync(0xFFFFFFFFu, need);
      float alpha = 1.f;
      if (need) {
        alpha = ex2_approx(m_use - m_new);
        m_use = m_new;
      }
      const float msub = (m_use == -INFINITY) ? 0.f : m_use;
      float r8[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) r8[u] = 0.f;
#pragma unroll
      for (int t = 0; t < kTileN; t += 2) {
        float p0, p1;
        if (fold) {
          ffma2_bcast(p0, p1, X(t), X(t + 1), c, -msub);
        } else {
          p0 = X(t) - msub;
          p1 = X(t + 1) - msub;
        }
        p0 = ex2_approx(p0);
        p1 = ex2_approx(p1);
        fadd2_acc(r8[(t >> 1) & 3], r8[4 + ((t >> 1) & 3)], p0, p1);
        xr[t >> 1] = pack2<F16>(p0, p1);
      }
      const float rs = ((r8[0] + r8[1]) + (r8[2] + r8[3])) + ((r8[4] + r8[5]) + (r8[6] + r8[7]));
      l = l * alpha + rs;
      if (!__all_sync(0xFFFFFFFFu, p_free) &&
          !__all_sync(0xFFFFFFFFu, mbar_wait(&s.o_done[sb], ((it >> 1) - 1) & 1, a.err, kErrFwdSoftmax))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      if (it >= 1 && warp_need) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&s.o_done[sb ^ 1], ((it - 1) >> 1) & 1, a.err, kErrFwdSoftmax))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t t32[32];
          const uint32_t addr = tmem + lane_off + kColO + ch * 32;
          tmem_ld_32x32b_x32(addr, t32);
          tmem_ld_wait(t32);
#pragma unroll
          for (int t = 0; t < 32; ++t) t32[t] = __float_as_uint(__uint_as_float(t32[t]) * alpha);
          tmem_st_32x32b_x32(addr, t32);
        }
      }
      const bool s_next = it + 1 < n_kv && mbar_test(&s.s_full[sb ^ 1], ((it + 1) >> 1) & 1);
      tmem_st_32x32b_x32(tmem + lane_off + kColP + sb * 64, *reinterpret_cast<const uint32_t(*)[32]>(&xr[0]));
      tmem_st_32x32b_x32(tmem + lane_off + kColP + sb * 64 + 32, *reinterpret_cast<const uint32_t(*)[32]>(&xr[32]));
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(&s.p_full[sb]);
      s_ready = __all_sync(0xFFFFFFFFu, s_next);
    }
    if (ok && n_kv > 0) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s.o_done[(n_kv - 1) & 1], ((n_kv - 1) >> 1) & 1, a.err, kErrFwdSoftmax));
      tc_fence_after_sync();
    }
    if (ok) {
      // relative to the true maximum from here on
      const bool empty = m_true == -INFINITY;
      const float f = empty ? 0.f : ex2_approx(m_use - m_true);
      const float mul = !direct ? f : (l > 0.f || l != l ? 1.f / l : 0.f);
      const int h = w.vh * a.gs + (r - i * a.gs);
      const int64_t row = static_cast<int64_t>(w.q_start + tok0 + i) * g.N + h;
      const int64_t pr = slot_id * a.rows_pad + r;
      uint32_t acc[D / 32][32];
      if (n_kv > 0) {
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) tmem_ld_32x32b_x32(tmem + lane_off + kColO + ch * 32, acc[ch]);
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) tmem_ld_wait(acc[ch]);
      } else {
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch)
#pragma unroll
          for (int t = 0; t < 32; ++t) acc[ch][t] = 0u;
      }
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        if (ch * 32 >= g.D) break;
        float o[32];
#pragma unroll
        for (int t = 0; t < 32; ++t) o[t] = __uint_as_float(acc[ch][t]) * mul;
        if (row_valid) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const int col = ch * 32 + q4 * 8;
            if (col >= g.D) continue;
            if (!direct) {
              store8<F16>(a.part_o, pr * D + col, &o[q4 * 8], true);
            } else if (in_bounds(row * g.D + col, 8, a.n_out, a.err)) {
              store8<F16>(a.out, row * g.D + col, &o[q4 * 8], false);
            }
          }
        }
      }
      if (row_valid) {
        if (!direct) {
          a.part_ml[pr] = make_float2(m_true, l * f);
        } else if (in_bounds(row, 1, a.n_stats, a.err)) {
          if (a.smax) a.smax[row] = empty ? -INFINITY : m_true * kLn2;
          if (a.ssum) a.ssum[row] = l * f;
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool F16, int CAP>
cudaError_t launch_tile_t(const PagedArgs& a, const PagedTable<CAP>& tab, const CUtensorMap& mk, const CUtensorMap& mv,
                          cudaStream_t stream) {
  const size_t smem = sizeof(TileSmem<D>) + 1024;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit(swa_paged_tile_kernel<D, F16, CAP>, smem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(swa_paged_tile_kernel<D, F16, CAP>, dim3(tab.n_items, a.splits), dim3(kThreads), smem, stream, a,
                    tab, mk, mv);
}

}  // namespace

template <int CAP>
cudaError_t launch_paged_tile(const PagedArgs& a, const PagedTable<CAP>& tab, const CUtensorMap& mk,
                              const CUtensorMap& mv, cudaStream_t stream) {
  if (tab.n_items == 0) return cudaSuccess;
  if (a.g.D <= 64)
    return a.f16 ? launch_tile_t<64, true>(a, tab, mk, mv, stream) : launch_tile_t<64, false>(a, tab, mk, mv, stream);
  return a.f16 ? launch_tile_t<128, true>(a, tab, mk, mv, stream) : launch_tile_t<128, false>(a, tab, mk, mv, stream);
}
template cudaError_t launch_paged_tile<kPagedSmallTable>(const PagedArgs&, const PagedTable<kPagedSmallTable>&,
                                                         const CUtensorMap&, const CUtensorMap&, cudaStream_t);
template cudaError_t launch_paged_tile<kPagedLargeTable>(const PagedArgs&, const PagedTable<kPagedLargeTable>&,
                                                         const CUtensorMap&, const CUtensorMap&, cudaStream_t);

}  // namespace swa
