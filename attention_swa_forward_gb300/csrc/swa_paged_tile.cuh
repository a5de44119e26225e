// swa_paged_tile.cuh — attention of a chunk over the paged cache on the 5th-gen
// tensor cores: row tiles of 128 (tokens x the query heads that share a
// key/value head), key tiles of 128.
//
// Per row (include/swa.h): O = sum_j softmax_j(scale q.k_j) v_j over visible
// keys, softmax_max, softmax_sum; online softmax in fp32 (log2 units).  P is
// rounded to the element type, which the second product's operands have (as in
// swa_fwd.cuh; swa_paged_rows.cuh says what that does to the result).
//
// Bound by the tensor pipe and its hand-offs to the softmax, like the dense
// forward, whose roles it keeps (swa_fwd.cuh): one thread per row in warps 0-3,
// S = Q K^T into one of two TMEM tiles by the thread of warp 5, O += P V by the
// thread of warp 6 with P taken from TMEM.  What is different:
//  * Packing the G heads of a key/value head into the rows (128 / G tokens per
//    tile) reads a key tile once for all of them, fills tiles of short chunks,
//    and cuts the masked part of the tiles at the window's edges by G.
//  * One CTA per SM walks several row tiles, every ring and barrier running on
//    from one to the next: the lengths, block table entries, K, V and Q of the
//    next tile arrive while this one is computed.  (One CTA per row tile paid
//    about 7 us each for its start and end.  On the same inputs again and again:
//    prompt of 8192 tokens 430 us, then 390; 2048 tokens under a 4096 window 128,
//    then 123, and 117 with the last round's tiles split; 8192 under it 349, then
//    315.  One call among others on inputs of its own: prompt 423, 2048 tokens
//    120.)  Tiles go by falling weight, in rounds of alternating direction.
//    At a boundary the softmax warps still wait for the last product and store
//    their rows (~5000 cycles).  Handing the stores to four more warps needed
//    setmaxnreg and waits without calls, and gained nothing (392 us);
//    transposing rows by shuffles, so that a store covers 128 bytes of a row,
//    cost more than it saved (405).
//  * Warps 4 and 7 gather the K and the V tiles from pages: each lane issues one
//    TMA box (up to 128 slots x 64 columns) at the page its own block table
//    entry names, loaded two tiles ahead.  An entry that is not to be followed
//    becomes the coordinate past the last page, which TMA fills with zeros.
//    (One warp for both, waiting for its table entries one tile ahead, took
//    ~3500 cycles per tile and held everything up.)
//  * Warp 7 also fetches Q: by one box of a tensor map where q's strides suit
//    one, else row by row.
//  * A key tile at either end of the chunk's keys may hold slots that no query
//    sees (stale or never written, possibly NaN): warp 6 zeroes those rows of
//    V in shared memory, since 0 * NaN would reach O.
// Sinks: the key tiles that hold them come before those of the window, in one
// list.  A tree: the tiles that hold the chunk's own keys take 32 bits per row
// and 32 columns.  The fast path without per-column tests is as it was.
// An 8-bit cache is written out as 16-bit pages first (swa_paged_unpack.cu).
// TMEM columns as in swa_fwd.cuh: S0 [0,128), S1 [128,256), O [256,256+D),
// P0 [384,448), P1 [448,512).
#pragma once
#include "swa_paged.h"
#include "swa_device.cuh"
#include "swa_paged_mask.cuh"

namespace swa {
namespace {

constexpr int kStages = 3;
constexpr int kThreads = 256;  // (more than 8 warps would cap a thread at 168 registers: the softmax spills)

template <int D>
struct TileSmem {
  static constexpr int kTileBytes = kPagedTileRows * D * 2;
  alignas(1024) uint8_t q[kTileBytes];
  alignas(1024) uint8_t k[kStages][kTileBytes];
  alignas(1024) uint8_t v[kStages][kTileBytes];
  uint64_t q_full, q_empty, o_free, k_full[kStages], v_full[kStages], k_empty[kStages], v_empty[kStages];
  uint64_t s_full[2], s_free[2], p_full[2], o_done[2], drain_s, drain_pv;
  uint64_t never;  // completed by nothing: the target of the stall test hook
  uint32_t tmem_base;
};
static_assert(sizeof(TileSmem<128>) + 1024 <= 232448, "shared memory budget");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256, kColP = 384;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // as in swa_fwd.cuh

// Where one lane of a gathering warp finds its part of successive key tiles:
// box `box` (box_rows slots) of the tile, in atom column `atom`.
struct PageWalk {
  int entry, slot;    // block table column and first slot of the next tile's box
  int step_e, step_s;  // 128 slots on
  int j;              // its first key
  int lo, hi, sinks, box_rows, page_size, num_pages;
  int sink_tiles, run_j;  // tiles left before the window's, and the first key of the box there
  const int32_t* row;  // the sequence's block table row
  int64_t left;        // entries of the table from `row` on (bounds-checked build)
  int32_t* err;

  __device__ __forceinline__ void seek(int j_) {
    j = j_;
    entry = j / page_size;
    slot = j - entry * page_size;
  }
  // From tile number `first` of the unit list on.
  __device__ __forceinline__ void start(const PagedBase& a, int b, const PagedUnits& tiles, int first, int box,
                                        const PagedKeys& keys) {
    lo = keys.lo;
    hi = keys.hi;
    sinks = keys.sinks;
    box_rows = a.box_rows;
    page_size = a.g.page_size;
    num_pages = a.g.num_pages;
    sink_tiles = tiles.sinks - first;
    run_j = (tiles.jump + tiles.sinks) * kPagedTileStep + box * box_rows;
    seek(tiles.at(first) * kPagedTileStep + box * box_rows);
    step_e = kPagedTileStep / page_size;
    step_s = kPagedTileStep - step_e * page_size;
    row = a.g.table + b * a.g.table_stride;
    left = a.g.n_table - b * a.g.table_stride;
    err = a.err;
  }
  // The raw entry of the next tile's box and its first slot (num_pages and -1
  // when no key of it is seen), and on to the tile after.  Nothing waits for
  // the load here.
  template <bool X>
  __device__ __forceinline__ void next(bool mine, int& raw, int& at) {
    raw = num_pages;
    at = -1;
    if (mine && j <= hi && (j + box_rows > lo || (X && j < sinks))) {
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
    if (X && --sink_tiles == 0) seek(run_j);
  }
};

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// One work unit: a split of a row tile, and the key tiles it walks.
struct Unit {
  PagedItem w;
  int64_t slot_id;  // of its status and partial rows
  int split, kv_len, tok0, n_tok, n_rows;
  PagedKeys keys;    // that its rows see
  PagedUnits tiles;  // the key tiles that hold them
  int first, n_kv;   // of those, the ones of this split
  __device__ __forceinline__ int key0(int it) const { return tiles.at(first + it) * kPagedTileStep; }
  bool bad_len, direct, idle;  // idle: another split has all the keys
};

// The k-th unit of this CTA, or -1 past the last: rounds of one unit per CTA,
// every other round backwards, so that a CTA that had a heavier unit in one
// round has a lighter one in the next (units go by falling weight).
__device__ __forceinline__ int unit_index(int k, int n_units) {
  const int g = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
  const int u = k * g + ((k & 1) ? g - 1 - b : b);
  return u < n_units ? u : -1;
}

// A role's walk over the CTA's units.  The length of the next unit's sequence
// is loaded one unit ahead.
template <bool X, int CAP>
struct UnitWalk {
  int k, u_next, kv_next;
  PagedItem w_next;

  // The first `whole` units are whole items, the others splits of the rest.
  static __device__ __forceinline__ int item_of(const PagedBase& a, int u) {
    return u < a.whole ? u : (a.splits > 1 ? a.whole + (u - a.whole) / a.splits : u);
  }
  __device__ __forceinline__ void fetch(const PagedBase& a, const PagedTable<CAP>& tab, int n_units) {
    u_next = unit_index(k, n_units);
    if (u_next < 0) return;
    w_next = resolve_paged(tab, a.groups, item_of(a, u_next));
    kv_next = in_bounds(w_next.b, 1, a.g.n_lens, a.err) ? a.g.kv_lens[w_next.b] : 0;
  }
  __device__ __forceinline__ void start(const PagedBase& a, const PagedTable<CAP>& tab, int n_units) {
    k = 0;
    fetch(a, tab, n_units);
  }
  __device__ __forceinline__ bool next(const ArgsOf<X>& a, const PagedTable<CAP>& tab, int n_units, Unit& x) {
    if (u_next < 0) return false;
    const bool whole = u_next < a.whole;
    x.w = w_next;
    x.split = whole ? 0 : (u_next - a.whole) - (item_of(a, u_next) - a.whole) * a.splits;
    x.slot_id = static_cast<int64_t>(a.item_base) * a.splits + u_next;
    const int raw = kv_next;
    ++k;
    fetch(a, tab, n_units);
    x.bad_len = raw < 0 || raw > a.g.kv_limit;
    x.kv_len = x.bad_len ? 0 : raw;
    x.tok0 = x.w.tile * a.tok;
    x.n_tok = min(a.tok, x.w.q_len - x.tok0);
    x.n_rows = x.n_tok * a.gs;
    x.keys = paged_keys<X>(a, x.kv_len, x.w.q_len, x.tok0, x.n_tok);
    x.tiles = paged_units<X>(x.keys, 7);
    const int steps = x.tiles.total;
    int st0, st1, active;
    if (whole) {
      st0 = 0;
      st1 = steps;
      active = 1;
    } else {
      paged_split(steps, a.par, a.cap, a.least, x.split, &st0, &st1, &active);
    }
    x.direct = active <= 1;
    x.idle = x.split > 0 && x.split >= active;
    x.first = st0;
    x.n_kv = st1 - st0;
    return true;
  }
};

// Position in a ring of kStages: stage, and the parity of its current use.
struct Ring {
  int st = 0;
  uint32_t use = 0;  // times the ring has wrapped
  __device__ __forceinline__ void advance() {
    if (++st == kStages) {
      st = 0;
      ++use;
    }
  }
};

template <PagedKind KIND, int D, bool F16, int CAP>
__global__ void __launch_bounds__(kThreads, 1)
    swa_paged_tile_kernel(const __grid_constant__ ArgsOf<KIND != PagedKind::kPlain> a, const __grid_constant__ PagedTable<CAP> tab,
                          const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                          const __grid_constant__ CUtensorMap mq) {
  extern __shared__ uint8_t smem_raw[];
  constexpr bool X = KIND != PagedKind::kPlain;
  TileSmem<D>& s = *reinterpret_cast<TileSmem<D>*>(align1024(smem_raw));
  constexpr int kTileBytes = TileSmem<D>::kTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  // the few-row kernel of the same call may fill the SMs that this one leaves
  // (it waits for this grid at its end); nothing else starts early
  if (a.signal) griddep_launch_dependents();
  if (a.clear_err && blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  const PagedGeom& g = a.g;
  const int n_units = a.whole + (tab.n_items - a.whole) * a.splits;
  UnitWalk<X, CAP> walk;
  walk.start(a, tab, n_units);
  Unit x;

  if (warp == 4 && lane == 0) {
    mbar_init(&s.q_full, a.q_tma ? 1 : 32);
    mbar_init(&s.q_empty, 1);
    mbar_init(&s.o_free, kPagedTileRows);
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
      mbar_init(&s.o_done[i], 1);
    }
    mbar_init(&s.drain_s, 1);
    mbar_init(&s.drain_pv, 1);
    mbar_init(&s.never, 1);
    fence_mbar_init();
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
    if (a.q_tma) tma_prefetch_desc(&mq);
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
    const CUtensorMap* map = is_k ? &mk : &mv;
    const PageDims pd = is_k ? a.kd : a.vd;
    const int box = lane / (D / 64), atom = lane % (D / 64);  // the lane's part of a tile
    const bool mine = box < kPagedTileStep / a.box_rows;
    Ring ring;
    int issued = 0;
    uint32_t uc = 0;  // units so far (Q)
    bool ok = true;
    while (ok && walk.next(a, tab, n_units, x)) {
      int bad = x.bad_len ? kPageErrLength : 0;
      const int hk = x.w.vh * a.gs / a.group;
      PageWalk pages;
      int raw0, at0, raw1, at1;  // block table entries of this tile and the next
      pages.start(a, x.w.b, x.tiles, x.first, box, x.keys);
      pages.template next<X>(mine && x.n_kv > 0, raw0, at0);
      pages.template next<X>(mine && x.n_kv > 1, raw1, at1);
      if (!is_k && x.n_kv > 0) {
        // Q, once the last scores of the unit before have read its place (the
        // unit's first V tile is needed well after).  By one box per atom
        // column where the strides suit a tensor map; smem rows past the box
        // keep stale values, which only rows that are not stored read.
        if (uc > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(&s.q_empty, (uc - 1) & 1, a.err, kErrFwdLoad))) {
          ok = false;
          break;
        }
        if (a.q_tma) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&s.q_full, a.tok * a.gs * D * 2);
#pragma unroll
            for (int y = 0; y < D / 64; ++y)
              tma_load_3d(s.q + y * kAtomBytes, &mq, &s.q_full, y * 64, x.w.vh * a.gs, x.w.q_start + x.tok0);
          }
        } else {  // 16 bytes a lane; rows past the tile are zero
          constexpr int kChunks = D / 8, kRowsPer = 32 / kChunks;  // 16 chunks: 2 rows a step; 8: 4 rows
          const int ch = lane % kChunks;
          for (int rr = lane / kChunks; rr < kPagedTileRows; rr += kRowsPer) {
            const int ii = row_token(rr, a.gs_magic);
            const int64_t e = static_cast<int64_t>(x.w.q_start + x.tok0 + ii) * a.q_row +
                              static_cast<int64_t>(x.w.vh * a.gs + rr - ii * a.gs) * a.q_head + ch * 8;
            const bool in = rr < x.n_rows && ch * 8 < g.D && in_bounds(e, 8, a.n_q, a.err);
            const uint16_t* src = static_cast<const uint16_t*>(a.q) + (in ? e : 0);
            const uint32_t dst = smem_u32(s.q) + (ch >> 3) * kAtomBytes + rr * 128 + (((ch ^ rr) & 7) << 4);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
                         : "memory");
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_proxy_async_smem();
          mbar_arrive(&s.q_full);
        }
        ++uc;
      }
      for (int it = 0; it < x.n_kv; ++it) {
        if (ring.use > 0 &&
            !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[ring.st], (ring.use - 1) & 1, a.err, kErrFwdLoad))) {
          ok = false;
          break;
        }
        // an entry that must not be followed becomes the page past the last
        int page = raw0;
        if (page < 0 || page > g.num_pages || (page == g.num_pages && at0 >= 0)) {
          bad = max(bad, static_cast<int>(kPageErrEntry));
          page = g.num_pages;
        }
        const int slot = max(at0, 0);
        if (lane == 0) mbar_arrive_expect_tx(&full[ring.st], kTileBytes);
        __syncwarp();
        if (mine) {
          const int c1 = pd.slot_at == 1 ? slot : (pd.head_at == 1 ? hk : page);
          const int c2 = pd.slot_at == 2 ? slot : (pd.head_at == 2 ? hk : page);
          const int c3 = pd.slot_at == 3 ? slot : (pd.head_at == 3 ? hk : page);
          tma_load_4d((is_k ? s.k[ring.st] : s.v[ring.st]) + atom * kAtomBytes + box * a.box_rows * 128, map,
                      &full[ring.st], atom * 64, c1, c2, c3);
        }
        ++issued;
        ring.advance();
        raw0 = raw1;
        at0 = at1;
        pages.template next<X>(mine && it + 2 < x.n_kv, raw1, at1);
      }
      bad = __reduce_max_sync(0xFFFFFFFFu, bad);
      if (is_k && lane == 0) a.page_err[x.slot_id] = bad;
    }
    if (lane == 0) {  // every copy issued has landed before the CTA may exit
      for (int st = 0; st < kStages; ++st) {
        const int uses = (issued - st + kStages - 1) / kStages;
        if (uses > 0) mbar_wait_drain(&full[st], (uses - 1) & 1);
      }
      if (uc > 0 && a.q_tma) mbar_wait_drain(&s.q_full, (uc - 1) & 1);
    }
  } else if (warp == 5) {
    // ------------------------------------------------ S = Q K^T issuer --
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_f16_f32(kTileM, kTileN, false, false, F16);
      const uint64_t dq_ = sdesc_sw128(smem_u32(s.q), 16, 1024);
      const int nk = (g.D + 15) >> 4;
      Ring ring;
      uint32_t uc = 0, t = 0;  // units, tiles so far
      bool ok = true;
      while (ok && walk.next(a, tab, n_units, x)) {
        if (x.n_kv == 0) continue;
        ok = mbar_wait(&s.q_full, uc & 1, a.err, kErrFwdMma);
        for (int it = 0; ok && it < x.n_kv; ++it) {
          const uint32_t sb = t & 1;
          ok = (t < 2 || mbar_wait(&s.s_free[sb], ((t >> 1) - 1) & 1, a.err, kErrFwdMma)) &&
               mbar_wait(&s.k_full[ring.st], ring.use & 1, a.err, kErrFwdMma);
          if (!ok) break;
          tc_fence_after_sync();
          const uint64_t dk_ = sdesc_sw128(smem_u32(s.k[ring.st]), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            if (kk >= nk) break;
            const uint32_t off = (kk >> 2) * kAtomBytes + (kk & 3) * 32;
            umma_bf16_ss(tmem + sb * kTileN, sdesc_advance(dq_, off), sdesc_advance(dk_, off), kIdS, kk > 0);
          }
          umma_commit(&s.s_full[sb]);
          umma_commit(&s.k_empty[ring.st]);
          ring.advance();
          ++t;
        }
        if (ok) umma_commit(&s.q_empty);
        ++uc;
      }
      umma_commit(&s.drain_s);
      mbar_wait_drain(&s.drain_s, 0);
    }
  } else if (warp == 6) {
    // ------------------------------------------------- O += P V issuer --
    constexpr uint32_t kIdO = idesc_f16_f32(kTileM, D, false, true, F16);
    Ring ring;
    uint32_t uc = 0, t = 0;
    bool ok = true;
    while (ok && walk.next(a, tab, n_units, x)) {
      if (x.n_kv == 0) continue;
      const PagedKeys seen = paged_keys<X>(a, x.kv_len, x.w.q_len, 0, x.w.q_len);
      for (int it = 0; it < x.n_kv; ++it) {
        const uint32_t pb = t & 1;
        const int j0 = x.key0(it);
        if ((j0 < seen.lo && !(X && j0 + kPagedTileStep - 1 < seen.sinks)) || j0 + kPagedTileStep - 1 > seen.hi) {
          // rows of V that no query of the chunk sees
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&s.v_full[ring.st], ring.use & 1, a.err, kErrFwdMma))) {
            ok = false;
            break;
          }
          const int sink_rows = X ? min(max(seen.sinks - j0, 0), kPagedTileStep) : 0;
          const int head_rows = min(max(seen.lo - j0, 0), kPagedTileStep) - sink_rows;
          const int tail_at = min(seen.hi - j0 + 1, kPagedTileStep);
          const int dead = head_rows + kPagedTileStep - tail_at;
          for (int y = lane; y < dead * (D / 8); y += 32) {
            const int d = y / (D / 8), c = y % (D / 8);
            const int r = d < head_rows ? sink_rows + d : tail_at + (d - head_rows);
            *reinterpret_cast<uint4*>(s.v[ring.st] + (c >> 3) * kAtomBytes + r * 128 + (c & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          // O may be overwritten once the rows of the unit before are in registers
          ok = mbar_wait(&s.p_full[pb], (t >> 1) & 1, a.err, kErrFwdMma) &&
               (it > 0 || uc == 0 || mbar_wait(&s.o_free, (uc - 1) & 1, a.err, kErrFwdMma)) &&
               mbar_wait(&s.v_full[ring.st], ring.use & 1, a.err, kErrFwdMma);
          if (ok) {
            tc_fence_after_sync();
            const uint64_t dv_ = sdesc_sw128(smem_u32(s.v[ring.st]), kAtomBytes, 1024);
#pragma unroll
            for (int kk = 0; kk < kTileN / 16; ++kk)  // O += P V  (A = P in TMEM)
              umma_bf16_ts(tmem + kColO, tmem + kColP + pb * 64 + kk * 8, sdesc_advance(dv_, kk * 2048), kIdO,
                           (it > 0 || kk > 0) ? 1u : 0u);
            umma_commit(&s.o_done[pb]);
            umma_commit(&s.v_empty[ring.st]);
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        ring.advance();
        ++t;
      }
      ++uc;
    }
    if (lane == 0) {
      umma_commit(&s.drain_pv);
      mbar_wait_drain(&s.drain_pv, 0);
    }
  } else {
    // ------------------------------------------ softmax + epilogue (rows) --
    const int r = threadIdx.x;  // 0..127 == TMEM lane
    const int i = row_token(r, a.gs_magic);  // token of the tile
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const float c = a.scale_log2;
    const bool fold = c > 0.f;
    bool ok = true;
    if (a.stall & kStallPaged)  // test hook: a wait that nothing completes
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s.never, 0, a.err, kErrFwdSoftmax));
    uint32_t t = 0;  // tiles so far
    bool more = walk.next(a, tab, n_units, x), more_after;
    Unit after;  // formed while the last product of this unit runs
    for (; ok && more; x = after, more = more_after) {
      // A unit begins with instructions of the whole warp (tensor memory loads and
      // stores): lanes of rows past the last tile's, which stored nothing, wait
      // here for the others.
      __syncwarp();
      if (x.idle) {
        more_after = walk.next(a, tab, n_units, after);
        continue;
      }
      const bool row_valid = r < x.n_rows;
      int wlo = 0, whi = x.kv_len - 1;
      // keys every valid row sees: from the last token's first to the first token's last
      int all_lo = 0, all_hi = x.kv_len - 1;
      if (a.sparse_mode == 4) {
        const int p0 = x.kv_len - x.w.q_len + x.tok0;
        const int p = X ? token_position<X>(a, x.w, x.kv_len, x.tok0 + min(i, x.n_tok - 1)) : p0 + i;
        wlo = max(0, p - a.pre);
        whi = min(x.kv_len - 1, p + a.next);
        all_lo = max(0, p0 + x.n_tok - 1 - a.pre);
        all_hi = min(x.kv_len - 1, p0 + a.next);
      }
      const int prefix = x.kv_len - x.w.q_len;  // a tree: keys before the chunk, whose own go by bits
      if (tree_of<X>(a)) {
        whi = all_hi = prefix - 1;
        if (a.sparse_mode == 4) all_lo = max(0, x.kv_len - 1 - a.pre);  // the deepest token may be q_len - 1 deep
      }
      if (!row_valid) {
        wlo = 0;
        whi = -1;
      }
      float m_use = -INFINITY, m_true = -INFINITY, l = 0.f;
      bool s_ready = false;  // S(t) known complete from a probe issued during the previous tile
      for (int it = 0; it < x.n_kv; ++it, ++t) {
        const uint32_t sb = t & 1;
        if (!s_ready && !__all_sync(0xFFFFFFFFu, mbar_wait(&s.s_full[sb], (t >> 1) & 1, a.err, kErrFwdSoftmax))) {
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
        const bool p_free = t < 2 || mbar_test(&s.o_done[sb], ((t >> 1) - 1) & 1);
        auto score = [&](int y) -> float { return __uint_as_float(xr[y]); };

        const int j0 = x.key0(it);
        const bool fast = fold && (j0 >= all_lo || (X && j0 + kPagedTileStep - 1 < sinks_of<X>(a))) &&
                          j0 + kPagedTileStep - 1 <= all_hi;
        float mx;
        {
          float m8[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) m8[u] = -INFINITY;
          if (!fast) {
            // visible columns as bits: one test and one select per score
            uint32_t seen[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int a0 = wlo - j0 - 32 * q, b0 = whi - j0 - 32 * q;  // columns [a0, b0] of this word
              const uint32_t from = a0 <= 0 ? ~0u : (a0 > 31 ? 0u : ~0u << a0);
              const uint32_t to = b0 >= 31 ? ~0u : (b0 < 0 ? 0u : (2u << b0) - 1u);
              seen[q] = from & to;
              if constexpr (X) {
                // and the sinks, up to the row's last key
                const int n = min(a.sinks, whi + 1) - j0 - 32 * q;
                seen[q] |= n <= 0 ? 0u : (n > 31 ? ~0u : (1u << n) - 1u);
                if (a.tree && row_valid) seen[q] |= tree_bits(a, x.w, x.tok0 + i, j0 + 32 * q - prefix);
              }
            }
            if (!fold) {
#pragma unroll
              for (int y = 0; y < kTileN; ++y) xr[y] = __float_as_uint(score(y) * c);
            }
#pragma unroll
            for (int y = 0; y < kTileN; ++y)
              xr[y] = (seen[y >> 5] & (1u << (y & 31))) ? xr[y] : __float_as_uint(-INFINITY);
          }
#pragma unroll
          for (int y = 0; y < kTileN; y += 2) m8[(y >> 1) & 7] = fmax3(m8[(y >> 1) & 7], score(y), score(y + 1));
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
        for (int y = 0; y < kTileN; y += 2) {
          float p0, p1;
          if (fold) {
            ffma2_bcast(p0, p1, score(y), score(y + 1), c, -msub);
          } else {
            p0 = score(y) - msub;
            p1 = score(y + 1) - msub;
          }
          p0 = ex2_approx(p0);
          p1 = ex2_approx(p1);
          fadd2_acc(r8[(y >> 1) & 3], r8[4 + ((y >> 1) & 3)], p0, p1);
          xr[y >> 1] = pack2<F16>(p0, p1);
        }
        const float rs = ((r8[0] + r8[1]) + (r8[2] + r8[3])) + ((r8[4] + r8[5]) + (r8[6] + r8[7]));
        l = l * alpha + rs;
        if (!__all_sync(0xFFFFFFFFu, p_free) &&
            !__all_sync(0xFFFFFFFFu, mbar_wait(&s.o_done[sb], ((t >> 1) - 1) & 1, a.err, kErrFwdSoftmax))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        if (it >= 1 && warp_need) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&s.o_done[sb ^ 1], ((t - 1) >> 1) & 1, a.err, kErrFwdSoftmax))) {
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
            for (int y = 0; y < 32; ++y) t32[y] = __float_as_uint(__uint_as_float(t32[y]) * alpha);
            tmem_st_32x32b_x32(addr, t32);
          }
        }
        const bool s_next = it + 1 < x.n_kv && mbar_test(&s.s_full[sb ^ 1], ((t + 1) >> 1) & 1);
        tmem_st_32x32b_x32(tmem + lane_off + kColP + sb * 64, *reinterpret_cast<const uint32_t(*)[32]>(&xr[0]));
        tmem_st_32x32b_x32(tmem + lane_off + kColP + sb * 64 + 32, *reinterpret_cast<const uint32_t(*)[32]>(&xr[32]));
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&s.p_full[sb]);
        s_ready = __all_sync(0xFFFFFFFFu, s_next);
      }
      if (!ok) break;
      more_after = walk.next(a, tab, n_units, after);
      uint32_t acc[D / 32][32];
      if (x.n_kv > 0) {
        if (!__all_sync(0xFFFFFFFFu,
                        mbar_wait(&s.o_done[(t - 1) & 1], ((t - 1) >> 1) & 1, a.err, kErrFwdSoftmax))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) tmem_ld_32x32b_x32(tmem + lane_off + kColO + ch * 32, acc[ch]);
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) tmem_ld_wait(acc[ch]);
        tc_fence_before_sync();
        mbar_arrive(&s.o_free);
      } else {
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch)
#pragma unroll
          for (int y = 0; y < 32; ++y) acc[ch][y] = 0u;
      }
      if (!row_valid) continue;
      // relative to the true maximum from here on
      const bool empty = m_true == -INFINITY;
      const float f = empty ? 0.f : ex2_approx(m_use - m_true);
      const float mul = !x.direct ? f : (l > 0.f || l != l ? 1.f / l : 0.f);
      const int h = x.w.vh * a.gs + (r - i * a.gs);
      const int64_t row = static_cast<int64_t>(x.w.q_start + x.tok0 + i) * g.N + h;
      const int64_t pr = (x.slot_id - a.whole) * a.rows_pad + r;
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        if (ch * 32 >= g.D) break;
        float o[32];
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] = __uint_as_float(acc[ch][y]) * mul;
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          const int col = ch * 32 + q4 * 8;
          if (col >= g.D) continue;
          if (!x.direct) {
            store8<F16>(a.part_o, pr * D + col, &o[q4 * 8], true);
          } else if (in_bounds(row * g.D + col, 8, a.n_out, a.err)) {
            store8<F16>(a.out, row * g.D + col, &o[q4 * 8], false);
          }
        }
      }
      if (!x.direct) {
        a.part_ml[pr] = make_float2(m_true, l * f);
      } else if (in_bounds(row, 1, a.n_stats, a.err)) {
        if (a.smax) a.smax[row] = empty ? -INFINITY : m_true * kLn2;
        if (a.ssum) a.ssum[row] = l * f;
      }
    }
  }
  __syncwarp();  // (the roles of one lane: its warp waits here, not inside the barrier)
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <PagedKind KIND, int D, bool F16, int CAP>
cudaError_t launch_tile_t(const ArgsOf<KIND != PagedKind::kPlain>& a, const PagedTable<CAP>& tab, const CUtensorMap& mk, const CUtensorMap& mv,
                          const CUtensorMap& mq, cudaStream_t stream) {
  const size_t smem = sizeof(TileSmem<D>) + 1024;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit(swa_paged_tile_kernel<KIND, D, F16, CAP>, smem, smem_set);
  if (e != cudaSuccess) return e;
  const int units = a.whole + (tab.n_items - a.whole) * a.splits;
  return launch_pdl(swa_paged_tile_kernel<KIND, D, F16, CAP>, dim3(units < kSms ? units : kSms), dim3(kThreads), smem,
                    stream, a, tab, mk, mv, mq);
}

}  // namespace

template <PagedKind KIND, int CAP>
cudaError_t launch_paged_tile(const PagedArgs& a, const PagedTable<CAP>& tab, const CUtensorMap& mk,
                              const CUtensorMap& mv, const CUtensorMap& mq, cudaStream_t stream) {
  if (tab.n_items == 0) return cudaSuccess;
  if (a.g.D <= 64)
    return a.f16 ? launch_tile_t<KIND, 64, true>(a, tab, mk, mv, mq, stream)
                 : launch_tile_t<KIND, 64, false>(a, tab, mk, mv, mq, stream);
  return a.f16 ? launch_tile_t<KIND, 128, true>(a, tab, mk, mv, mq, stream)
               : launch_tile_t<KIND, 128, false>(a, tab, mk, mv, mq, stream);
}

}  // namespace swa
