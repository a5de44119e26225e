// swa_paged_rows_e4m3.cu — attention of a few query rows per sequence and
// key/value head over the 8-bit paged cache, with sinks and trees.
//
// The same work as swa_paged_rows.cuh on half the bytes, so what a warp does per
// 16 keys sets the time unless it is kept short:
//  * Each warp has a ring of three groups of 16 keys (four of heads up to 64).  One
//    lane brings a group in: K and V by a TMA box each (swizzled), the exponents by
//    two copies of 16 bytes, all on one barrier.  Rows that start on 8 bytes only
//    (head dims that are no multiples of 16) are copied by all lanes, 8 bytes at a
//    time, into six of heads up to 64.
//  * The products are transposed, S^T = K Q^T and O^T = V^T P^T, with keys and
//    columns as the 16 rows of an instruction and 8 query rows as its columns: up
//    to 8 rows (a token of 8 heads) take half the instructions, exponentials and
//    registers of the other way round, and 16 warps an SM find room instead of 12.
//  * Codes go from shared memory to registers 16 bytes a thread and become fp16
//    pairs by the conversion instruction.  The sums over the head dim and over
//    the keys, and the result's columns, are taken in the order in which a thread
//    holds them: thread c of a quad has head dims c D / 4 on of two keys for the
//    scores, and D / 8 columns of four keys' values for the second product.  Only
//    P moves between threads, 8 x 8 at a time.
//  * Products are fp16 whatever the type of q, which is brought into range by a
//    power of two per row (exactly, but for bits below 2^-39 of its largest).  The
//    exponent of a key multiplies its scores in fp32; that of a value goes into
//    its weight, rounded to fp16 as w = p 2^e ref: 11 bits down to 2^-14, 2^-25
//    below.  The power of two `ref` is a query row's own, and so what a row gets
//    does not depend on values that it does not see or gives no weight: it is
//    brought down, and the row's result with it, where a weight passes 2^15, to
//    leave the largest at 2^6 or more (at first it is the most that some row may
//    need: a weight of 1 on the least exponent).  The running maximum moves in
//    whole powers of two, and the weights' scale against them, so that weights are
//    as they were.  A lane makes the factor of one of the 32 exponents.
// Bound by HBM where the keys are many: 64 tokens of 100 to 16384 keys, 32 / 8
// heads of 128, 199 us (1.13 GB; a copy would take 166), of 8192 keys each 181.
// (Measured on the first of those on the way here: codes as bf16, by moving bits
// with integer instructions and multiplying each pair by its row's power of two,
// 765 instructions a group, 448 us; as fp16 394; by TMA instead of copies by all
// lanes 317; transposed, and in shorter runs of keys, 196; with `ref` a row's own instead of
// one for all that the warp has seen, 199.)
#include "swa_paged_rows_end.cuh"

#include <cfloat>

namespace swa {
namespace {

// CTAs an SM, as registers and shared memory allow.  64 tokens of 100 to 16384
// keys, 8 key/value heads, 16 rows: heads of 128 285 us with 3, 312 with 2, 427
// (spills) with 4; of 64 191 with 4, 250 with 2; 8 rows, heads of 64: 144 with 6,
// 149 with 4.  Clusters are few CTAs, and spills would cost them time; copies by
// all lanes want more stages instead (heads of 40: 162 us, 186 with 6 CTAs).
template <int DP, int NB, bool WIDE, bool CL>
constexpr int rows8_ctas() {
  if (!WIDE || CL) return NB == 1 ? 4 : 2;
  return DP == 64 ? (NB == 1 ? 6 : 4) : (NB == 1 ? 4 : 3);
}
template <int DP, bool WIDE>
struct Rows8Smem {
  static constexpr int kStages = DP == 128 ? 3 : (WIDE ? 4 : 6);
  static constexpr int kGroupBytes = 16 * DP;
  alignas(1024) uint8_t ring[kRowsWarps][kStages][2][kGroupBytes];
  alignas(16) int8_t exps[kRowsWarps][kStages][2][16];
  uint64_t full[kRowsWarps][kStages];
  float ml[kRowsWarps][kRowsTile][2];
  static_assert(RowsEnd<DP>::kBytes <= kRowsWarps * kStages * 2 * kGroupBytes, "join space");
};

__device__ __align__(16) const int8_t kNoExponents[16] = {0};  // of a page that is not followed

__device__ __forceinline__ void bulk_load16(void* dst, const void* src, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 16, [%2];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}
// An arrival on the barrier once the thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Where 16-byte chunk c of row r lies (the swizzles of 128 and of 64 bytes).
template <int DP>
__device__ __forceinline__ int place(int r, int c) {
  return r * DP + ((c ^ (DP == 128 ? r & 7 : (r >> 1) & 3)) << 4);
}

// A weight is p 2^e ref with p <= 2^8 and e <= kExpMost: at most 2^122.
constexpr int kRefMost = 7 - kExpLeastBf16;
constexpr float kWeightMost = 32768.f;  // (fp16 holds twice that)
// The power of two that x > 0 begins with.
__device__ __forceinline__ int pow2_exponent(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 127; }

// The transpose of an 8 x 8 matrix of 16-bit elements, a row's pair a thread.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// WIDE: rows of the cache start on 16 bytes, and TMA brings them in.  NB: blocks
// of 8 query rows.
template <int DP, int NB, bool WIDE, bool CL, int CAP>
__global__ void __launch_bounds__(kRowsThreads, (rows8_ctas<DP, NB, WIDE, CL>()))
    swa_paged_rows_e4m3_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedTable<CAP> tab,
                               const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using Smem = Rows8Smem<DP, WIDE>;
  constexpr int kStages = Smem::kStages;
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(align1024(smem_raw));
  const PagedGeom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = lane >> 2, quad = lane & 3;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&s.full[warp][i], WIDE ? 1 : 32);
    fence_mbar_init();
    if (WIDE) {
      tma_prefetch_desc(&mk);
      tma_prefetch_desc(&mv);
    }
  }
  __syncwarp();
  if (a.overlap) __threadfence();  // (swa_paged_rows.cuh)
  else griddep_wait();
  griddep_launch_dependents();
  const PagedItem w = resolve_paged(tab, a.groups, static_cast<int>(blockIdx.x));
  const int split = blockIdx.y;
  if (a.clear_err && blockIdx.x == 0 && split == 0 && threadIdx.x == 0) *a.err = 0;
  const int64_t item = a.item_base + static_cast<int64_t>(blockIdx.x);
  const int tok0 = w.tile * a.tok;
  const int n_tok = min(a.tok, w.q_len - tok0), n_rows = n_tok * a.gs;
  const int kv_raw = in_bounds(w.b, 1, g.n_lens, a.err) ? g.kv_lens[w.b] : 0;  // in flight behind the loads of Q

  // Q as B fragments: head dims quad DP / 4 + 4 kk .. + 3 of row 8 x + lane / 4
  uint32_t qf[NB][DP / 16][2];
#pragma unroll
  for (int x = 0; x < NB; ++x) {
    const int r = row + 8 * x;
    const bool valid = r < n_rows;
    const int i = valid ? row_token(r, a.gs_magic) : 0;
    const int h = w.vh * a.gs + (r - i * a.gs);
    const int64_t e = static_cast<int64_t>(w.q_start + tok0 + i) * a.q_row + h * a.q_head;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + e;
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      const int c = quad * (DP / 4) + kk * 4;
      const uint2 d = valid && c < g.D && in_bounds(e + c, 4, a.n_q, a.err) ? *reinterpret_cast<const uint2*>(q + c)
                                                                            : make_uint2(0u, 0u);
      qf[x][kk][0] = d.x;
      qf[x][kk][1] = d.y;
    }
  }
  // the scale of the thread's query rows 8 x + 2 quad + y, with what they were divided by
  float c_row[NB][2];
#pragma unroll
  for (int x = 0; x < NB; ++x) c_row[x][0] = c_row[x][1] = a.scale_log2;
  if (!a.f16) {
#pragma unroll
    for (int x = 0; x < NB; ++x) {
      uint32_t top = 0;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          top = max(top, max(qf[x][kk][y] << 16 & 0x7FFFFFFFu, qf[x][kk][y] & 0x7FFF0000u));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const int sh = row_shift(top);
      const float down = pow2(-sh), up = pow2(sh);
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          qf[x][kk][y] = pack2<true>(__uint_as_float(qf[x][kk][y] << 16) * up,
                                     __uint_as_float(qf[x][kk][y] & 0xFFFF0000u) * up);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        // a positive scale stays one, and a number: 2^-126 of any score is nothing, and 0 or infinity would make NaN
        // of a masked score or of one of 0
        const float c = a.scale_log2 * __shfl_sync(0xFFFFFFFFu, down, (2 * quad + y) * 4);
        c_row[x][y] = fminf(fmaxf(c, a.scale_log2 > 0.f ? FLT_MIN : -FLT_MAX), FLT_MAX);
      }
    }
  }

  int bad = 0;
  int kv_len = kv_raw;
  if (kv_len < 0 || kv_len > g.kv_limit) {
    bad = kPageErrLength;
    kv_len = 0;
  }
  const PagedKeys keys = paged_keys<true>(a, kv_len, w.q_len, tok0, n_tok);
  const PagedUnits groups = paged_units<true>(keys, 4);
  const int steps = (groups.total + kRowsWarps - 1) / kRowsWarps;
  int st0, st1, active;
  paged_split(steps, a.par, a.cap, a.least, split, &st0, &st1, &active);
  const bool direct = active <= 1;  // no other CTA has keys of this item: write the result itself
  if (!CL && split > 0 && split >= active) {  // nothing to do (split 0 writes the result of an empty item)
    if (threadIdx.x == 0) a.page_err[item * a.splits + split] = 0;
    return;
  }

  // keys that the thread's rows see, and that every row of the tile sees (swa_paged_rows.cuh).  Those of 16 rows, whose
  // registers are all taken, are formed where they are needed, at the ends of what is seen (draft of 4 tokens,
  // 32 / 8 heads of 128: 285 us, 312 with them kept; one token of 1003 keys 7.7, 7.9 formed there).
  const int prefix = kv_len - w.q_len;
  int row_lo[NB][2], row_hi[NB][2], row_tok[NB][2], all_lo = 0, all_hi = kv_len - 1;
  auto row_keys = [&](int x, int y) {
    const int r = 8 * x + 2 * quad + y;
    row_tok[x][y] = tok0 + (r < n_rows ? row_token(r, a.gs_magic) : 0);
    row_lo[x][y] = 0;
    row_hi[x][y] = kv_len - 1;
    if (a.sparse_mode == 4) {
      const int p = token_position(a, w, kv_len, row_tok[x][y]);
      row_lo[x][y] = max(0, p - a.pre);
      row_hi[x][y] = min(kv_len - 1, p + a.next);
    }
    if (a.tree) row_hi[x][y] = prefix - 1;
  };
  if constexpr (NB == 1) {
    row_keys(0, 0);
    row_keys(0, 1);
  }
  if (a.sparse_mode == 4) {
    all_lo = max(0, (a.tree ? kv_len - 1 : prefix + tok0 + n_tok - 1) - a.pre);
    all_hi = min(kv_len - 1, prefix + tok0 + a.next);
  }
  if (a.tree) all_hi = prefix - 1;

  const int hk = w.vh * a.gs / a.group;
  const int n_it = st1 - st0;  // the warp's groups: number (st0 + it) * 4 + warp
  const int gw = st0 * kRowsWarps + warp;
  auto first_key = [&](int it) { return groups.at(gw + it * kRowsWarps) * 16; };
  auto some_see = [&](int j) { return (j >= keys.lo || j < keys.sinks) && j <= keys.hi; };

  // page number and first slot of the warp's next 32 groups, one per lane
  int my_page = 0, my_slot = 0;
  auto fetch_pages = [&](int it0) {
    const int j = first_key(it0 + lane);
    my_page = g.num_pages;  // (past the last: TMA fills with zeros)
    my_slot = 0;
    if (it0 + lane < n_it && j <= keys.hi) {
      const int entry = j / g.page_size;
      my_slot = j - entry * g.page_size;
      const int64_t e = w.b * g.table_stride + entry;
      const int page = in_bounds(e, 1, g.n_table, a.err) ? g.table[e] : -1;
      if (page >= 0 && page < g.num_pages) my_page = page;
      else bad = kPageErrEntry;
    }
  };
  // The copies of the warp's group `it`; nothing past the last.
  auto issue = [&](int it) {
    if ((it & 31) == 0) fetch_pages(it);
    const int page = __shfl_sync(0xFFFFFFFFu, my_page, it & 31), slot = __shfl_sync(0xFFFFFFFFu, my_slot, it & 31);
    if (it >= n_it) return;
    const int st = it % kStages;
    const int64_t e = static_cast<int64_t>(page) * a.ex.page + hk * g.page_size + slot;
    if constexpr (WIDE) {
      if (lane == 0) {
        uint64_t* bar = &s.full[warp][st];
        mbar_arrive_expect_tx(bar, 2 * Smem::kGroupBytes + 32);
        auto at = [&](const PageDims& d, int dim) { return d.slot_at == dim ? slot : (d.head_at == dim ? hk : page); };
        tma_load_4d(s.ring[warp][st][0], &mk, bar, 0, at(a.kd, 1), at(a.kd, 2), at(a.kd, 3));
        tma_load_4d(s.ring[warp][st][1], &mv, bar, 0, at(a.vd, 1), at(a.vd, 2), at(a.vd, 3));
        const bool in = page < g.num_pages && in_bounds(e, 16, a.ex.n, a.err);
        bulk_load16(s.exps[warp][st][0], in ? a.ex.k + e : kNoExponents, bar);
        bulk_load16(s.exps[warp][st][1], in ? a.ex.v + e : kNoExponents, bar);
      }
    } else {
      // two lanes a row, 8 bytes at a time
      const int r = lane >> 1, half = lane & 1, j = first_key(it) + r;
      const bool ok = page < g.num_pages && some_see(j);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint8_t* base = static_cast<const uint8_t*>(v ? a.v_pages : a.k_pages);
        const int64_t e0 = hk * (v ? g.v_head : g.k_head) + page * (v ? g.v_page : g.k_page) +
                           (slot + r) * (v ? g.v_slot : g.k_slot);
        const uint32_t dst = smem_u32(s.ring[warp][st][v]);
#pragma unroll
        for (int y = 0; y < DP / 16; ++y) {
          const int c = 2 * y + half;  // of 8 codes
          const bool in = ok && c * 8 < g.D && in_bounds(e0 + c * 8, 8, v ? g.n_v : g.n_k, a.err);
          cp_async8(dst + place<DP>(r, y) + half * 8, in ? base + e0 + c * 8 : base, in);
        }
      }
      if (lane < 4) {  // exponents: 8 of K, 8 of K, 8 of V, 8 of V
        const int8_t* exps = lane < 2 ? a.ex.k : a.ex.v;
        const bool in = page < g.num_pages && in_bounds(e + half * 8, 8, a.ex.n, a.err);
        cp_async8(smem_u32(s.exps[warp][st][lane >> 1] + half * 8), in ? exps + e + half * 8 : exps, in);
      }
      cp_async_arrive(&s.full[warp][st]);
    }
  };

  // O^T: element (column (lane / 4) DP / 8 + t, row 8 x + 2 quad + y) is o[x][t / 2][2 (t mod 2) + y]
  float o[NB][DP / 16][4];
#pragma unroll
  for (int x = 0; x < NB; ++x)
#pragma unroll
    for (int t = 0; t < DP / 16; ++t)
#pragma unroll
      for (int y = 0; y < 4; ++y) o[x][t][y] = 0.f;
  float m[NB][2], m_true[NB][2], l[NB][2];
#pragma unroll
  for (int x = 0; x < NB; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      m[x][y] = m_true[x][y] = -INFINITY;
      l[x][y] = 0.f;
    }
  float ref[NB][2];  // of the weights
#pragma unroll
  for (int x = 0; x < NB; ++x) ref[x][0] = ref[x][1] = pow2(kRefMost);
  const int least = a.f16 ? kExpLeastF16 : kExpLeastBf16;  // an exponent below it counts as it
  const bool fold = a.scale_log2 > 0.f;  // the scale folds into the exponent's multiply-add

#pragma unroll 1
  for (int it = 0; it < kStages; ++it) issue(it);
  int done = 0;  // groups that have landed
#pragma unroll 1
  for (int it = 0; it < n_it; ++it) {
    const int st = it % kStages;
    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&s.full[warp][st], (it / kStages) & 1, a.err, kErrFwdLoad))) break;
    ++done;
    const int j0 = first_key(it);
    const uint32_t kd = smem_u32(s.ring[warp][st][0]), vd = smem_u32(s.ring[warp][st][1]);
    uint32_t kw[2][DP / 16];     // DP / 4 codes of keys lane / 4 and lane / 4 + 8
    uint32_t vw[4][DP / 32];     // DP / 8 codes of keys 2 quad + {0, 1, 8, 9}
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int x = 0; x < DP / 64; ++x) {
        const uint4 v = lds128(kd + place<DP>(row + 8 * t, quad * (DP / 64) + x));
        kw[t][4 * x] = v.x;
        kw[t][4 * x + 1] = v.y;
        kw[t][4 * x + 2] = v.z;
        kw[t][4 * x + 3] = v.w;
      }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = 2 * quad + (t & 1) + 8 * (t >> 1);
      if constexpr (DP == 128) {
        const uint4 v = lds128(vd + place<DP>(r, row));
        vw[t][0] = v.x;
        vw[t][1] = v.y;
        vw[t][2] = v.z;
        vw[t][3] = v.w;
      } else {
        const uint2 v = lds64(vd + place<DP>(r, row >> 1) + (row & 1) * 8);
        vw[t][0] = v.x;
        vw[t][1] = v.y;
      }
    }
    // lanes 0-15: of the keys; 16-31: of the values
    int e = max(lds_s8(smem_u32(s.exps[warp][st][0]) + lane), least);
    __syncwarp();
    issue(it + kStages);  // the stage is free
    // what slots that no row sees hold counts for nothing, a NaN's code and exponent neither
    if (j0 < keys.lo || j0 + 15 > keys.hi) {
      if (!some_see(j0 + (lane & 15))) e = least;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const bool seen = some_see(j0 + 2 * quad + (t & 1) + 8 * (t >> 1));
#pragma unroll
        for (int x = 0; x < DP / 32; ++x) vw[t][x] = seen ? vw[t][x] : 0u;
      }
    }
    // of the scores' keys lane / 4 and lane / 4 + 8
    const float factor = exp_f32(e);
    float kf[2], vf[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      kf[t] = __shfl_sync(0xFFFFFFFFu, factor, row + 8 * t);
      vf[t] = __shfl_sync(0xFFFFFFFFu, factor, row + 8 * t + 16);
    }
    float sc[NB][4];  // S^T: (key lane / 4 + 8 t, row 8 x + 2 quad + y) is sc[x][2 t + y]
    {
      float s2[2][NB][4];  // two chains each
#pragma unroll
      for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int z = 0; z < 4; ++z) s2[0][x][z] = s2[1][x][z] = 0.f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        const uint32_t k[4] = {codes_f16(kw[0][kk]), codes_f16(kw[1][kk]), codes_f16(kw[0][kk] >> 16),
                               codes_f16(kw[1][kk] >> 16)};
#pragma unroll
        for (int x = 0; x < NB; ++x) mma16816<true>(s2[kk & 1][x], k, qf[x][kk][0], qf[x][kk][1]);
      }
#pragma unroll
      for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int z = 0; z < 4; ++z) sc[x][z] = (s2[0][x][z] + s2[1][x][z]) * kf[z >> 1];
    }
    if (!fold || (j0 < all_lo && j0 + 15 >= a.sinks) || j0 + 15 > all_hi) {
#pragma unroll
      for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if constexpr (NB > 1) row_keys(x, y);
          // bit t: key j0 + t is a token of the chunk that the row sees
          const uint32_t drafted = a.tree && j0 - prefix > -16 ? tree_bits(a, w, row_tok[x][y], j0 - prefix) : 0u;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int j = j0 + row + 8 * t;
            const bool vis = ((j >= row_lo[x][y] || j < a.sinks) && j <= row_hi[x][y]) || ((drafted >> (j - j0)) & 1u) != 0;
            float& z = sc[x][2 * t + y];
            z = vis ? (fold ? z : z * c_row[x][y]) : -INFINITY;
          }
        }
    }
    bool grow = false;
#pragma unroll
    for (int x = 0; x < NB; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float mx = fmaxf(sc[x][y], sc[x][2 + y]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
        m_true[x][y] = fmaxf(m_true[x][y], fold ? mx * c_row[x][y] : mx);
        grow |= m_true[x][y] > m[x][y] + kRescale;
      }
    if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
      for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          // to the next whole number (from -inf: all so far is 0)
          const float d = m_true[x][y] > m[x][y] ? ceilf(m_true[x][y]) - m[x][y] : 0.f;
          m[x][y] = d > 0.f ? ceilf(m_true[x][y]) : m[x][y];
          l[x][y] *= ex2_approx(-d);
          const int up = min(__float2int_rn(fminf(d, 256.f)), kRefMost - pow2_exponent(ref[x][y]));
          ref[x][y] *= pow2(up);
          const float f = ex2_approx(up - d);  // (1 but where ref is at its most)
#pragma unroll
          for (int t = 0; t < DP / 16; ++t) {
            o[x][t][y] *= f;
            o[x][t][2 + y] *= f;
          }
        }
    }
    float wt[NB][4], most = 0.f;  // weights of the values, as sc
#pragma unroll
    for (int x = 0; x < NB; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float ms = m[x][y] == -INFINITY ? 0.f : m[x][y], c = fold ? c_row[x][y] : 1.f;
        const float p0 = ex2_approx(fmaf(sc[x][y], c, -ms)), p1 = ex2_approx(fmaf(sc[x][2 + y], c, -ms));
        l[x][y] += p0 + p1;
        wt[x][y] = p0 * (vf[0] * ref[x][y]);
        wt[x][2 + y] = p1 * (vf[1] * ref[x][y]);
        most = fmaxf(most, fmaxf(wt[x][y], wt[x][2 + y]));
      }
    if (__any_sync(0xFFFFFFFFu, most > kWeightMost)) {
#pragma unroll
      for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float top = fmaxf(wt[x][y], wt[x][2 + y]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
          const float f = top > kWeightMost ? pow2(6 - pow2_exponent(top)) : 1.f;
          ref[x][y] *= f;
          wt[x][y] *= f;
          wt[x][2 + y] *= f;
#pragma unroll
          for (int t = 0; t < DP / 16; ++t) {
            o[x][t][y] *= f;
            o[x][t][2 + y] *= f;
          }
        }
    }
    uint32_t p[NB][2];  // P^T as B fragments: keys 2 quad + {0, 1}, {8, 9} of row 8 x + lane / 4
#pragma unroll
    for (int x = 0; x < NB; ++x) {
      p[x][0] = transpose8(pack2<true>(wt[x][0], wt[x][1]));
      p[x][1] = transpose8(pack2<true>(wt[x][2], wt[x][3]));
    }
#pragma unroll
    for (int t = 0; t < DP / 16; ++t) {
      const int x0 = (2 * t) >> 2, c0 = (2 * t) & 3;
      const uint32_t v[4] = {codes_of(vw[0][x0], vw[1][x0], c0), codes_of(vw[0][x0], vw[1][x0], c0 + 1),
                             codes_of(vw[2][x0], vw[3][x0], c0), codes_of(vw[2][x0], vw[3][x0], c0 + 1)};
#pragma unroll
      for (int x = 0; x < NB; ++x) mma16816<true>(o[x][t], v, p[x][0], p[x][1]);
    }
  }
  // copies in flight (after a wait that gave up) land before their place is used again
  for (int it = done; it < min(n_it, done + kStages); ++it) mbar_wait_drain(&s.full[warp][it % kStages], (it / kStages) & 1);
#pragma unroll
  for (int x = 0; x < NB; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[x][y] += __shfl_xor_sync(0xFFFFFFFFu, l[x][y], d);
  bad = __reduce_max_sync(0xFFFFFFFFu, bad);
  __syncthreads();  // every warp is done with its ring
  float* so = reinterpret_cast<float*>(&s.ring[0][0][0][0]);
#pragma unroll
  for (int x = 0; x < NB; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      // relative to the true maximum from here on
      const int r = 8 * x + 2 * quad + y;
      const float f = m_true[x][y] == -INFINITY ? 0.f : ex2_approx(m[x][y] - m_true[x][y]);
      if (row == 0) {
        s.ml[warp][r][0] = m_true[x][y];
        s.ml[warp][r][1] = l[x][y] * f;
      }
      const float fo = f * pow2(-pow2_exponent(ref[x][y]));
      float* dst = so + (warp * kRowsTile + r) * RowsEnd<DP>::kOPitch + row * (DP / 8);
#pragma unroll
      for (int t = 0; t < DP / 8; t += 4)
        *reinterpret_cast<float4*>(dst + t) = make_float4(o[x][t / 2][y] * fo, o[x][t / 2][2 + y] * fo,
                                                          o[x][t / 2 + 1][y] * fo, o[x][t / 2 + 1][2 + y] * fo);
    }
  if (a.f16) rows_end<DP, true, CL>(a, w, split, item, tok0, n_rows, direct, bad, so, s.ml);
  else rows_end<DP, false, CL>(a, w, split, item, tok0, n_rows, direct, bad, so, s.ml);
  if (a.overlap && blockIdx.x == 0 && blockIdx.y == 0) griddep_wait();  // (no early return: split 0 always runs)
}

template <int DP, int NB, bool WIDE, bool CL, int CAP>
cudaError_t launch_rows8_t(const PagedArgs& a, const PagedTable<CAP>& tab, const CUtensorMap& mk, const CUtensorMap& mv,
                           cudaStream_t stream) {
  const size_t smem = sizeof(Rows8Smem<DP, WIDE>) + 1024;
  auto kernel = swa_paged_rows_e4m3_kernel<DP, NB, WIDE, CL, CAP>;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit(kernel, smem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_rows_grid<CL>(kernel, dim3(tab.n_items, a.splits), smem, stream, a, tab, mk, mv);
}

}  // namespace

template <int CAP>
cudaError_t launch_paged_rows_e4m3(const PagedArgs& a, const PagedTable<CAP>& tab, const CUtensorMap& mk,
                                   const CUtensorMap& mv, cudaStream_t stream) {
  if (tab.n_items == 0) return cudaSuccess;
  using std::integral_constant;
  auto go = [&](auto dp, auto nb, auto wide) {
    return a.cluster ? launch_rows8_t<dp.value, nb.value, wide.value, true>(a, tab, mk, mv, stream)
                     : launch_rows8_t<dp.value, nb.value, wide.value, false>(a, tab, mk, mv, stream);
  };
  auto pick = [&](auto dp, auto nb) {
    return a.ex.wide ? go(dp, nb, std::true_type{}) : go(dp, nb, std::false_type{});
  };
  using One = integral_constant<int, 1>;
  using Two = integral_constant<int, 2>;
  if (a.g.D <= 64)
    return a.most_rows <= 8 ? pick(integral_constant<int, 64>{}, One{}) : pick(integral_constant<int, 64>{}, Two{});
  return a.most_rows <= 8 ? pick(integral_constant<int, 128>{}, One{}) : pick(integral_constant<int, 128>{}, Two{});
}
template cudaError_t launch_paged_rows_e4m3<kPagedSmallTable>(const PagedArgs&, const PagedTable<kPagedSmallTable>&,
                                                              const CUtensorMap&, const CUtensorMap&, cudaStream_t);
template cudaError_t launch_paged_rows_e4m3<kPagedLargeTable>(const PagedArgs&, const PagedTable<kPagedLargeTable>&,
                                                              const CUtensorMap&, const CUtensorMap&, cudaStream_t);

}  // namespace swa
