// swa_paged.h — shapes shared by the host side and the kernels of the rotary
// and paged-cache operators (include/swa.h, "Rotary positions, a paged
// key/value cache, and attention over it").
#pragma once
#include <type_traits>

#include "swa_internal.h"

#if defined(__CUDACC__)
#define SWA_PAGED_HD __host__ __device__ __forceinline__
#else
#define SWA_PAGED_HD inline
#endif

namespace swa {

// Sequences of one launch, passed as a kernel parameter.  b < 0: the one entry
// stands for all sequences, whose chunks have the same length q_len (sequence
// b's starts at b * q_len), as in a decoding step of any batch size.
struct PagedDesc {
  int32_t q_start, q_len, b;
  int32_t tiles;       // row tiles per head group (attention)
  int32_t item_begin;  // first work item of this entry (attention)
};
template <int CAP>
struct PagedTable {
  int32_t count;    // entries used
  int32_t n_items;  // work items of this launch (attention)
  PagedDesc d[CAP];
};

// The cache and the chunk as a kernel sees them.
struct PagedGeom {
  int32_t N, N_kv, D;
  int32_t page_size, num_pages;
  int32_t kv_limit;  // largest valid kv_lens[b]
  int64_t table_stride;
  int64_t k_page, k_head, k_slot;  // strides in elements
  int64_t v_page, v_head, v_slot;
  const int32_t* table;
  const int32_t* kv_lens;
  // extents of the caller's tensors in elements, for the bounds-checked build
  int64_t n_k, n_v, n_table, n_lens;
};

// 8-bit cache: the exponents of its rows, [pages][N_kv][page_size].
struct PagedExps {
  int8_t *k, *v;  // NULL: a 16-bit cache
  int64_t page;   // exponents of a page
  int64_t n;      // extent, for the bounds-checked build
  int32_t wide;   // rows of codes start on 16 bytes and are multiples of 16 long (else of 8)
};

// The exponents of an 8-bit row: least (bf16, fp16) and most.  A larger one
// marks a row with a NaN.
constexpr int kExpLeastBf16 = -100, kExpLeastF16 = -15, kExpMost = 7, kExpNan = 127;

// ------------------------------------------------------- rotary / append --
constexpr int kRopeMaxTok = 16;  // rows (tokens) per CTA at most
constexpr int kRopeResident = 4, kAppendResident = 5;  // CTAs per SM (an append to an 8-bit cache: 4)
constexpr int kRopeThreads = 256;

struct RopeArgs {
  // segments: 0 q, 1 k, 2 v (append only).  heads[s] = 0: absent
  const void* src[3];
  void* dst[3];
  int64_t src_b[3], src_r[3], src_h[3];  // strides: batch, row, head
  int64_t dst_b[3], dst_r[3], dst_h[3];  // (pages: dst_b / dst_r unused)
  int64_t n_src[3], n_dst[3];            // extents, for the bounds-checked build
  int32_t heads[3];
  int32_t H;          // heads[0] + heads[1] + heads[2]
  uint32_t h_magic;   // ceil(2^32 / H); 8-bit cache: ceil(2^32 / heads[1])
  int32_t D, R;
  int32_t units;      // 2 * VEC-element units of a head row
  int32_t unit_shift; // 8-bit cache: log2(units)
  int32_t row_lanes;  // rows a CTA takes at a time: threads / units
  int32_t tok, tok_shift;  // tokens per CTA (tok_inner: a power of two, 1 << tok_shift)
  int32_t tok_inner;  // 1: walk the tokens of a head first
  int32_t n_axes, inverse;
  int32_t S;          // rows per batch
  int64_t rows;       // tokens in all
  int64_t n_pos;      // positions per axis
  const int32_t* positions;  // NULL (append): the token's position in its sequence
  PagedGeom pg;       // append only
  int32_t* err;       // append: status word; else NULL
  int32_t clear_err;  // append: 1 in the first launch of a call
  int32_t* page_err;  // append: page status per token
  int32_t tok_begin;  // append: first token of this launch
  uint64_t freq[64];  // angle per position as a fraction of a turn, 2^64 = one turn
  uint8_t axis[64];
  PagedExps ex;       // append
};

// The tokens of a chunk read back from the pages.
constexpr int kGatherThreads = 256, kGatherMostTok = 16;
struct GatherArgs {
  PagedGeom pg;
  PagedExps ex;
  const void* src[2];           // k, v pages
  void* dst[2];
  int64_t dst_r[2], dst_h[2];   // strides: row, head
  int64_t n_dst[2];             // extents, for the bounds-checked build
  int32_t lanes, lane_shift;    // threads of a row: a power of two
  int32_t tok, tok_begin;       // tokens per CTA, first token of this launch
  int64_t rows;                 // last token + 1 of this launch
  int32_t* err;
  int32_t clear_err;
  int32_t* page_err;  // per token
};
template <int CAP>
cudaError_t launch_gather(const GatherArgs& a, const PagedTable<CAP>& tab, bool f16, int n_ctas, cudaStream_t stream);

template <int CAP>
cudaError_t launch_append(const RopeArgs& a, const PagedTable<CAP>& tab, int dtype, bool interleaved, int n_ctas,
                          cudaStream_t stream);
cudaError_t launch_rope(const RopeArgs& a, int dtype, bool interleaved, cudaStream_t stream);
// Elements per load: 8 where R is a multiple of 16 (16-byte loads of 16-bit
// types), else 4; always 4 for fp32.
inline int rope_vec(int dtype, int64_t R) { return dtype == SWA_DTYPE_FP32 || R % 16 != 0 ? 4 : 8; }

// -------------------------------------------------------------- attention --
// Which coordinate (1..3) of a page tensor map is the slot, the head, the
// page: a map's dimensions go by ascending stride.
struct PageDims {
  int32_t slot_at, head_at, page_at;
};

// Row tile: `tok` tokens x `gs` query heads that share one key/value head,
// row r = token r / gs, head r mod gs of head group vh (heads vh*gs ...).
struct PagedBase {
  PagedGeom g;
  int32_t gs, tok, groups;  // groups = N / gs head groups
  uint32_t gs_magic;        // ceil(2^16 / gs)
  int32_t group;            // N / N_kv: head group vh reads key/value head vh * gs / group
  int32_t f16;
  int32_t sparse_mode;
  int32_t pre, next;  // clamped so that position sums stay inside int32
  float scale_log2;
  int32_t whole;      // tile kernel: the first items of the launch, one unit each; the others are split
  int32_t splits;     // CTAs (units) per split item along the keys, at most
  int32_t par, cap, least;  // paged_split
  int32_t cluster;    // few-row kernel: the splits are a cluster, which joins them itself
  int32_t rows_pad;   // rows of a partial tile
  int32_t stall;      // test hook (kStallPaged)
  int32_t box_rows;   // slots per TMA box: the largest power of two dividing the page size, up to 128
  PageDims kd, vd;
  int32_t q_tma;      // tile kernel: Q comes through a tensor map
  int64_t q_row, q_head;
  const void* q;
  const void* k_pages;
  const void* v_pages;
  void* out;
  float* smax;        // may be NULL
  float* ssum;        // may be NULL
  float* part_o;      // [items - whole][splits][rows_pad][DP] (splits > 1)
  float2* part_ml;    // [items - whole][splits][rows_pad]: maximum (log2 units), sum
  int32_t item_base;  // items of earlier launches of the call (0 where whole > 0)
  int32_t* err;
  int32_t clear_err;
  int32_t signal;     // tile kernel: let the next grid start on the SMs that it leaves
  int32_t overlap;    // few-row kernel: that next grid
  int32_t* page_err;  // per unit of the call: [whole], then [items - whole][splits]
  int64_t n_q, n_out, n_stats;  // extents, for the bounds-checked build
};
// What only some calls have: the kernels of the others are launched without it.
struct PagedArgs : PagedBase {
  int32_t sinks;      // BAND: keys below this one stay visible behind the window
  int32_t most_rows;  // rows that some tile has
  // a chunk that is a tree of drafted tokens: bit c of row t: token t sees token c of its chunk
  const uint32_t* tree;
  int64_t tree_row;      // words between rows
  const int32_t* depth;  // of each token; NULL: its place in the chunk
  int64_t n_tree, n_depth;  // extents, for the bounds-checked build
  PagedExps ex;
};

// Row r of a tile belongs to its token r / gs (r < 128; gs_magic = ceil(2^16 / gs), exact there).
SWA_PAGED_HD int row_token(int r, uint32_t gs_magic) { return static_cast<int>((r * gs_magic) >> 16); }

// A resolved work item.
struct PagedItem {
  int32_t b, vh, tile, q_start, q_len;
};
template <int CAP>
SWA_PAGED_HD PagedItem resolve_paged(const PagedTable<CAP>& tab, int groups, int k) {
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.d[mid].item_begin <= k) lo = mid; else hi = mid - 1;
  }
  const PagedDesc& d = tab.d[lo];
  const int local = k - d.item_begin;
  PagedItem it;
  // sequence, then tile (the latest tokens, which see most, first), then head
  // group: items go by falling weight, and those in flight share pages
  const int per = d.tiles * groups;
  int x = local, seq = 0;
  if (d.b < 0) {
    seq = local / per;
    x = local - seq * per;
  }
  const int rank = x / groups;
  it.vh = x - rank * groups;
  it.tile = d.tiles - 1 - rank;
  it.q_len = d.q_len;
  it.b = d.b < 0 ? seq : d.b;
  it.q_start = d.b < 0 ? seq * d.q_len : d.q_start;
  return it;
}

// Keys that some row of a tile sees: [lo, hi] (empty when lo > hi), and the
// sinks [0, sinks) where those end before lo.
struct PagedKeys {
  int lo, hi, sinks;
};
// Chunk token i has position kv_len - q_len + i; a token of a tree that of its
// depth, at least that of depth 0, and it may see the whole chunk.  X: there may
// be sinks or a tree.
template <bool X>
using ArgsOf = std::conditional_t<X, PagedArgs, PagedBase>;
template <bool X>
SWA_PAGED_HD const uint32_t* tree_of(const ArgsOf<X>& a) {
  if constexpr (X) return a.tree;
  else return nullptr;
}
template <bool X>
SWA_PAGED_HD int sinks_of(const ArgsOf<X>& a) {
  if constexpr (X) return a.sinks;
  else return 0;
}
template <bool X>
SWA_PAGED_HD PagedKeys paged_keys(const ArgsOf<X>& a, int kv_len, int q_len, int tok0, int n_tok) {
  PagedKeys k{0, kv_len - 1, 0};
  if (a.sparse_mode == 4) {
    const bool tree = tree_of<X>(a) != nullptr;
    const int p0 = kv_len - q_len + (tree ? 0 : tok0), p1 = p0 + n_tok - 1;
    const int pre = tree && a.pre < 0 ? 0 : a.pre;  // (a window that begins ahead still leaves a tree its chunk)
    k.lo = p0 - pre > 0 ? p0 - pre : 0;
    if (!tree) k.hi = p1 + a.next < k.hi ? p1 + a.next : k.hi;
    if (const int sinks = sinks_of<X>(a); sinks > 0) {
      const int n = sinks < k.hi + 1 ? sinks : k.hi + 1;
      if (k.lo > k.hi) {
        k.lo = 0;
        k.hi = n - 1;
      } else if (n >= k.lo) {
        k.lo = 0;
      } else {
        k.sinks = n;
      }
    }
  }
  return k;
}
// The same keys in runs of 2^shift: unit x of `total` is number x < sinks ? x : jump + x.
struct PagedUnits {
  int sinks, jump, total;
  SWA_PAGED_HD int at(int x) const { return x < sinks ? x : jump + x; }
};
template <bool X>
SWA_PAGED_HD PagedUnits paged_units(const PagedKeys& k, int shift) {
  PagedUnits u{0, k.lo >> shift, 0};
  if (k.lo > k.hi) return u;
  if (X && k.sinks > 0) {
    const int n = ((k.sinks - 1) >> shift) + 1;
    u.sinks = n < u.jump ? n : u.jump;
  }
  u.total = u.sinks + (k.hi >> shift) - u.jump + 1;
  u.jump -= u.sinks;
  return u;
}

// Key steps of split s: [begin, end) of the item's `steps`, in `*active` equal
// runs.  A run takes a `par`-th of them (as many CTAs as fill the GPU), at
// most `cap` (a sequence far longer than the others must not hold one CTA up)
// and at least `least`.
SWA_PAGED_HD void paged_split(int steps, int par, int cap, int least, int s, int* begin, int* end, int* active) {
  int per = (steps + par - 1) / par;
  if (per > cap) per = cap;
  if (per < least) per = least;
  *active = steps > 0 ? (steps + per - 1) / per : 0;
  if (*active > 1) per = (steps + *active - 1) / *active;
  *begin = s * per < steps ? s * per : steps;
  *end = *begin + per < steps ? *begin + per : steps;
}

constexpr int kSms = 152;         // SMs of the part this library is built for; sizes grids only
constexpr int kRowsTile = 16;     // rows of a tile of the few-row kernel
constexpr int kRowsStep = 64;     // keys per step of the few-row kernel (4 warps x 16)
constexpr int kPagedTileRows = 128;  // rows of a tile of the tensor-memory kernel
constexpr int kPagedTileStep = 128;  // keys per step of it

// What a kernel can do beside the window: sinks and trees (extended masks).
// Each is a translation unit of its own, and calls that need neither run what
// they ran without them.
enum class PagedKind { kPlain, kMasks };

template <PagedKind KIND, int CAP>
cudaError_t launch_paged_rows(const PagedArgs& a, const PagedTable<CAP>& tab, cudaStream_t stream);
template <int CAP>
cudaError_t launch_paged_rows_e4m3(const PagedArgs& a, const PagedTable<CAP>& tab, const CUtensorMap& mk,
                                   const CUtensorMap& mv, cudaStream_t stream);
template <PagedKind KIND, int CAP>
cudaError_t launch_paged_tile(const PagedArgs& a, const PagedTable<CAP>& tab, const CUtensorMap& mk,
                              const CUtensorMap& mv, const CUtensorMap& mq, cudaStream_t stream);
// The keys that row tiles see of an 8-bit cache as 16-bit pages of 128 slots.
struct UnpackArgs {
  void *k, *v;           // [page][N_kv][128][D]
  int32_t* table;        // the block table of those pages
  int64_t table_stride;
  int64_t status_base;   // the pages' status words, behind the attention's
  int32_t lanes, lane_shift;  // threads of a row: a power of two
};
// An entry's `item_begin` and `tiles` count pages here.
template <int CAP>
cudaError_t launch_paged_unpack(const PagedArgs& a, const PagedTable<CAP>& tab, const UnpackArgs& u, int pages,
                                cudaStream_t stream);
// Join the splits' partial results; `step_keys` as of the kernel that wrote them.
template <int CAP>
cudaError_t launch_paged_join(const PagedArgs& a, const PagedTable<CAP>& tab, int step_keys, cudaStream_t stream);

constexpr int kPagedSmallTable = 16;
constexpr int kPagedLargeTable = 512;

// Codes of the per-CTA page status.
enum : int32_t { kPageErrEntry = 1, kPageErrLength = 2 };

}  // namespace swa
