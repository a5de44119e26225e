// swa_paged.cpp — host side of the rotary and paged-cache operators
// (include/swa.h): argument checks, split of the work, launches.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>

#include "swa_paged.h"
#include "swa_turn.h"

using namespace swa;

namespace {

constexpr int64_t kMaxKv = int64_t(1) << 28;
constexpr int64_t kMaxStride = int64_t(1) << 38;  // elements; a TMA stride is below 2^40 bytes
// Keys one CTA of the few-row kernel takes at most, so that one long sequence
// does not hold a batch up.  201 sequences of up to 2000 keys and one of 131072:
// 358 us, 354 with 8192 (twice the CTAs, most with nothing to do), 408 with 4096.
constexpr int64_t kRowsMostKeys = 16384;
// The same over an 8-bit cache.  64 sequences of 100 to 16384 keys: 199 us, 201 with
// 2048, 206 with 4096, 207 with 1024, 250 with 16384; 24 of them 79, 85 with 2048; 64
// of up to 4000 keys 69.5, 73.7; 64 of 8192 181, 178.  (A bound on the lengths far above
// them costs more with short runs, whose CTAs start to find nothing: those 64 sequences
// 294 us with a bound of 131072 keys, 1066 with 2^20; over a 16-bit cache 397, 401 and 412.)
constexpr int64_t kRows8MostKeys = 1536;
constexpr int64_t kMostSplits = 65535;  // a grid's second dimension
constexpr int64_t kClusterMost = 8;   // CTAs of a cluster of the few-row kernel (any GPU schedules 8)
constexpr int64_t kClusterSteps = 5;  // key steps a CTA of it takes where more CTAs could be had
constexpr int64_t kTailSteps = 12;  // key tiles that splitting a last round must save (0.76 us each)
constexpr double kLog2e = 1.4426950408889634;
// Pages of 16-bit values that an 8-bit cache is unpacked into at a time, in all sequences of a pass together
// (one sequence may take more).
constexpr int64_t kScratchBytes = int64_t(1) << 30;
constexpr int64_t kGatherWaves = 8;  // CTAs per SM that a gather spreads its tokens over, before a CTA takes several

template <typename... A>
swa_status_t fail(swa_status_t st, const char* fmt, A... a) {
  return set_error(st, fmt, a...);
}
swa_status_t cuda_fail(cudaError_t e, const char* what) {
  return set_error(SWA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t less_slack(int64_t extent) { return std::max<int64_t>(extent - debug_extent_slack(), 0); }

// Largest divisor of n that is at most `most`.
int64_t divisor_up_to(int64_t n, int64_t most) {
  for (int64_t d = std::min(n, most); d > 1; --d)
    if (n % d == 0) return d;
  return 1;
}

swa_status_t check_heads(int64_t N, int64_t* N_kv, int64_t D) {
  if (N < 1 || N > 256) return fail(SWA_ERR_PARAM_INVALID, "N must be in [1, 256], got %lld", (long long)N);
  if (*N_kv == 0) *N_kv = N;
  if (*N_kv < 1 || *N_kv > 256) return fail(SWA_ERR_PARAM_INVALID, "N_kv must be in [1, 256], got %lld", (long long)*N_kv);
  if (D < 1 || D > 768) return fail(SWA_ERR_PARAM_INVALID, "D must be in [1, 768], got %lld", (long long)D);
  if (D % 8 != 0 || D > 128)
    return fail(SWA_ERR_UNSUPPORTED, "D = %lld is not built (a multiple of 8 up to 128)", (long long)D);
  return SWA_OK;
}

swa_status_t check_pointer(const void* p, const char* name) {
  if (!p) return fail(SWA_ERR_PARAM_NULLPTR, "%s is NULL", name);
  if (!aligned16(p)) return fail(SWA_ERR_PARAM_INVALID, "%s must be 16-byte aligned", name);
  return SWA_OK;
}

// One stride of a dimension of `n` entries: a multiple of 8 elements; `least`
// apart where the entries must not overlap (0: they may coincide).
swa_status_t check_stride(int64_t* stride, int64_t n, int64_t least, const char* name, const char* dim) {
  if (n <= 1) {
    *stride = 0;  // never used
    return SWA_OK;
  }
  if (*stride < least || *stride > kMaxStride || *stride % 8 != 0)
    return fail(SWA_ERR_PARAM_INVALID, "%s: %s stride %lld is not a multiple of 8 in [%lld, 2^38]", name, dim,
                (long long)*stride, (long long)least);
  return SWA_OK;
}

// Strides of a [B,N,S,D] / [B*S,N,D] tensor; `extent` its elements from first to last.
swa_status_t tensor_strides(const swa_strides_t* given, int32_t layout, int64_t B, int64_t S, int64_t N, int64_t D,
                            bool output, const char* name, swa_strides_t* s, int64_t* extent) {
  if (layout == SWA_LAYOUT_BNSD) *s = swa_strides_t{N * S * D, D, S * D};
  else *s = swa_strides_t{S * N * D, N * D, D};
  if (given) {
    s->row = given->row;
    s->head = given->head;
    if (layout == SWA_LAYOUT_BNSD) s->batch = given->batch;
  }
  if (layout == SWA_LAYOUT_TND) {
    S *= B;
    B = 1;
  }
  const int64_t least = output ? D : 0;
  swa_status_t st = check_stride(&s->batch, B, least, name, "batch");
  if (st == SWA_OK) st = check_stride(&s->row, S, least, name, "row");
  if (st == SWA_OK) st = check_stride(&s->head, N, least, name, "head");
  if (st != SWA_OK) return st;
  const long double last = (long double)(B - 1) * s->batch + (long double)(S - 1) * s->row + (long double)(N - 1) * s->head;
  if (last > (long double)(int64_t(1) << 60)) return fail(SWA_ERR_PARAM_INVALID, "%s: strides too large", name);
  *extent = (B - 1) * s->batch + (S - 1) * s->row + (N - 1) * s->head + D;
  return SWA_OK;
}

// The rows of a result must not overlap: in ascending order, each stride is past
// all that the smaller ones span.
swa_status_t check_apart(const swa_strides_t& s, int32_t layout, int64_t B, int64_t S, int64_t N, int64_t D,
                         const char* name) {
  const bool tnd = layout == SWA_LAYOUT_TND;
  struct Dim {
    int64_t n, stride;
  } d[3] = {{tnd ? 1 : B, s.batch}, {tnd ? B * S : S, s.row}, {N, s.head}};
  std::sort(d, d + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  int64_t span = D;
  for (const Dim& x : d) {
    if (x.n <= 1) continue;
    if (x.stride < span)
      return fail(SWA_ERR_PARAM_INVALID, "%s: stride %lld overlaps rows, which span %lld elements", name,
                  (long long)x.stride, (long long)span);
    span += (x.n - 1) * x.stride;
  }
  return SWA_OK;
}

// No C++ exception leaves a C entry point.
template <typename F>
swa_status_t guarded(F&& body) noexcept {
  try {
    try {
      return body();
    } catch (...) {
      return fail(SWA_ERR_CUDA, "out of host memory");
    }
  } catch (...) {  // (not even for the message)
    return SWA_ERR_CUDA;
  }
}

// ----------------------------------------------------------------- rotary --
swa_status_t rope_plan(const swa_rope_params_t* p, RopeArgs& a, int64_t* n_kv) {
  if (!p) return fail(SWA_ERR_PARAM_NULLPTR, "params is NULL");
  if (p->layout != SWA_LAYOUT_BNSD && p->layout != SWA_LAYOUT_TND)
    return fail(SWA_ERR_PARAM_INVALID, "layout %d is neither BNSD (0) nor TND (1)", p->layout);
  *n_kv = p->N_kv;
  swa_status_t st = check_heads(p->N, n_kv, p->D);
  if (st != SWA_OK) return st;
  if (p->B < 1 || p->S < 1 || p->B > (int64_t(1) << 31) || p->S > (int64_t(1) << 31) ||
      p->B * p->S >= (int64_t(1) << 31))
    return fail(SWA_ERR_PARAM_INVALID, "B and S must be >= 1 with B * S below 2^31");
  if (p->dtype != SWA_DTYPE_BF16 && p->dtype != SWA_DTYPE_FP16 && p->dtype != SWA_DTYPE_FP32)
    return fail(SWA_ERR_PARAM_INVALID, "dtype should be 0 (bf16), 1 (fp16) or 2 (fp32), got %d", p->dtype);
  if (p->interleaved != 0 && p->interleaved != 1)
    return fail(SWA_ERR_PARAM_INVALID, "interleaved should be 0 or 1, got %d", p->interleaved);
  const int64_t R = p->rotary_dim == 0 ? p->D : p->rotary_dim;
  if (R < 1 || R > p->D) return fail(SWA_ERR_PARAM_INVALID, "rotary_dim must be in [1, D], got %lld", (long long)R);
  if (R % 8 != 0) return fail(SWA_ERR_UNSUPPORTED, "rotary_dim = %lld is not built (a multiple of 8)", (long long)R);
  if (p->n_axes < 1 || p->n_axes > 4)
    return fail(SWA_ERR_PARAM_INVALID, "n_axes must be in [1, 4], got %d", p->n_axes);
  if (!p->inv_freq && !(p->base > 0.0 && std::isfinite(p->base)))
    return fail(SWA_ERR_PARAM_INVALID, "base must be positive and finite, got %g", p->base);
  a = RopeArgs{};
  a.D = static_cast<int32_t>(p->D);
  a.R = static_cast<int32_t>(R);
  a.n_axes = p->n_axes;
  for (int64_t i = 0; i < R / 2; ++i) {
    const double f = p->inv_freq ? p->inv_freq[i] : std::pow(p->base, -2.0 * static_cast<double>(i) / static_cast<double>(R));
    if (!std::isfinite(f) || std::fabs(f) > 1048576.0)
      return fail(SWA_ERR_PARAM_INVALID, "inv_freq[%lld] = %g is not within 2^20", (long long)i, f);
    const int32_t ax = p->pair_axis ? p->pair_axis[i] : 0;
    if (ax < 0 || ax >= p->n_axes)
      return fail(SWA_ERR_PARAM_INVALID, "pair_axis[%lld] = %d is outside [0, n_axes)", (long long)i, ax);
    a.freq[i] = turn_fraction(f);
    a.axis[i] = static_cast<uint8_t>(ax);
  }
  return SWA_OK;
}

// Split of the tokens over CTAs, and of a CTA over its threads: units of
// 2 * VEC elements, row_lanes rows at a time.
void set_split(RopeArgs& a, int dtype, int64_t rows) {
  const bool q8 = a.ex.k != nullptr;
  a.H = a.heads[0] + a.heads[1] + a.heads[2];
  a.h_magic = static_cast<uint32_t>(((uint64_t(1) << 32) + a.H - 1) / a.H);
  a.units = static_cast<int32_t>(ceil_div(a.D, 2 * rope_vec(dtype, a.R)));
  if (q8) {  // a row's threads then share a warp
    while (a.units & (a.units - 1)) ++a.units;
    while ((1 << a.unit_shift) < a.units) ++a.unit_shift;
    a.h_magic = static_cast<uint32_t>(((uint64_t(1) << 32) + a.heads[1] - 1) / a.heads[1]);
  }
  a.row_lanes = kRopeThreads / a.units;
  const int x = a.heads[0] ? 0 : 1;
  a.tok_inner = a.src_r[x] < a.src_h[x] ? 1 : 0;
  // Tokens per CTA: the fewest token times over all rounds of resident CTAs,
  // a CTA costing about one token beside its own; a CTA's tokens stay within
  // 80 KB, or 112 KB for an append, whose start is longer (length, then block
  // table).  32768 tokens of 40 heads in BNSD: 106 us with 8 (7 rounds), 112
  // with 16, 116 with 4; an append of 6739 tokens of 48 heads of 96: 21.7 us
  // with 9 (one round), 25.4 with 3; TND rotation 103 us under 80 KB, 106 above.
  const int64_t most_bytes = (a.heads[2] ? 112 : 80) * 1024;
  const int64_t slots = kSms * (a.heads[2] && !q8 ? kAppendResident : kRopeResident);
  const int64_t bytes = int64_t(a.H) * a.D * (dtype == SWA_DTYPE_FP32 ? 4 : 2);
  int64_t best = 0;
  for (int tok = 1; tok <= (a.tok_inner ? 8 : kRopeMaxTok) && (tok == 1 || tok * bytes <= most_bytes);
       tok += a.tok_inner ? tok : 1) {
    const int64_t cost = ceil_div(ceil_div(rows, tok), slots) * (tok + 1);
    if (best == 0 || cost < best) {
      best = cost;
      a.tok = tok;
    }
  }
  while ((1 << a.tok_shift) < a.tok) ++a.tok_shift;
}

swa_status_t rope_call(const swa_rope_params_t* p, const void* q, const swa_strides_t* q_s, const void* k,
                       const swa_strides_t* k_s, const int32_t* positions, void* q_out, const swa_strides_t* qo_s,
                       void* k_out, const swa_strides_t* ko_s, int inverse, swa_stream_t stream) {
  RopeArgs a;
  int64_t n_kv;
  swa_status_t st = rope_plan(p, a, &n_kv);
  if (st != SWA_OK) return st;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) || (!q && !k) || !positions)
    return fail(SWA_ERR_PARAM_NULLPTR, "q and q_out, or k and k_out, or both, and positions are required");
  const bool bnsd = p->layout == SWA_LAYOUT_BNSD;
  if (reinterpret_cast<uintptr_t>(positions) & 3u)
    return fail(SWA_ERR_PARAM_INVALID, "positions must be 4-byte aligned");
  const void* src[2] = {q, k};
  void* dst[2] = {q_out, k_out};
  const swa_strides_t* ss[2] = {q_s, k_s};
  const swa_strides_t* ds[2] = {qo_s, ko_s};
  const int64_t heads[2] = {p->N, n_kv};
  const char* names[4] = {"q", "k", "q_out", "k_out"};
  for (int x = 0; x < 2; ++x) {
    if (!src[x]) continue;
    if ((st = check_pointer(src[x], names[x])) != SWA_OK || (st = check_pointer(dst[x], names[2 + x])) != SWA_OK)
      return st;
    swa_strides_t s;
    int64_t n;
    st = tensor_strides(ss[x], p->layout, p->B, p->S, heads[x], p->D, false, names[x], &s, &n);
    if (st != SWA_OK) return st;
    a.src[x] = src[x];
    a.src_b[x] = s.batch;
    a.src_r[x] = s.row;
    a.src_h[x] = s.head;
    a.n_src[x] = less_slack(n);
    st = tensor_strides(ds[x], p->layout, p->B, p->S, heads[x], p->D, true, names[2 + x], &s, &n);
    if (st == SWA_OK) st = check_apart(s, p->layout, p->B, p->S, heads[x], p->D, names[2 + x]);
    if (st != SWA_OK) return st;
    a.dst[x] = dst[x];
    a.dst_b[x] = s.batch;
    a.dst_r[x] = s.row;
    a.dst_h[x] = s.head;
    a.n_dst[x] = less_slack(n);
    a.heads[x] = static_cast<int32_t>(heads[x]);
  }
  a.inverse = inverse;
  a.rows = p->B * p->S;
  a.n_pos = a.rows;
  a.S = static_cast<int32_t>(bnsd ? p->S : a.rows);
  a.positions = positions;
  set_split(a, p->dtype, a.rows);
  const cudaError_t e = launch_rope(a, p->dtype, p->interleaved != 0, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : cuda_fail(e, "rotary launch");
}

// ------------------------------------------------------------------ paged --
struct PagedPlan {
  int64_t N_kv = 0;
  int64_t max_kv = 0;
  std::vector<int64_t> start, len;  // per sequence
  int64_t uniform = 0;              // > 0: the first `n_uniform` sequences have this chunk length, the others none
  int64_t n_uniform = 0;
};

swa_status_t paged_plan(const swa_paged_params_t* p, PagedPlan& plan) {
  if (!p) return fail(SWA_ERR_PARAM_NULLPTR, "params is NULL");
  plan.N_kv = p->N_kv;
  swa_status_t st = check_heads(p->N, &plan.N_kv, p->D);
  if (st != SWA_OK) return st;
  if (p->N % plan.N_kv != 0)
    return fail(SWA_ERR_PARAM_INVALID, "N = %lld must be a multiple of N_kv = %lld", (long long)p->N,
                (long long)plan.N_kv);
  if (p->dtype == SWA_DTYPE_FP32) return fail(SWA_ERR_UNSUPPORTED, "a paged cache of fp32 is not built");
  if (p->dtype != SWA_DTYPE_BF16 && p->dtype != SWA_DTYPE_FP16)
    return fail(SWA_ERR_PARAM_INVALID, "dtype should be 0 (bf16) or 1 (fp16), got %d", p->dtype);
  if (p->sparse_mode != 0 && p->sparse_mode != 4)
    return fail(SWA_ERR_PARAM_INVALID, "sparse_mode should be 0 or 4, got %d", p->sparse_mode);
  if (p->sparse_mode == 4 && (long double)p->pre_tokens + (long double)p->next_tokens < 0)
    return fail(SWA_ERR_PARAM_INVALID, "pre_tokens + next_tokens < 0: every row would be empty");
  if (!std::isfinite(static_cast<float>(p->scale * kLog2e)))
    return fail(SWA_ERR_PARAM_INVALID, "scale is not a finite fp32 number");
  if (p->sink_tokens < 0)
    return fail(SWA_ERR_PARAM_INVALID, "sink_tokens must be >= 0, got %lld", (long long)p->sink_tokens);
  if (p->cache_dtype != SWA_CACHE_SAME && p->cache_dtype != SWA_CACHE_E4M3)
    return fail(SWA_ERR_PARAM_INVALID, "cache_dtype should be 0 (as dtype) or 1 (e4m3), got %d", p->cache_dtype);
  if (p->cache_layout != SWA_LAYOUT_BNSD && p->cache_layout != SWA_LAYOUT_TND)
    return fail(SWA_ERR_PARAM_INVALID, "cache_layout %d is neither BNSD (0) nor TND (1)", p->cache_layout);
  if (p->num_pages < 1 || p->num_pages > 2147483647)
    return fail(SWA_ERR_PARAM_INVALID, "num_pages must be in [1, 2^31), got %lld", (long long)p->num_pages);
  if (p->page_size < 1 || p->page_size > 65536)
    return fail(SWA_ERR_PARAM_INVALID, "page_size must be in [1, 65536], got %lld", (long long)p->page_size);
  if (p->page_size % 16 != 0)
    return fail(SWA_ERR_UNSUPPORTED, "page_size = %lld is not built (a multiple of 16)", (long long)p->page_size);
  if (p->max_pages < 1 || p->max_pages > (int64_t(1) << 24))
    return fail(SWA_ERR_PARAM_INVALID, "max_pages must be in [1, 2^24], got %lld", (long long)p->max_pages);
  if (p->max_kv_len < 0 || p->max_kv_len > kMaxKv)
    return fail(SWA_ERR_PARAM_INVALID, "max_kv_len must be in [0, 2^28], got %lld", (long long)p->max_kv_len);
  const int64_t held = std::min(p->max_pages * p->page_size, kMaxKv);
  plan.max_kv = p->max_kv_len == 0 ? held : std::min(p->max_kv_len, held);
  if (p->B < 1 || p->B > (int64_t(1) << 20)) return fail(SWA_ERR_PARAM_INVALID, "B must be in [1, 2^20]");
  if (p->T_q < 1 || p->T_q > kMaxRows)
    return fail(SWA_ERR_PARAM_INVALID, "T_q must be in [1, %lld]", (long long)kMaxRows);
  if (!p->cu_seqlens_q) return fail(SWA_ERR_PARAM_NULLPTR, "cu_seqlens_q is NULL");
  st = parse_cumulative(p->cu_seqlens_q, p->B, p->T_q, "cu_seqlens_q", plan.start, plan.len);
  if (st != SWA_OK) return st;
  int64_t n = 0;
  while (n < p->B && plan.len[n] > 0 && plan.len[n] == plan.len[0]) ++n;
  if (n > 0 && n * plan.len[0] == p->T_q) {
    plan.uniform = plan.len[0];
    plan.n_uniform = n;
  }
  return SWA_OK;
}

// The page dimensions by ascending stride (those of one entry last).
struct PageOrder {
  int64_t n[3], stride[3];
  int at[3];  // coordinate (1..3) of slot, head, page
};
PageOrder page_order(const swa_page_strides_t& s, const swa_paged_params_t* p, int64_t N_kv) {
  const int64_t n[3] = {p->page_size, N_kv, p->num_pages}, st[3] = {s.slot, s.head, s.page};
  int idx[3] = {0, 1, 2};
  auto key = [&](int x) { return n[x] > 1 ? st[x] : INT64_MAX; };
  std::stable_sort(idx, idx + 3, [&](int x, int y) { return key(x) < key(y); });
  PageOrder o{};
  for (int i = 0; i < 3; ++i) {
    o.n[i] = n[idx[i]];
    o.stride[i] = st[idx[i]];
    // a dimension of one entry: any valid stride
    if (o.n[i] <= 1) o.stride[i] = i == 0 ? p->D : o.stride[i - 1];
    o.at[idx[i]] = i + 1;
  }
  return o;
}

swa_status_t page_strides(const swa_page_strides_t* given, const swa_paged_params_t* p, int64_t N_kv, const char* name,
                          swa_page_strides_t* s, int64_t* extent) {
  const int64_t P = p->page_size, D = p->D;
  if (p->cache_layout == SWA_LAYOUT_BNSD) *s = swa_page_strides_t{N_kv * P * D, P * D, D};
  else *s = swa_page_strides_t{P * N_kv * D, D, N_kv * D};
  if (given) *s = *given;
  swa_status_t st = check_stride(&s->page, p->num_pages, D, name, "page");
  if (st == SWA_OK) st = check_stride(&s->head, N_kv, D, name, "head");
  if (st == SWA_OK) st = check_stride(&s->slot, P, D, name, "slot");
  if (st != SWA_OK) return st;
  const long double last =
      (long double)(p->num_pages - 1) * s->page + (long double)(N_kv - 1) * s->head + (long double)(P - 1) * s->slot;
  if (last > (long double)(int64_t(1) << 60)) return fail(SWA_ERR_PARAM_INVALID, "%s: strides too large", name);
  const PageOrder o = page_order(*s, p, N_kv);
  for (int i = 1; i < 3; ++i)
    if (o.n[i] > 1 && (o.stride[i] % o.stride[i - 1] != 0 || o.stride[i] / o.stride[i - 1] < o.n[i - 1]))
      return fail(SWA_ERR_UNSUPPORTED, "%s: stride %lld is not a multiple, past %lld entries, of stride %lld", name,
                  (long long)o.stride[i], (long long)o.n[i - 1], (long long)o.stride[i - 1]);
  *extent = (p->num_pages - 1) * s->page + (N_kv - 1) * s->head + (P - 1) * s->slot + D;
  return SWA_OK;
}

swa_status_t paged_geom(const swa_paged_params_t* p, const PagedPlan& plan, const void* k_pages,
                        const swa_page_strides_t* k_s, const void* v_pages, const swa_page_strides_t* v_s,
                        const int8_t* k_exp, const int8_t* v_exp, const int32_t* table, int64_t table_stride,
                        const int32_t* kv_lens, PagedGeom& g, PagedExps& ex) {
  swa_status_t st;
  const bool q8 = p->cache_dtype == SWA_CACHE_E4M3;
  if (q8) {
    if ((st = check_pointer(k_exp, "k_exponents")) != SWA_OK || (st = check_pointer(v_exp, "v_exponents")) != SWA_OK)
      return st;
  } else if (k_exp || v_exp) {
    return fail(SWA_ERR_PARAM_INVALID, "exponents are taken with an e4m3 cache only");
  }
  if ((st = check_pointer(k_pages, "k_pages")) != SWA_OK || (st = check_pointer(v_pages, "v_pages")) != SWA_OK)
    return st;
  if (!table || !kv_lens) return fail(SWA_ERR_PARAM_NULLPTR, "block_table or kv_lens is NULL");
  if ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(kv_lens)) & 3u)
    return fail(SWA_ERR_PARAM_INVALID, "block_table and kv_lens must be 4-byte aligned");
  if (table_stride == 0) table_stride = p->max_pages;
  if (table_stride < p->max_pages || table_stride > (int64_t(1) << 40))
    return fail(SWA_ERR_PARAM_INVALID, "table_stride %lld is below max_pages", (long long)table_stride);
  g = PagedGeom{};
  g.N = static_cast<int32_t>(p->N);
  g.N_kv = static_cast<int32_t>(plan.N_kv);
  g.D = static_cast<int32_t>(p->D);
  g.page_size = static_cast<int32_t>(p->page_size);
  g.num_pages = static_cast<int32_t>(p->num_pages);
  g.kv_limit = static_cast<int32_t>(plan.max_kv);
  g.table_stride = table_stride;
  g.table = table;
  g.kv_lens = kv_lens;
  swa_page_strides_t s;
  if ((st = page_strides(k_s, p, plan.N_kv, "k_pages", &s, &g.n_k)) != SWA_OK) return st;
  g.k_page = s.page;
  g.k_head = s.head;
  g.k_slot = s.slot;
  if ((st = page_strides(v_s, p, plan.N_kv, "v_pages", &s, &g.n_v)) != SWA_OK) return st;
  g.v_page = s.page;
  g.v_head = s.head;
  g.v_slot = s.slot;
  g.n_k = less_slack(g.n_k);
  g.n_v = less_slack(g.n_v);
  if (q8) {
    ex.k = const_cast<int8_t*>(k_exp);
    ex.v = const_cast<int8_t*>(v_exp);
    ex.page = plan.N_kv * p->page_size;
    ex.n = less_slack(p->num_pages * ex.page);
    ex.wide = (p->D | g.k_page | g.k_head | g.k_slot | g.v_page | g.v_head | g.v_slot) % 16 == 0 ? 1 : 0;
  }
  g.n_table = (p->B - 1) * table_stride + p->max_pages;
  g.n_lens = p->B;
  return SWA_OK;
}

// Tensor map of the pages: boxes of `box_rows` slots x 64 columns, 128-byte
// swizzle (8-bit: x 64 or 128 columns, a swizzle of as many bytes); columns past
// D and pages past the last read as zeros.
swa_status_t page_map(CUtensorMap* m, PageDims* dims, const void* ptr, const swa_page_strides_t& s,
                      const swa_paged_params_t* p, int64_t N_kv, int box_rows, const char* name) {
  auto fn = encode_fn();
  if (!fn) return fail(SWA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const PageOrder o = page_order(s, p, N_kv);
  const bool q8 = p->cache_dtype == SWA_CACHE_E4M3;
  const cuuint32_t columns = q8 && p->D > 64 ? 128 : 64;
  cuuint64_t d[4] = {static_cast<cuuint64_t>(p->D)}, st[3];
  cuuint32_t box[4] = {columns, 1, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    d[i + 1] = static_cast<cuuint64_t>(o.n[i]);
    st[i] = static_cast<cuuint64_t>(o.stride[i]) * (q8 ? 1 : 2);
  }
  box[o.at[0]] = static_cast<cuuint32_t>(box_rows);
  *dims = PageDims{o.at[0], o.at[1], o.at[2]};
  const CUtensorMapDataType type =
      q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
         : (p->dtype == SWA_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
  const CUresult r = fn(m, type, 4, const_cast<void*>(ptr), d, st, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        q8 && columns == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SWA_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with %d", name, (int)r);
  return SWA_OK;
}

swa_status_t check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws || bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return fail(SWA_ERR_WORKSPACE, "workspace must be >= %zu bytes and 256-byte aligned (got %zu)", need, bytes);
  return SWA_OK;
}

// Launch on the sequences (in `order`, or as they come) that `take` fills an entry for, at most CAP of them per
// table, and none that is `full` for the table so far.
template <int CAP, typename Take, typename Launch, typename Full>
cudaError_t each_table(const PagedPlan& plan, const std::vector<int32_t>& order, Take&& take, Launch&& launch,
                       Full&& full) {
  static thread_local std::unique_ptr<PagedTable<CAP>> storage;
  if (!storage) storage.reset(new PagedTable<CAP>());
  PagedTable<CAP>& tab = *storage;
  std::memset(&tab, 0, sizeof tab);
  auto flush = [&]() -> cudaError_t {
    if (tab.count == 0) return cudaSuccess;
    const cudaError_t e = launch(tab);
    std::memset(&tab, 0, sizeof tab);
    return e;
  };
  for (size_t x = 0; x < plan.len.size(); ++x) {
    const int32_t b = order.empty() ? static_cast<int32_t>(x) : order[x];
    PagedDesc d{};
    if (plan.len[b] == 0) continue;
    if (tab.count > 0 && full(b)) {
      const cudaError_t e = flush();
      if (e != cudaSuccess) return e;
    }
    if (!take(b, d, tab)) continue;
    tab.d[tab.count++] = d;
    if (tab.count == CAP) {
      const cudaError_t e = flush();
      if (e != cudaSuccess) return e;
    }
  }
  return flush();
}

int64_t live_sequences(const PagedPlan& plan) {
  int64_t n = 0;
  for (int64_t x : plan.len) n += x > 0;
  return n;
}

// Launches over the chunk's tokens, `tok` of them a CTA: go(table, first token, past the last, CTAs).
template <typename Go>
cudaError_t over_tokens(const swa_paged_params_t* p, const PagedPlan& plan, int64_t tok, Go&& go) {
  if (plan.uniform > 0) {
    PagedTable<kPagedSmallTable> tab{};
    tab.count = 1;
    tab.d[0].b = -1;
    tab.d[0].q_len = static_cast<int32_t>(plan.uniform);
    return go(tab, 0, p->T_q, static_cast<int>(ceil_div(p->T_q, tok)));
  }
  auto take = [&](int b, PagedDesc& d, auto&) {
    d.q_start = static_cast<int32_t>(plan.start[b]);
    d.q_len = static_cast<int32_t>(plan.len[b]);
    d.b = b;
    return true;
  };
  auto one = [&](auto& tab) {
    const PagedDesc& last = tab.d[tab.count - 1];
    const int64_t begin = tab.d[0].q_start, end = last.q_start + last.q_len;
    return go(tab, begin, end, static_cast<int>(ceil_div(end - begin, tok)));
  };
  auto never = [](int) { return false; };
  return live_sequences(plan) <= kPagedSmallTable ? each_table<kPagedSmallTable>(plan, {}, take, one, never)
                                                  : each_table<kPagedLargeTable>(plan, {}, take, one, never);
}

// Workspace of an append or a gather call: the header and one page status per token.
size_t append_bytes(const swa_paged_params_t* p) { return kHeaderBytes + round256(static_cast<size_t>(p->T_q) * 4); }

// -------------------------------------------------------------- attention --
// The row tiles and splits of one kernel over the sequences it takes.
struct Part {
  int64_t gs = 1, tok = 1, rows = 0;  // heads and tokens of a tile, rows of a partial
  int64_t most = 0;                   // rows that some tile has
  int64_t items = 0, splits = 1, par = 1, cap = 1, least = 1, step = 1;
  int64_t whole = 0;  // items that are one unit each (tiles); the others are split
  bool cluster = false;
  size_t status_at = 0, ml_at = 0, o_at = 0;  // workspace offsets
  int64_t units() const { return whole + (items - whole) * splits; }
};
// The row tiles' keys of an 8-bit cache, unpacked: in passes over some of the
// sequences each, one after the other, so that the pages of a pass fit the scratch.
struct Scratch {
  std::vector<int64_t> pages;  // per sequence, at most
  int64_t held = 0;            // pages of the scratch
  int64_t total = 0;           // of all passes
  int64_t entries = 0;         // columns of its block table
  size_t status_at = 0, table_at = 0, k_at = 0, v_at = 0;
};
struct ForwardPlan {
  PagedPlan seq;
  Scratch scratch;
  // sequences with at most 16 query rows per key/value head (chunk length x
  // group), and the others
  Part rows, tile;
  size_t total = 0;
};
bool few_rows(int64_t q_len, int64_t group) { return q_len * group <= kRowsTile; }
// The sequences with row tiles, long chunks first: they tend to hold the heaviest tiles.
std::vector<int32_t> tile_order(const PagedPlan& seq) {
  std::vector<int32_t> order(seq.len.size());
  for (size_t b = 0; b < order.size(); ++b) order[b] = static_cast<int32_t>(b);
  std::stable_sort(order.begin(), order.end(), [&](int32_t x, int32_t y) { return seq.len[x] > seq.len[y]; });
  return order;
}

// Tensor map of q: boxes of the tile's tokens x heads x 64 columns, heads
// innermost, as the rows of a tile go.  *usable = 0 where the row stride is not
// a multiple of the head stride past all heads (the kernel then gathers rows).
swa_status_t query_map(CUtensorMap* m, int32_t* usable, const void* q, const swa_strides_t& s,
                       const swa_paged_params_t* p, const Part& tile) {
  const int64_t row = p->T_q > 1 ? s.row : p->N * p->D;
  const int64_t head = p->N > 1 ? s.head : row;
  *usable = row % head == 0 && row / head >= (p->N > 1 ? p->N : 1) ? 1 : 0;
  if (!*usable) return SWA_OK;
  auto fn = encode_fn();
  if (!fn) return fail(SWA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t d[3] = {static_cast<cuuint64_t>(p->D), static_cast<cuuint64_t>(p->N),
                           static_cast<cuuint64_t>(p->T_q)};
  const cuuint64_t st[2] = {static_cast<cuuint64_t>(head) * 2, static_cast<cuuint64_t>(row) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(tile.gs), static_cast<cuuint32_t>(tile.tok)};
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = fn(m, p->dtype == SWA_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        3, const_cast<void*>(q), d, st, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SWA_ERR_CUDA, "cuTensorMapEncodeTiled(q) failed with %d", (int)r);
  return SWA_OK;
}

swa_status_t forward_plan(const swa_paged_params_t* p, ForwardPlan& f) {
  swa_status_t st = paged_plan(p, f.seq);
  if (st != SWA_OK) return st;
  const int64_t G = p->N / f.seq.N_kv, DP = p->D <= 64 ? 64 : 128;
  f.total = kHeaderBytes;
  Scratch& sc = f.scratch;
  if (p->cache_dtype == SWA_CACHE_E4M3) {
    sc.entries = ceil_div(f.seq.max_kv, kPagedTileStep);
    sc.pages.assign(f.seq.len.size(), 0);
    int64_t most = 0;
    for (size_t b = 0; b < f.seq.len.size(); ++b) {
      const int64_t n = f.seq.len[b];
      if (n == 0 || few_rows(n, G)) continue;
      sc.pages[b] = sc.entries;
      if (p->sparse_mode == 4) {  // the window of a chunk (or a tree, which sees as far as its deepest token), and the sinks
        const long double w = (long double)p->pre_tokens + (long double)std::max<int64_t>(p->next_tokens, 0) + (long double)n;
        const int64_t sinks = ceil_div(std::min(p->sink_tokens, f.seq.max_kv), kPagedTileStep);
        if (w < (long double)f.seq.max_kv)
          sc.pages[b] = std::min(sc.entries, ceil_div(std::max<int64_t>(static_cast<int64_t>(w), 1), kPagedTileStep) + 1 + sinks);
      }
      sc.total += sc.pages[b];
      most = std::max(most, sc.pages[b]);
    }
    const int64_t page_bytes = 2 * f.seq.N_kv * kPagedTileStep * p->D * 2;
    sc.held = std::min(sc.total, std::max(most, kScratchBytes / page_bytes));
    if (sc.total > 2147483647) return fail(SWA_ERR_PARAM_INVALID, "too many keys for one call");
  }
  auto lay_out = [&](Part& part, bool few, int64_t most_rows, int64_t step) {
    part.gs = divisor_up_to(G, most_rows);
    part.tok = most_rows / part.gs;
    part.rows = most_rows;
    part.step = step;
    part.items = 0;
    for (int64_t n : f.seq.len)
      if (few_rows(n, G) == few) {
        part.items += ceil_div(n, part.tok) * (p->N / part.gs);
        part.most = std::max(part.most, std::min(n, part.tok) * part.gs);
      }
    // keys a tile can see, in steps (one more: a run may begin inside a step)
    int64_t keys = f.seq.max_kv;
    if (p->sparse_mode == 4) {
      // (sinks: whole steps of their own)
      const int64_t sinks = ceil_div(std::min(p->sink_tokens, keys), step) * step;
      const long double w =
          (long double)p->pre_tokens + (long double)p->next_tokens + (long double)part.tok + (long double)sinks;
      if (w < (long double)keys) keys = std::max<int64_t>(1, static_cast<int64_t>(w));
    }
    const int64_t steps = ceil_div(keys, step) + 1;
    const int64_t items = std::max<int64_t>(part.items, 1);
    if (few) {
      // One CTA draws up to ~46 GB/s, so one per SM nearly saturates HBM and
      // two per SM are resident: just over one per SM, or one per item where
      // the items are as many.  Measured (64 items of 8192 keys): 49 us in 128
      // CTAs, 48 in 256, 60 in 320, which start a second wave; 8 items of
      // 131072 keys: 83 us in 152, 92 in 304.
      // An 8-bit cache: four CTAs an SM, each of which draws 11 GB/s, and so shorter
      // runs (kRows8MostKeys).
      const bool q8 = p->cache_dtype == SWA_CACHE_E4M3;
      part.par = std::min(ceil_div(int64_t(kSms) * (q8 ? 4 : 1), items), steps);
      part.cap = std::max((q8 ? kRows8MostKeys : kRowsMostKeys) / step + 2, ceil_div(steps, kMostSplits));
      // (runs that a few more CTAs than the GPU holds would shorten by little: one
      // sequence of 131072 keys, 76 splits 54 us, 79 68)
      if (q8 && ceil_div(steps, part.cap) * 4 <= part.par * 5) part.cap = std::max(part.cap, ceil_div(steps, part.par));
      part.least = 1;
      // Up to 8 splits are one cluster, which joins them without a second
      // launch: a power of two of CTAs, all resident at once.  One token of
      // 1003 keys: 6.2 us against 7.0 in 17 splits joined by a kernel; 4
      // sequences of 2000 keys: 9.4 against 12.2.  Long runs of few items keep
      // more splits (4000 keys: 10.3 in a cluster of 8, 9.3 in 19 splits).
      const int64_t most = std::min<int64_t>(part.par, kClusterMost);
      if (part.par > 1 && (part.par <= kClusterMost || steps <= kClusterMost * kClusterSteps) &&
          steps <= part.cap * most) {
        part.par = 2;
        while (part.par < most) part.par *= 2;
        part.cluster = true;
      }
    } else {
      // A split writes and reads 64 KB and needs the join (a few us): only
      // where SMs would stay empty.  That is all items when they are fewer than
      // half the SMs, and the items of a last round that fills less than half
      // of them, if they are long: a tile of the longest sequence has the
      // cache behind the chunk to itself, as far as the window reaches.
      // Measured with the last round split and whole (32 / 8 heads): 2048
      // tokens (512 items) under a window of 4096 116.5 and 122.7 us, 640
      // tokens (160 items) 55.5 and 65.5, under a window of 8192 85 and 115.
      part.least = 4;
      part.cap = steps;
      int64_t longest = 0;
      for (int64_t n : f.seq.len) longest = std::max(longest, few_rows(n, G) ? 0 : n);
      const int64_t sure = std::min(keys, std::max<int64_t>(f.seq.max_kv - longest, 0)) / step;
      const int64_t last = part.items % kSms;
      const bool one_launch = sc.held == sc.total && ((f.seq.uniform > 0 && sc.total == 0) ||
                                                      live_sequences(f.seq) <= kPagedLargeTable);
      if (part.items <= kSms / 2) {
        part.par = std::min(kSms / items, ceil_div(steps, part.least));
      } else if (one_launch && part.items > kSms && last > 0 && last <= kSms / 2) {
        const int64_t ways = std::min(kSms / last, ceil_div(sure, 2 * part.least));
        if (ways > 1 && sure - ceil_div(sure, ways) >= kTailSteps) {
          part.par = ways;
          part.whole = part.items - last;
        }
      }
    }
    part.splits = std::max(part.par, ceil_div(steps, part.cap));
    part.status_at = f.total;
    f.total += round256(part.units() * 4);
    if (part.splits > 1 && !part.cluster) {
      const size_t rows = static_cast<size_t>(part.items - part.whole) * part.splits * part.rows;
      part.ml_at = f.total;
      part.o_at = part.ml_at + round256(rows * 8);
      f.total = part.o_at + round256(rows * DP * 4);
    }
  };
  lay_out(f.rows, true, kRowsTile, kRowsStep);
  lay_out(f.tile, false, kPagedTileRows, kPagedTileStep);
  if (sc.total > 0) {
    const size_t half = static_cast<size_t>(sc.held) * f.seq.N_kv * kPagedTileStep * p->D * 2;
    sc.status_at = f.total;
    sc.table_at = sc.status_at + round256(static_cast<size_t>(sc.total) * 4);
    sc.k_at = sc.table_at + round256(static_cast<size_t>(p->B) * sc.entries * 4);
    sc.v_at = sc.k_at + round256(half);
    f.total = sc.v_at + round256(half);
  }
  if (f.rows.items > 2147483647 || f.tile.items > 2147483647) return fail(SWA_ERR_PARAM_INVALID, "too many query rows for one call");
  return SWA_OK;
}

template <int CAP>
cudaError_t run_part(const swa_paged_params_t* p, const ForwardPlan& f, const Part& part, PagedArgs a,
                     const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mq, bool joins, cudaStream_t s) {
  const bool few = &part == &f.rows;
  a.gs = static_cast<int32_t>(part.gs);
  a.gs_magic = static_cast<uint32_t>(ceil_div(65536, part.gs));
  a.tok = static_cast<int32_t>(part.tok);
  a.groups = static_cast<int32_t>(p->N / part.gs);
  a.whole = static_cast<int32_t>(part.whole);
  a.splits = static_cast<int32_t>(part.splits);
  a.par = static_cast<int32_t>(part.par);
  a.cap = static_cast<int32_t>(part.cap);
  if (a.tree && p->sparse_mode == 4)  // a tile of a tree may see the whole chunk, past the window's keys that the plan counts
    a.cap += static_cast<int32_t>(ceil_div(*std::max_element(f.seq.len.begin(), f.seq.len.end()), part.step) + 1);
  a.least = static_cast<int32_t>(part.least);
  a.cluster = part.cluster ? 1 : 0;
  a.rows_pad = static_cast<int32_t>(part.rows);
  a.most_rows = static_cast<int32_t>(part.most);
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.err);
  a.page_err = reinterpret_cast<int32_t*>(ws + part.status_at);
  a.part_ml = reinterpret_cast<float2*>(ws + part.ml_at);
  a.part_o = reinterpret_cast<float*>(ws + part.o_at);
  // The sequences of `tab` unpacked into the scratch; `a` reads its pages from then on.
  const PagedArgs packed = a;
  int64_t unpacked = 0;  // pages of the passes before
  auto unpack = [&](const PagedTable<CAP>& tab) {
    const Scratch& sc = f.scratch;
    UnpackArgs u{};
    u.k = ws + sc.k_at;
    u.v = ws + sc.v_at;
    u.table = reinterpret_cast<int32_t*>(ws + sc.table_at);
    u.table_stride = sc.entries;
    while ((16 << u.lane_shift) < p->D) ++u.lane_shift;
    u.lanes = 1 << u.lane_shift;
    PagedTable<CAP> pages = tab;
    int64_t n = 0;
    for (int32_t x = 0; x < pages.count; ++x) {
      pages.d[x].item_begin = static_cast<int32_t>(n);
      n += pages.d[x].tiles = static_cast<int32_t>(sc.pages[pages.d[x].b]);
    }
    PagedArgs from = packed;
    from.page_err = reinterpret_cast<int32_t*>(ws + sc.status_at);
    from.clear_err = a.clear_err;
    u.status_base = unpacked;
    const cudaError_t e = launch_paged_unpack(from, pages, u, static_cast<int>(n), s);
    unpacked += n;
    a.clear_err = 0;
    a.k_pages = u.k;
    a.v_pages = u.v;
    a.ex = PagedExps{};
    a.g.table = u.table;
    a.g.table_stride = sc.entries;
    a.g.page_size = kPagedTileStep;
    a.g.num_pages = static_cast<int32_t>(sc.held);
    a.g.n_table = p->B * sc.entries;
    return e;
  };
  auto go = [&](PagedTable<CAP>& tab) {
    cudaError_t e = cudaSuccess;
    // calls without sinks and tree run the kernels that know nothing of them
    const bool masks = a.sinks > 0 || a.tree;
    if (!joins && !few && f.scratch.total > 0) e = unpack(tab);
    if (e != cudaSuccess) return e;
    if (joins) e = launch_paged_join(a, tab, static_cast<int>(part.step), s);
    else if (!few) e = masks ? launch_paged_tile<PagedKind::kMasks>(a, tab, mk, mv, mq, s)
                             : launch_paged_tile<PagedKind::kPlain>(a, tab, mk, mv, mq, s);
    else if (a.ex.k) e = launch_paged_rows_e4m3(a, tab, mk, mv, s);
    else e = masks ? launch_paged_rows<PagedKind::kMasks>(a, tab, s) : launch_paged_rows<PagedKind::kPlain>(a, tab, s);
    a.item_base += tab.n_items;
    a.clear_err = 0;
    return e;
  };
  const bool scratch = !few && f.scratch.total > 0;
  if (f.seq.uniform > 0 && !scratch) {
    PagedTable<CAP> tab{};
    tab.count = 1;
    tab.d[0].q_len = static_cast<int32_t>(f.seq.uniform);
    tab.d[0].b = -1;
    tab.d[0].tiles = static_cast<int32_t>(ceil_div(f.seq.uniform, part.tok));
    tab.n_items = static_cast<int32_t>(part.items);
    return go(tab);
  }
  int64_t held = 0;  // pages of the scratch that the table's sequences take
  auto take = [&](int b, PagedDesc& d, PagedTable<CAP>& tab) {
    if (few_rows(f.seq.len[b], a.group) != few) return false;
    if (scratch) held = (tab.count == 0 ? 0 : held) + f.scratch.pages[b];
    d.q_start = static_cast<int32_t>(f.seq.start[b]);
    d.q_len = static_cast<int32_t>(f.seq.len[b]);
    d.b = b;
    d.tiles = static_cast<int32_t>(ceil_div(d.q_len, part.tok));
    d.item_begin = tab.n_items;
    tab.n_items += d.tiles * a.groups;
    return true;
  };
  std::vector<int32_t> order;
  if (!few) order = tile_order(f.seq);
  auto full = [&](int b) { return scratch && !few_rows(f.seq.len[b], a.group) && held + f.scratch.pages[b] > f.scratch.held; };
  return each_table<CAP>(f.seq, order, take, go, full);
}

// The first page status of n words at `at` that is not 0.
swa_status_t read_pages(size_t n, const void* workspace, size_t at) {
  if (n == 0) return SWA_OK;
  std::vector<int32_t> host(n);
  const cudaError_t e =
      cudaMemcpy(host.data(), static_cast<const uint8_t*>(workspace) + at, n * 4, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "reading the page status");
  for (int32_t w : host) {
    if (w == kPageErrLength) return fail(SWA_ERR_PAGE, "an entry of kv_lens is outside [0, max_kv_len]");
    if (w != 0) return fail(SWA_ERR_PAGE, "an entry of block_table is outside [0, num_pages)");
  }
  return SWA_OK;
}

}  // namespace

// ------------------------------------------------------------------ ABI --
extern "C" {

void swa_rope_params_default(swa_rope_params_t* p) {
  if (!p) return;
  std::memset(p, 0, sizeof *p);
  p->n_axes = 1;
  p->base = 10000.0;
}

swa_status_t swa_rope_forward(const swa_rope_params_t* p, const void* q, const swa_strides_t* q_strides, const void* k,
                              const swa_strides_t* k_strides, const int32_t* positions, void* q_out,
                              const swa_strides_t* q_out_strides, void* k_out, const swa_strides_t* k_out_strides,
                              swa_stream_t stream) {
  return guarded([&]() -> swa_status_t {
    return rope_call(p, q, q_strides, k, k_strides, positions, q_out, q_out_strides, k_out, k_out_strides, 0, stream);
  });
}

swa_status_t swa_rope_backward(const swa_rope_params_t* p, const void* dq_out, const swa_strides_t* dq_out_strides,
                               const void* dk_out, const swa_strides_t* dk_out_strides, const int32_t* positions,
                               void* dq, const swa_strides_t* dq_strides, void* dk, const swa_strides_t* dk_strides,
                               swa_stream_t stream) {
  return guarded([&]() -> swa_status_t {
    return rope_call(p, dq_out, dq_out_strides, dk_out, dk_out_strides, positions, dq, dq_strides, dk, dk_strides, 1,
                     stream);
  });
}

void swa_paged_params_default(swa_paged_params_t* p) {
  if (!p) return;
  std::memset(p, 0, sizeof *p);
  p->scale = 1.0;
  p->pre_tokens = 2147483647;
  p->next_tokens = 2147483647;
}

swa_status_t swa_paged_append_workspace_size(const swa_paged_params_t* p, size_t* bytes) {
  return guarded([&]() -> swa_status_t {
    if (!bytes) return fail(SWA_ERR_PARAM_NULLPTR, "bytes is NULL");
    PagedPlan plan;
    const swa_status_t st = paged_plan(p, plan);
    if (st != SWA_OK) return st;
    *bytes = append_bytes(p);
    return SWA_OK;
  });
}

swa_status_t swa_paged_append(const swa_paged_params_t* p, const void* k, const swa_strides_t* k_strides,
                              const void* v, const swa_strides_t* v_strides, void* k_pages,
                              const swa_page_strides_t* k_page_strides, void* v_pages,
                              const swa_page_strides_t* v_page_strides, const int32_t* block_table,
                              int64_t table_stride, const int32_t* kv_lens, const swa_rope_params_t* rope,
                              const int32_t* positions, const void* q, const swa_strides_t* q_strides, void* q_out,
                              const swa_strides_t* q_out_strides, void* workspace, size_t workspace_bytes,
                              swa_stream_t stream) {
  return swa_paged_append_ext(p, k, k_strides, v, v_strides, k_pages, k_page_strides, v_pages, v_page_strides, nullptr,
                              nullptr, block_table, table_stride, kv_lens, rope, positions, q, q_strides, q_out,
                              q_out_strides, workspace, workspace_bytes, stream);
}

swa_status_t swa_paged_append_ext(const swa_paged_params_t* p, const void* k, const swa_strides_t* k_strides,
                                  const void* v, const swa_strides_t* v_strides, void* k_pages,
                                  const swa_page_strides_t* k_page_strides, void* v_pages,
                                  const swa_page_strides_t* v_page_strides, int8_t* k_exponents, int8_t* v_exponents,
                                  const int32_t* block_table, int64_t table_stride, const int32_t* kv_lens,
                                  const swa_rope_params_t* rope, const int32_t* positions, const void* q,
                                  const swa_strides_t* q_strides, void* q_out, const swa_strides_t* q_out_strides,
                                  void* workspace, size_t workspace_bytes, swa_stream_t stream) {
  return guarded([&]() -> swa_status_t {
    PagedPlan plan;
    swa_status_t st = paged_plan(p, plan);
    if (st != SWA_OK) return st;
    RopeArgs a{};
    if (rope) {
      int64_t rope_kv;
      if ((st = rope_plan(rope, a, &rope_kv)) != SWA_OK) return st;
      if (rope->layout != SWA_LAYOUT_TND || rope->B * rope->S != p->T_q || rope->N != p->N || rope_kv != plan.N_kv ||
          rope->D != p->D || rope->dtype != p->dtype)
        return fail(SWA_ERR_PARAM_INVALID, "rope must be TND with B * S = T_q and the cache's N, N_kv, D and dtype");
      if (reinterpret_cast<uintptr_t>(positions) & 3u)
        return fail(SWA_ERR_PARAM_INVALID, "positions must be 4-byte aligned");
    } else if (positions || q || q_out) {
      return fail(SWA_ERR_PARAM_INVALID, "positions, q and q_out are taken with rope only");
    }
    if ((q == nullptr) != (q_out == nullptr)) return fail(SWA_ERR_PARAM_NULLPTR, "q and q_out come together");
    if ((st = check_pointer(k, "k")) != SWA_OK || (st = check_pointer(v, "v")) != SWA_OK) return st;
    if (q && ((st = check_pointer(q, "q")) != SWA_OK || (st = check_pointer(q_out, "q_out")) != SWA_OK)) return st;
    st = paged_geom(p, plan, k_pages, k_page_strides, v_pages, v_page_strides, k_exponents, v_exponents, block_table,
                    table_stride, kv_lens, a.pg, a.ex);
    if (st != SWA_OK) return st;
    const size_t need = append_bytes(p);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != SWA_OK) return st;

    a.D = static_cast<int32_t>(p->D);
    const void* src[3] = {q, k, v};
    const swa_strides_t* ss[3] = {q_strides, k_strides, v_strides};
    const int64_t heads[3] = {q ? p->N : 0, plan.N_kv, plan.N_kv};
    const char* names[3] = {"q", "k", "v"};
    for (int x = 0; x < 3; ++x) {
      if (!src[x]) continue;
      swa_strides_t s;
      int64_t n;
      st = tensor_strides(ss[x], SWA_LAYOUT_TND, 1, p->T_q, heads[x], p->D, false, names[x], &s, &n);
      if (st != SWA_OK) return st;
      a.src[x] = src[x];
      a.src_r[x] = s.row;
      a.src_h[x] = s.head;
      a.n_src[x] = less_slack(n);
      a.heads[x] = static_cast<int32_t>(heads[x]);
    }
    if (q) {
      swa_strides_t s;
      int64_t n;
      st = tensor_strides(q_out_strides, SWA_LAYOUT_TND, 1, p->T_q, p->N, p->D, true, "q_out", &s, &n);
      if (st == SWA_OK) st = check_apart(s, SWA_LAYOUT_TND, 1, p->T_q, p->N, p->D, "q_out");
      if (st != SWA_OK) return st;
      a.dst_r[0] = s.row;
      a.dst_h[0] = s.head;
      a.n_dst[0] = less_slack(n);
    }
    a.dst[0] = q_out;
    a.dst[1] = k_pages;
    a.dst[2] = v_pages;
    a.dst_h[1] = a.pg.k_head;
    a.dst_h[2] = a.pg.v_head;
    a.n_dst[1] = a.pg.n_k;
    a.n_dst[2] = a.pg.n_v;
    a.S = static_cast<int32_t>(p->T_q);
    a.n_pos = p->T_q;
    a.positions = positions;
    set_split(a, p->dtype, p->T_q);
    a.err = static_cast<int32_t*>(workspace);
    a.page_err = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + kHeaderBytes);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    a.clear_err = SWA_CHECKS ? 0 : 1;
    if (SWA_CHECKS) e = cudaMemsetAsync(workspace, 0, sizeof(int32_t), s);
    if (e != cudaSuccess) return cuda_fail(e, "clearing the workspace header");
    const bool il = rope && rope->interleaved != 0;
    e = over_tokens(p, plan, a.tok, [&](const auto& tab, int64_t begin, int64_t end, int n_ctas) {
      a.tok_begin = static_cast<int32_t>(begin);
      a.rows = end;
      const cudaError_t le = launch_append(a, tab, p->dtype, il, n_ctas, s);
      a.clear_err = 0;
      return le;
    });
    return e == cudaSuccess ? SWA_OK : cuda_fail(e, "append launch");
  });
}

swa_status_t swa_paged_forward_workspace_size(const swa_paged_params_t* p, size_t* bytes) {
  return guarded([&]() -> swa_status_t {
    if (!bytes) return fail(SWA_ERR_PARAM_NULLPTR, "bytes is NULL");
    ForwardPlan f;
    const swa_status_t st = forward_plan(p, f);
    if (st != SWA_OK) return st;
    *bytes = f.total;
    return SWA_OK;
  });
}

swa_status_t swa_paged_forward(const swa_paged_params_t* p, const void* q, const swa_strides_t* q_strides,
                               const void* k_pages, const swa_page_strides_t* k_page_strides, const void* v_pages,
                               const swa_page_strides_t* v_page_strides, const int32_t* block_table,
                               int64_t table_stride, const int32_t* kv_lens, void* out, float* softmax_max,
                               float* softmax_sum, void* workspace, size_t workspace_bytes, swa_stream_t stream) {
  return swa_paged_forward_ext(p, q, q_strides, k_pages, k_page_strides, v_pages, v_page_strides, nullptr, block_table,
                               table_stride, kv_lens, out, softmax_max, softmax_sum, workspace, workspace_bytes, stream);
}

swa_status_t swa_paged_forward_ext(const swa_paged_params_t* p, const void* q, const swa_strides_t* q_strides,
                                   const void* k_pages, const swa_page_strides_t* k_page_strides, const void* v_pages,
                                   const swa_page_strides_t* v_page_strides, const swa_paged_extra_t* extra,
                                   const int32_t* block_table, int64_t table_stride, const int32_t* kv_lens, void* out,
                                   float* softmax_max, float* softmax_sum, void* workspace, size_t workspace_bytes,
                                   swa_stream_t stream) {
  return guarded([&]() -> swa_status_t {
    ForwardPlan f;
    swa_status_t st = forward_plan(p, f);
    if (st != SWA_OK) return st;
    const swa_paged_extra_t x = extra ? *extra : swa_paged_extra_t{};
    if ((st = check_pointer(q, "q")) != SWA_OK || (st = check_pointer(out, "out")) != SWA_OK) return st;
    if ((reinterpret_cast<uintptr_t>(softmax_max) | reinterpret_cast<uintptr_t>(softmax_sum)) & 3u)
      return fail(SWA_ERR_PARAM_INVALID, "softmax_max and softmax_sum must be 4-byte aligned");
    PagedArgs a{};
    st = paged_geom(p, f.seq, k_pages, k_page_strides, v_pages, v_page_strides, x.k_exponents, x.v_exponents,
                    block_table, table_stride, kv_lens, a.g, a.ex);
    if (st != SWA_OK) return st;
    if (x.tree) {
      const int64_t words = ceil_div(*std::max_element(f.seq.len.begin(), f.seq.len.end()), 32);
      const int64_t row = x.tree_stride == 0 ? words : x.tree_stride;
      if ((reinterpret_cast<uintptr_t>(x.tree) | reinterpret_cast<uintptr_t>(x.depth)) & 3u)
        return fail(SWA_ERR_PARAM_INVALID, "tree and depth must be 4-byte aligned");
      if (row < words || row > (int64_t(1) << 40))
        return fail(SWA_ERR_PARAM_INVALID, "tree_stride %lld is below the %lld words of the longest chunk", (long long)row,
                    (long long)words);
      if (p->sparse_mode == 4 && p->next_tokens < 0)
        return fail(SWA_ERR_PARAM_INVALID, "next_tokens must be >= 0 with a tree, got %lld", (long long)p->next_tokens);
      a.tree = x.tree;
      a.tree_row = row;
      a.depth = x.depth;
      a.n_tree = less_slack((p->T_q - 1) * row + words);
      a.n_depth = less_slack(p->T_q);
    } else if (x.depth || x.tree_stride != 0) {
      return fail(SWA_ERR_PARAM_INVALID, "depth and tree_stride are taken with a tree only");
    }
    swa_strides_t qs;
    // the row stride may not fold rows onto each other: tensor maps want it
    st = tensor_strides(q_strides, SWA_LAYOUT_TND, 1, p->T_q, p->N, p->D, true, "q", &qs, &a.n_q);
    if (st != SWA_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, f.total)) != SWA_OK) return st;
    a.n_q = less_slack(a.n_q);
    a.group = static_cast<int32_t>(p->N / f.seq.N_kv);
    a.f16 = p->dtype == SWA_DTYPE_FP16 ? 1 : 0;
    a.sparse_mode = p->sparse_mode;
    const int64_t lim = int64_t(1) << 29;  // positions stay within +-2^28: no sum passes int32
    a.pre = static_cast<int32_t>(std::min(std::max(p->pre_tokens, -lim), lim));
    a.next = static_cast<int32_t>(std::min(std::max(p->next_tokens, -lim), lim));
    a.sinks = p->sparse_mode == 4 ? static_cast<int32_t>(std::min(p->sink_tokens, lim)) : 0;
    a.scale_log2 = static_cast<float>(p->scale * kLog2e);
    a.stall = debug_stall_bits();
    a.q_row = qs.row;
    a.q_head = qs.head;
    a.q = q;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.out = out;
    a.smax = softmax_max;
    a.ssum = softmax_sum;
    a.err = static_cast<int32_t*>(workspace);
    a.clear_err = SWA_CHECKS ? 0 : 1;
    a.n_out = less_slack(p->T_q * p->N * p->D);
    a.n_stats = less_slack(p->T_q * p->N);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    CUtensorMap mk{}, mv{}, mq{}, rk{}, rv{};
    if (f.rows.items > 0 && a.ex.k && a.ex.wide) {  // groups of 16 slots, for the few-row kernel
      st = page_map(&rk, &a.kd, k_pages, swa_page_strides_t{a.g.k_page, a.g.k_head, a.g.k_slot}, p, f.seq.N_kv, 16,
                    "k_pages");
      if (st == SWA_OK)
        st = page_map(&rv, &a.vd, v_pages, swa_page_strides_t{a.g.v_page, a.g.v_head, a.g.v_slot}, p, f.seq.N_kv, 16,
                      "v_pages");
      if (st != SWA_OK) return st;
    }
    PageDims rows_kd = a.kd, rows_vd = a.vd;
    if (f.tile.items > 0) {
      swa_paged_params_t of = *p;  // the pages that the tiles read
      swa_page_strides_t ks{a.g.k_page, a.g.k_head, a.g.k_slot}, vs{a.g.v_page, a.g.v_head, a.g.v_slot};
      const void *kp = k_pages, *vp = v_pages;
      if (f.scratch.total > 0) {
        kp = static_cast<uint8_t*>(workspace) + f.scratch.k_at;
        vp = static_cast<uint8_t*>(workspace) + f.scratch.v_at;
        of.cache_dtype = SWA_CACHE_SAME;
        of.page_size = kPagedTileStep;
        of.num_pages = f.scratch.held;
        ks = vs = swa_page_strides_t{f.seq.N_kv * kPagedTileStep * p->D, kPagedTileStep * p->D, p->D};
      }
      const int64_t low = of.page_size & -of.page_size;
      a.box_rows = static_cast<int32_t>(std::min<int64_t>(low, kPagedTileStep));
      st = page_map(&mk, &a.kd, kp, ks, &of, f.seq.N_kv, a.box_rows, "k_pages");
      if (st == SWA_OK) st = page_map(&mv, &a.vd, vp, vs, &of, f.seq.N_kv, a.box_rows, "v_pages");
      if (st == SWA_OK) st = query_map(&mq, &a.q_tma, q, qs, p, f.tile);
      if (st != SWA_OK) return st;
    }
    if (SWA_CHECKS) e = cudaMemsetAsync(workspace, 0, sizeof(int32_t), s);
    if (e != cudaSuccess) return cuda_fail(e, "clearing the workspace header");
    const bool small = (f.seq.uniform > 0 && f.scratch.total == 0) || live_sequences(f.seq) <= kPagedSmallTable;
    auto run = [&](const Part& part, bool joins) {
      if (part.items == 0 || e != cudaSuccess || (joins && (part.splits <= 1 || part.cluster))) return;
      const bool few = &part == &f.rows;
      const CUtensorMap &k = few ? rk : mk, &v = few ? rv : mv;
      if (few && a.ex.k) {
        a.kd = rows_kd;
        a.vd = rows_vd;
      }
      e = small ? run_part<kPagedSmallTable>(p, f, part, a, k, v, mq, joins, s)
                : run_part<kPagedLargeTable>(p, f, part, a, k, v, mq, joins, s);
      a.clear_err = 0;
    };
    // A batch of both kinds whose tables fit one launch each: the few-row kernel
    // takes the SMs that the other leaves.  The joins come last: each waits for
    // the grid before it, and that one for the tiles.
    const bool both = f.tile.items > 0 && f.rows.items > 0 && live_sequences(f.seq) <= kPagedLargeTable &&
                      f.scratch.held == f.scratch.total;
    a.signal = both ? 1 : 0;
    run(f.tile, false);
    a.overlap = both ? 1 : 0;
    run(f.rows, false);
    run(f.tile, true);
    run(f.rows, true);
    return e == cudaSuccess ? SWA_OK : cuda_fail(e, "paged attention launch");
  });
}

swa_status_t swa_paged_gather(const swa_paged_params_t* p, const void* k_pages, const swa_page_strides_t* k_page_strides,
                              const void* v_pages, const swa_page_strides_t* v_page_strides, const int8_t* k_exponents,
                              const int8_t* v_exponents, const int32_t* block_table, int64_t table_stride,
                              const int32_t* kv_lens, void* k, const swa_strides_t* k_strides, void* v,
                              const swa_strides_t* v_strides, void* workspace, size_t workspace_bytes,
                              swa_stream_t stream) {
  return guarded([&]() -> swa_status_t {
    PagedPlan plan;
    swa_status_t st = paged_plan(p, plan);
    if (st != SWA_OK) return st;
    if ((st = check_pointer(k, "k")) != SWA_OK || (st = check_pointer(v, "v")) != SWA_OK) return st;
    GatherArgs a{};
    st = paged_geom(p, plan, k_pages, k_page_strides, v_pages, v_page_strides, k_exponents, v_exponents, block_table,
                    table_stride, kv_lens, a.pg, a.ex);
    if (st != SWA_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, append_bytes(p))) != SWA_OK) return st;
    a.src[0] = k_pages;
    a.src[1] = v_pages;
    void* dst[2] = {k, v};
    const swa_strides_t* given[2] = {k_strides, v_strides};
    const char* names[2] = {"k", "v"};
    for (int x = 0; x < 2; ++x) {
      swa_strides_t s;
      int64_t n;
      st = tensor_strides(given[x], SWA_LAYOUT_TND, 1, p->T_q, plan.N_kv, p->D, true, names[x], &s, &n);
      if (st == SWA_OK) st = check_apart(s, SWA_LAYOUT_TND, 1, p->T_q, plan.N_kv, p->D, names[x]);
      if (st != SWA_OK) return st;
      a.dst[x] = dst[x];
      a.dst_r[x] = s.row;
      a.dst_h[x] = s.head;
      a.n_dst[x] = less_slack(n);
    }
    const int64_t pieces = ceil_div(p->D, a.ex.k ? 16 : 8);  // threads of a row
    while ((int64_t(1) << a.lane_shift) < pieces) ++a.lane_shift;
    a.lanes = 1 << a.lane_shift;
    // few tokens: over the SMs; many: as many per CTA as a thread needs for its rows in flight
    a.tok = static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>(p->T_q / (kSms * kGatherWaves), 1), kGatherMostTok));
    a.err = static_cast<int32_t*>(workspace);
    a.page_err = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + kHeaderBytes);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    a.clear_err = SWA_CHECKS ? 0 : 1;
    if (SWA_CHECKS) e = cudaMemsetAsync(workspace, 0, sizeof(int32_t), s);
    if (e != cudaSuccess) return cuda_fail(e, "clearing the workspace header");
    const bool f16 = p->dtype == SWA_DTYPE_FP16;
    e = over_tokens(p, plan, a.tok, [&](const auto& tab, int64_t begin, int64_t end, int n_ctas) {
      a.tok_begin = static_cast<int32_t>(begin);
      a.rows = end;
      const cudaError_t le = launch_gather(a, tab, f16, n_ctas, s);
      a.clear_err = 0;
      return le;
    });
    return e == cudaSuccess ? SWA_OK : cuda_fail(e, "gather launch");
  });
}

swa_status_t swa_paged_append_status(const swa_paged_params_t* p, const void* workspace, swa_stream_t stream) {
  return guarded([&]() -> swa_status_t {
    PagedPlan plan;
    swa_status_t st = paged_plan(p, plan);
    if (st == SWA_OK) st = swa_workspace_status(workspace, stream);
    return st == SWA_OK ? read_pages(p->T_q, workspace, kHeaderBytes) : st;
  });
}

swa_status_t swa_paged_forward_status(const swa_paged_params_t* p, const void* workspace, swa_stream_t stream) {
  return guarded([&]() -> swa_status_t {
    ForwardPlan f;
    swa_status_t st = forward_plan(p, f);
    if (st != SWA_OK) return st;
    st = swa_workspace_status(workspace, stream);
    for (const Part* part : {&f.rows, &f.tile})
      if (st == SWA_OK) st = read_pages(part->units(), workspace, part->status_at);
    if (st == SWA_OK) st = read_pages(f.scratch.total, workspace, f.scratch.status_at);
    return st;
  });
}

}  // extern "C"
