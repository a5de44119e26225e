// swa_rope.cu — rotary positions of q and k, and the append of a chunk's keys
// and values to the paged cache (include/swa.h).
//
// One kernel: a CTA takes up to 16 tokens, all heads of q, k (and v) of each.
// Pair i of a row at position p turns by p * inv_freq[i].  The angle is kept as
// a 64-bit fraction of a turn, F_i = round(2^64 * (inv_freq_i / 2 pi mod 1))
// (swa_turn.h): p * F_i mod 2^64 is the angle modulo a turn by one integer
// multiply, off by |p| 2^-65 turns, at most 2^-34 for any int32 p; its distance
// from the nearest quarter turn goes through sincospif.  A token's R/2 angles
// are computed once, into shared memory, for all its heads.
//
// Bound by HBM: every element is read and written once.  Each thread keeps one
// place in the head row (VEC elements and their partners) and walks over
// (token, head) rows, four in flight through registers.  671 MB (32768 tokens,
// 32 + 8 heads of 128) take 106 us, 0.93 of the measured copy rate.  Walking
// the heads of a token first in BNSD, 256 bytes at a time, took 122 us; 16
// tokens per CTA 112, 4 tokens 116; all rows staged through shared memory by
// cp.async, 4 tokens per CTA, 130: what is left are instructions, not bytes in
// flight.
#include "swa_paged.h"
#include "swa_device.cuh"

namespace swa {
namespace {

template <typename T, int VEC>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> { using type = uint4; };
template <>
struct Raw<__nv_bfloat16, 4> { using type = uint2; };
template <>
struct Raw<__half, 8> { using type = uint4; };
template <>
struct Raw<__half, 4> { using type = uint2; };
template <>
struct Raw<float, 4> { using type = float4; };

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }

struct RopeSmem {
  int64_t src[kRopeMaxTok][3], dst[kRopeMaxTok][3];  // element offsets of (token, head 0); dst < 0: not stored
  int32_t pos[kRopeMaxTok];                          // position in its sequence (append)
  alignas(16) float cs[kRopeMaxTok][64], sn[kRopeMaxTok][64];
};

// in_bounds without a status word to report to: the access is skipped.
__device__ __forceinline__ bool rope_in_bounds(int64_t first, int64_t count, int64_t extent, int32_t* err) {
  if constexpr (SWA_CHECKS == 0) return true;
  if (err) return in_bounds(first, count, extent, err);
  return first >= 0 && first + count <= extent;
}

template <typename T, int VEC, bool IL>
__device__ __forceinline__ void turn(T (&a)[VEC], T (&b)[VEC], const float* cs_, const float* sn_) {
  alignas(16) float cs[VEC], sn[VEC];  // (VEC is a multiple of 4 and so is the first pair)
#pragma unroll
  for (int i = 0; i < VEC; i += 4) {
    *reinterpret_cast<float4*>(cs + i) = *reinterpret_cast<const float4*>(cs_ + i);
    *reinterpret_cast<float4*>(sn + i) = *reinterpret_cast<const float4*>(sn_ + i);
  }
  if constexpr (IL) {  // pairs inside a chunk: VEC / 2 of a, then VEC / 2 of b
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const float ca = cs[i], sa = sn[i], cb = cs[VEC / 2 + i], sb = sn[VEC / 2 + i];
      const float x0 = to_f(a[2 * i]), y0 = to_f(a[2 * i + 1]), x1 = to_f(b[2 * i]), y1 = to_f(b[2 * i + 1]);
      a[2 * i] = from_f<T>(x0 * ca - y0 * sa);
      a[2 * i + 1] = from_f<T>(y0 * ca + x0 * sa);
      b[2 * i] = from_f<T>(x1 * cb - y1 * sb);
      b[2 * i + 1] = from_f<T>(y1 * cb + x1 * sb);
    }
  } else {  // element i of a pairs with element i of b
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float c = cs[i], s = sn[i], x = to_f(a[i]), y = to_f(b[i]);
      a[i] = from_f<T>(x * c - y * s);
      b[i] = from_f<T>(y * c + x * s);
    }
  }
}

template <typename T, int VEC, bool IL, bool PAGED, int CAP>
__global__ void __launch_bounds__(kRopeThreads, PAGED ? kAppendResident : kRopeResident)
    swa_rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ PagedTable<CAP> tab) {
  using R = typename Raw<T, VEC>::type;
  __shared__ RopeSmem s;
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  if (PAGED && a.clear_err && blockIdx.x == 0 && tid == 0) *a.err = 0;
  const int64_t t0 = static_cast<int64_t>(PAGED ? a.tok_begin : 0) + static_cast<int64_t>(blockIdx.x) * a.tok;
  const int n_tok = static_cast<int>(a.rows - t0 < a.tok ? a.rows - t0 : a.tok);
  int bad = 0;
  if (tid < n_tok) {
    const int64_t t = t0 + tid;
    const int64_t bt = t / a.S, row = t - bt * a.S;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      s.src[tid][k] = bt * a.src_b[k] + row * a.src_r[k];
      s.dst[tid][k] = bt * a.dst_b[k] + row * a.dst_r[k];
    }
    if constexpr (PAGED) {
      // the token's sequence and place in it
      int b, i, q_len;
      if (tab.d[0].b < 0) {
        q_len = tab.d[0].q_len;
        b = static_cast<int>(t) / q_len;
        i = static_cast<int>(t) - b * q_len;
      } else {
        int lo = 0, hi = tab.count - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (tab.d[mid].q_start <= t) lo = mid; else hi = mid - 1;
        }
        b = tab.d[lo].b;
        q_len = tab.d[lo].q_len;
        i = static_cast<int>(t) - tab.d[lo].q_start;
      }
      int len = rope_in_bounds(b, 1, a.pg.n_lens, a.err) ? a.pg.kv_lens[b] : 0;
      if (len < 0 || len > a.pg.kv_limit) {
        bad = kPageErrLength;
        len = 0;
      }
      const int pos = len - q_len + i;
      s.pos[tid] = pos;
      int64_t kd = -1, vd = -1;
      if (pos >= 0) {
        const int entry = pos / a.pg.page_size, slot = pos - entry * a.pg.page_size;
        const int64_t e = b * a.pg.table_stride + entry;
        const int page = rope_in_bounds(e, 1, a.pg.n_table, a.err) ? a.pg.table[e] : -1;
        if (page >= 0 && page < a.pg.num_pages) {
          kd = page * a.pg.k_page + slot * a.pg.k_slot;
          vd = page * a.pg.v_page + slot * a.pg.v_slot;
        } else {
          bad = kPageErrEntry;
        }
      }
      s.dst[tid][1] = kd;
      s.dst[tid][2] = vd;
    }
  }
  if (PAGED && tid < n_tok) a.page_err[t0 + tid] = bad;
  __syncthreads();

  // the angles of the CTA's tokens
  const int half = a.R >> 1;
  for (int x = tid; x < n_tok * 64; x += kRopeThreads) {
    const int tk = x >> 6, i = x & 63;
    if (i < half) {
      int p;
      if (PAGED && a.positions == nullptr) {
        p = max(s.pos[tk], 0);
      } else {
        const int64_t e = a.axis[i] * a.n_pos + t0 + tk;
        p = rope_in_bounds(e, 1, a.n_axes * a.n_pos, a.err) ? a.positions[e] : 0;
      }
      const uint64_t turn64 = static_cast<uint64_t>(static_cast<int64_t>(p)) * a.freq[i];
      // its nearest quarter turn and the distance from there, in half turns within
      // a quarter: rounded to fp32, that is off by 2^-24 of itself, where the
      // whole angle was by 2^-25 half turns, much of a sine near its zeros
      const int quarter = static_cast<int>((turn64 + (uint64_t(1) << 61)) >> 62);
      const int64_t rest = static_cast<int64_t>(turn64 - (static_cast<uint64_t>(quarter) << 62));
      float sn, cs;
      sincospif(__ll2float_rn(rest) * 1.0842021724855044e-19f, &sn, &cs);  // 2^-63
      if (quarter & 1) {
        const float x = sn;
        sn = cs;
        cs = -x;
      }
      if (quarter & 2) {
        sn = -sn;
        cs = -cs;
      }
      s.cs[tk][i] = cs;
      s.sn[tk][i] = a.inverse ? -sn : sn;
    }
  }
  __syncthreads();

  // The CTA's (token, head) rows in the order in which they lie in memory:
  // tokens first where a row's stride is the smaller one (BNSD: the CTA's
  // tokens of a head are contiguous), heads first otherwise (TND).  Thread =
  // one place of a row (VEC elements and their partners) of every row_lanes-th
  // row, a few in flight.
  const int u = tid % a.units, lane = tid / a.units;
  if (lane >= a.row_lanes) return;
  const int n_rows = a.tok_inner ? a.H << a.tok_shift : n_tok * a.H;
  constexpr int kBatch = PAGED ? 2 : 4;
  struct Place {
    int tk, sg, ia, ib;
    int64_t src, dst;
  };
  auto locate = [&](int r, Place& w) -> bool {
    if (r >= n_rows) return false;
    int h;
    if (a.tok_inner) {
      w.tk = r & (a.tok - 1);
      h = r >> a.tok_shift;
      if (w.tk >= n_tok) return false;
    } else {
      w.tk = a.H == 1 ? r : static_cast<int>(__umulhi(static_cast<uint32_t>(r), a.h_magic));
      h = r - w.tk * a.H;
    }
    w.sg = h < a.heads[0] ? 0 : (h < a.heads[0] + a.heads[1] ? 1 : 2);
    h -= w.sg == 0 ? 0 : (w.sg == 1 ? a.heads[0] : a.heads[0] + a.heads[1]);
    const int rot = w.sg == 2 ? 0 : a.R;  // v is copied
    // first chunk and its partner
    if (!IL && u * VEC < (rot >> 1)) {
      w.ia = u * VEC;
      w.ib = (rot >> 1) + u * VEC;
    } else {
      w.ia = 2 * u * VEC;
      w.ib = w.ia + VEC;
    }
    w.src = s.src[w.tk][w.sg] + h * a.src_h[w.sg];
    w.dst = s.dst[w.tk][w.sg];
    if (PAGED && w.dst < 0) return false;
    w.dst += h * a.dst_h[w.sg];
    return true;
  };
  for (int r0 = lane; r0 < n_rows; r0 += kBatch * a.row_lanes) {
    R ra[kBatch], rb[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      Place w;
      if (!locate(r0 + k * a.row_lanes, w)) continue;
      const T* p = static_cast<const T*>(a.src[w.sg]);
      if (rope_in_bounds(w.src + w.ia, VEC, a.n_src[w.sg], a.err))
        ra[k] = __ldcs(reinterpret_cast<const R*>(p + w.src + w.ia));
      if (w.ib < a.D && rope_in_bounds(w.src + w.ib, VEC, a.n_src[w.sg], a.err))
        rb[k] = __ldcs(reinterpret_cast<const R*>(p + w.src + w.ib));
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      Place w;  // (again: cheaper than keeping four of them)
      if (!locate(r0 + k * a.row_lanes, w)) continue;
      alignas(16) T xa[VEC], xb[VEC];
      *reinterpret_cast<R*>(xa) = ra[k];
      *reinterpret_cast<R*>(xb) = rb[k];
      // the chunk's pairs: VEC of them, from pair u * VEC on in both forms
      if (w.sg != 2 && u * 2 * VEC < a.R) turn<T, VEC, IL>(xa, xb, &s.cs[w.tk][u * VEC], &s.sn[w.tk][u * VEC]);
      T* p = static_cast<T*>(a.dst[w.sg]);
      if (rope_in_bounds(w.dst + w.ia, VEC, a.n_dst[w.sg], a.err))
        *reinterpret_cast<R*>(p + w.dst + w.ia) = *reinterpret_cast<R*>(xa);
      if (w.ib < a.D && rope_in_bounds(w.dst + w.ib, VEC, a.n_dst[w.sg], a.err))
        *reinterpret_cast<R*>(p + w.dst + w.ib) = *reinterpret_cast<R*>(xb);
    }
  }
}

template <bool PAGED, int CAP>
cudaError_t launch_any(const RopeArgs& a, const PagedTable<CAP>& tab, int dtype, bool il, int ctas, cudaStream_t st) {
  const bool wide = rope_vec(dtype, a.R) == 8;
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(ctas), dim3(kRopeThreads), 0, st, a, tab); };
  if constexpr (!PAGED) {  // a paged cache holds 16-bit elements
    if (dtype == SWA_DTYPE_FP32)
      return il ? go(swa_rope_kernel<float, 4, true, PAGED, CAP>) : go(swa_rope_kernel<float, 4, false, PAGED, CAP>);
  }
  if (dtype == SWA_DTYPE_FP16) {
    if (wide)
      return il ? go(swa_rope_kernel<__half, 8, true, PAGED, CAP>) : go(swa_rope_kernel<__half, 8, false, PAGED, CAP>);
    return il ? go(swa_rope_kernel<__half, 4, true, PAGED, CAP>) : go(swa_rope_kernel<__half, 4, false, PAGED, CAP>);
  }
  if (wide)
    return il ? go(swa_rope_kernel<__nv_bfloat16, 8, true, PAGED, CAP>)
              : go(swa_rope_kernel<__nv_bfloat16, 8, false, PAGED, CAP>);
  return il ? go(swa_rope_kernel<__nv_bfloat16, 4, true, PAGED, CAP>)
            : go(swa_rope_kernel<__nv_bfloat16, 4, false, PAGED, CAP>);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, bool interleaved, cudaStream_t stream) {
  PagedTable<1> none{};
  const int64_t ctas = (a.rows + a.tok - 1) / a.tok;
  return launch_any<false, 1>(a, none, dtype, interleaved, static_cast<int>(ctas), stream);
}

template <int CAP>
cudaError_t launch_append(const RopeArgs& a, const PagedTable<CAP>& tab, int dtype, bool interleaved, int n_ctas,
                          cudaStream_t stream) {
  return launch_any<true, CAP>(a, tab, dtype, interleaved, n_ctas, stream);
}
template cudaError_t launch_append<kPagedSmallTable>(const RopeArgs&, const PagedTable<kPagedSmallTable>&, int, bool,
                                                     int, cudaStream_t);
template cudaError_t launch_append<kPagedLargeTable>(const RopeArgs&, const PagedTable<kPagedLargeTable>&, int, bool,
                                                     int, cudaStream_t);

}  // namespace swa
