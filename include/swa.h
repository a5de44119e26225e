/*
 * swa.h — C ABI of libswa: sliding-window (BAND) / unmasked FlashAttention
 * forward and backward on GB300 (sm_103a).
 *
 * The operation (FlashAttentionVarLenScore doc, "计算公式"; PyPTO-Gym
 * FlashAttentionScoreGrad article, "前向公式" / "反向公式"):
 *
 *   forward   O = Dropout(Softmax(Mask(scale * Q K^T)), keep_prob) V
 *             softmax_max_i = max_{j visible} scale * q_i.k_j
 *             softmax_sum_i = sum_{j visible} exp(scale * q_i.k_j - softmax_max_i)
 *   backward  P  = exp(scale * Q K^T - softmax_max) / softmax_sum
 *             D  = rowsum(dY * O)
 *             dP = (dY V^T) * z / keep_prob
 *             dS = P * (dP - D)
 *             dV = (P * z / keep_prob)^T dY,  dQ = scale dS K,  dK = scale dS^T Q
 *
 * Mask ("sparse_mode", FlashAttentionVarLenScore doc, parameter
 * sparseModeOptional; the split into swa_forward / swa_backward limited to
 * modes 0 and 4 follows the pzsr.cn article, §1.2 and §3):
 *   0  no mask: query i sees every key of its sequence;
 *   4  BAND: query i sees key j iff  i - pre_tokens <= j <= i + next_tokens
 *      (indices local to the sequence, top-left aligned when Sq != Skv).
 * With sink_tokens the first keys of a sequence stay visible behind the window.
 * A query row that sees no key gets out = 0, softmax_max = -inf,
 * softmax_sum = 0 and a zero dq row; it contributes nothing to dk / dv.
 *
 * Dropout (doc parameter dropMaskOptional / keepProbOptional): drop_mask is
 * a packed bit mask, 8 elements per byte, least significant bit first,
 * 1 = keep.  Element order: BNSD e = ((b*N + n)*Sq + i)*Skv + j; TND
 * e = sum_{b'<b} N*Sq_b'*Skv_b' + (n*Sq_b + i)*Skv_b + j (no padding).
 * softmax_sum excludes dropout; kept probabilities are scaled by 1/keep_prob.
 * Instead of a mask, a seed and an offset may stand for it (dropout_gen = 1;
 * the pages' high-level backward regenerates the mask from seed / offset,
 * SWA article §1.1): element (query row r, local key j) is kept iff byte
 * (j mod 16) of Philox4x32-10(counter = (j/16, lo32 r, hi32 r,
 * lo32 dropout_offset), key = (lo32 dropout_seed, hi32 dropout_seed)),
 * bytes little-endian across the four output words, is below
 * round(keep_prob * 256); r is the statistics index of the row (BNSD
 * (b*N + n)*S_q + i, TND t*N + n).  swa_dropout_mask writes that mask out.
 *
 * Layouts (doc parameter list, inputLayout; PyPTO-Gym article, I/O table):
 *   BNSD  q, dy, out, dq: [B, N, S_q, D];  k, v, dk, dv: [B, N, S_kv, D]
 *         softmax_max / softmax_sum: [B, N, S_q] fp32
 *   TND   q, dy, out, dq: [T_q, N, D];     k, v, dk, dv: [T_kv, N, D]
 *         softmax_max / softmax_sum: [T_q, N] fp32
 *   All tensors are dense, row-major, of p->dtype (bf16 by default) unless
 *   stated (statistics are fp32), device memory,
 *   16-byte aligned.  D is a multiple of 8 from 8 to 128 (a row of D
 *   elements then starts on a 16-byte boundary).  The kernels compute on 64
 *   (D <= 64) or 128 columns per row; the tensor maps fill the columns past D
 *   with zeros, which changes no result, and nothing past D is written.  The
 *   grad API's own pre-processing pads special head dims such as 72 and 88
 *   (aclnnFlashAttentionUnpaddingScoreGradV2 article §8.2, the API layer);
 *   here the padding costs no copy.
 *
 * Variable length (TND): cu_seqlens_q / cu_seqlens_kv are HOST arrays of
 * length B holding cumulative sequence ends without a leading 0 (doc
 * parameters actualSeqQLenOptional / actualSeqKvLenOptional).  A length-0
 * sequence is allowed; a trailing run of zeros marks skipped batches
 * (aclnnFlashAttentionUnpaddingScoreGradV2 article, §6.4).  The last
 * non-zero entry must equal T.
 *
 * Two-phase calls (doc, "两段式接口"): ask for the workspace size, let the
 * caller allocate it in device memory, then call.  The library allocates
 * nothing, keeps no pointer after a call returns and reads host arrays only
 * during the call.  Calls only enqueue work on `stream` (a cudaStream_t) and
 * return; results are ready when the stream is.  A workspace may be reused
 * by later calls on the same stream but not by calls running concurrently.
 *
 * The parameter structs grow at their ends from version to version, and the
 * library reads them whole: compile a program against the header of the library
 * that it runs with, and set a struct by its _default function first.
 *
 * Status codes follow the aclnn numbering (doc, "返回值").
 */
#ifndef SWA_H
#define SWA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SWA_API __attribute__((visibility("default")))
#else
#define SWA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *swa_stream_t; /* same type as cudaStream_t */

typedef enum { SWA_LAYOUT_BNSD = 0, SWA_LAYOUT_TND = 1 } swa_layout_t;

typedef enum {
  SWA_OK = 0,
  SWA_ERR_PARAM_NULLPTR = 161001, /* a required pointer is NULL */
  SWA_ERR_PARAM_INVALID = 161002, /* a value is outside its documented range */
  SWA_ERR_UNSUPPORTED = 161100,   /* valid per the API but not built (e.g. D past 128 or not a multiple of 8) */
  SWA_ERR_WORKSPACE = 161101,     /* workspace NULL or smaller than the size query says */
  SWA_ERR_CUDA = 161102,          /* a CUDA runtime call failed (text in swa_last_error) */
  SWA_ERR_TIMEOUT = 161103,       /* a kernel gave up a bounded wait (swa_workspace_status) */
  SWA_ERR_BOUNDS = 161104,        /* bounds-checked build only: a kernel skipped an access outside its
                                     tensor (swa_workspace_status) */
  SWA_ERR_PAGE = 161105           /* a block table entry or a cache length that a paged call read on the
                                     device is out of range (swa_paged_forward_status,
                                     swa_paged_append_status) */
} swa_status_t;

typedef struct {
  int32_t layout;               /* swa_layout_t */
  int64_t B, N, D;              /* batch, heads (headNum), head dim (8..128, a multiple of 8) */
  int64_t S_q, S_kv;            /* BNSD sequence lengths (ignored for TND) */
  int64_t T_q, T_kv;            /* TND total rows (ignored for BNSD) */
  const int64_t *cu_seqlens_q;  /* TND: host, length B, cumulative ends (see above) */
  const int64_t *cu_seqlens_kv; /* TND: host, length B */
  double scale;                 /* score scale, default 1.0, usually D^-0.5 */
  int64_t pre_tokens;           /* BAND left extent, default 2147483647 */
  int64_t next_tokens;          /* BAND right extent, default 2147483647 */
  int32_t sparse_mode;          /* 0 or 4 */
  double keep_prob;             /* dropout keep probability in (0, 1], default 1.0 */
  int64_t N_kv;                 /* key/value heads for grouped-query attention: N must be a
                                   multiple of N_kv (aclnnFlashAttentionUnpaddingScoreGradV2
                                   article, shape constraints: Nq/Nkv a non-zero integer);
                                   query head n reads key/value head n / (N / N_kv).
                                   k, v, dk, dv then have N_kv heads ([B,N_kv,S_kv,D] or
                                   [T_kv,N_kv,D]).  0 (the default) means N_kv = N. */
  int32_t dropout_gen;          /* 1: keep_prob < 1 with drop_mask NULL, the mask being the one
                                   dropout_seed / dropout_offset stand for (see above); 0: the
                                   caller's drop_mask.  Default 0. */
  uint64_t dropout_seed;
  uint64_t dropout_offset;
  int32_t dtype;                /* element type of q, k, v, dy, out, dq, dk, dv (doc: FLOAT16 /
                                   BFLOAT16 / FLOAT32): SWA_DTYPE_BF16 (0, default),
                                   SWA_DTYPE_FP16 (1) or SWA_DTYPE_FP32 (2).  fp32: the
                                   tensor-core operands are bf16 copies of the inputs
                                   (rounded to nearest even, made in the workspace), every
                                   accumulation is fp32 as for the other types, and the
                                   outputs are stored in fp32 */
  int64_t sink_tokens;          /* BAND: the first sink_tokens keys of a sequence stay visible behind
                                   the window: query i sees key j iff j <= i + next_tokens and
                                   (j >= i - pre_tokens or j < sink_tokens).  Default 0; no effect
                                   without BAND (an addition of this library) */
} swa_params_t;

typedef enum { SWA_DTYPE_BF16 = 0, SWA_DTYPE_FP16 = 1, SWA_DTYPE_FP32 = 2 } swa_dtype_t;

/* Fill `p` with the documented defaults (FlashAttentionScore REG_OP
 * attribute defaults): scale 1.0, keep_prob 1.0, pre/next 2147483647,
 * sparse_mode 0; everything else zero / NULL. */
SWA_API void swa_params_default(swa_params_t *p);

/* Device workspace bytes that swa_forward needs for these parameters (a
 * status word; the work schedule travels as a kernel parameter; with fp32
 * inputs also bf16 copies of q, k and v).  Errors: SWA_ERR_PARAM_NULLPTR,
 * SWA_ERR_PARAM_INVALID, SWA_ERR_UNSUPPORTED. */
SWA_API swa_status_t swa_forward_workspace_size(const swa_params_t *p, size_t *bytes);

/* Forward (doc formula; PyPTO-Gym "前向公式").
 *   q, k, v       device, p->dtype (bf16 / fp16 / fp32), layout per p->layout
 *   drop_mask     device, packed keep bits, 16-byte aligned; NULL iff keep_prob == 1
 *                 or dropout_gen == 1
 *   out           device, p->dtype, q's shape
 *   softmax_max   device, fp32, [B,N,S_q] or [T_q,N]
 *   softmax_sum   device, fp32, same shape
 *   workspace     device, >= swa_forward_workspace_size bytes, 256-byte aligned
 * Errors: the size query's, plus SWA_ERR_WORKSPACE and SWA_ERR_CUDA.  Nothing
 * is enqueued when a status other than SWA_OK is returned. */
SWA_API swa_status_t swa_forward(const swa_params_t *p, const void *q, const void *k, const void *v,
                         const uint8_t *drop_mask, void *out, float *softmax_max, float *softmax_sum,
                         void *workspace, size_t workspace_bytes, swa_stream_t stream);

/* Device workspace bytes that swa_backward needs: a status word, and per
 * query row D = rowsum(dY*O) and the log2-sum-exp of the forward statistics
 * (8 bytes per query row and head); with fp32 inputs also bf16 copies of q,
 * k, v, dy and out; with sink_tokens also fp32 partial dk and dv rows of the
 * 128-key tiles that hold sinks, whose queries are split over several CTAs
 * (64 KB at D <= 64, else 128 KB, per CTA; the sums have a fixed order). */
SWA_API swa_status_t swa_backward_workspace_size(const swa_params_t *p, size_t *bytes);

/* Backward (PyPTO-Gym "反向公式"; aclnnFlashAttentionUnpaddingScoreGradV2
 * article §2.3).  out / softmax_max / softmax_sum are this library's forward
 * results for the same q, k, v, drop_mask and parameters.
 *   dy            device, p->dtype, q's shape (gradient of out)
 *   dq, dk, dv    device, p->dtype, shapes of q, k, v; fully overwritten
 * Errors: as swa_forward. */
SWA_API swa_status_t swa_backward(const swa_params_t *p, const void *q, const void *k, const void *v, const void *dy,
                          const void *out, const float *softmax_max, const float *softmax_sum,
                          const uint8_t *drop_mask, void *dq, void *dk, void *dv, void *workspace,
                          size_t workspace_bytes, swa_stream_t stream);

/* swa_backward without a workspace argument, for callers that cannot hand the
 * library device memory (the pages have no counterpart; this is an addition of
 * this library).  Example callers: a plugin inside a framework that owns all
 * device memory through its own pool and forbids extra cudaMalloc calls, or a
 * latency-critical loop that must not allocate after start-up.
 *
 * Arguments and results are those of swa_backward.  The scratch it needs
 * (status word, per-row D and log2-sum-exp) lives in a
 * fixed 64 MiB device array compiled into the library: every GPU that loads
 * the library keeps it until the process exits.  A problem needing more than
 * 64 MiB of scratch (swa_backward_workspace_size) is rejected with
 * SWA_ERR_WORKSPACE.  Every call looks up the array's device address in the
 * current context (cudaGetSymbolAddress), so an address never outlives its
 * context; the first lookup on a device may load the library's device code,
 * so make the first call before any stream capture.  The library carries its
 * own copy of the CUDA runtime (linked statically): do not reset the device
 * (cudaDeviceReset, or a primary-context reset through the driver) between
 * calls while the library stays loaded, since whether its runtime then
 * reloads its device code is not specified.  All calls on a device
 * share the array and
 * each call clears what must start at zero, so calls whose kernels overlap on
 * the GPU (concurrent streams, other threads) race and must be serialised by
 * the caller.  Allocates nothing: no cudaMalloc, cudaFree or allocating
 * library routine.  The status word of a bounded wait that gave up is not
 * observable through this entry point. */
SWA_API swa_status_t swa_backward_noalloc(const swa_params_t *p, const void *q, const void *k, const void *v,
                                          const void *dy, const void *out, const float *softmax_max,
                                          const float *softmax_sum, const uint8_t *drop_mask, void *dq, void *dk,
                                          void *dv, swa_stream_t stream);

/* Forward + backward of one problem whose tensors live in HOST memory (an
 * addition of this library; the pages' operators take device tensors).  The
 * heads are split into `chunks` equal groups; the first group is split into
 * halves, its first half again, and so on while 2^l * chunks divides N and
 * N_kv (at most three levels), and the last group the same way mirrored, so
 * that less is copied before the first computation and after the last.  Each
 * group is copied to its own compact device tensors inside `device_buffer`,
 * computed (swa_forward, then swa_backward) and copied back, and the copies
 * of the next and the previous group run on internal streams while a group
 * computes.  A group's forward starts once its q, k and v are in, and its
 * out and statistics go back while its backward runs.  Consecutive groups
 * compute on two further internal streams in turn, so one group's kernels
 * may start while the previous group's last CTAs still run; each of those
 * has its own device -> host stream.  The five internal streams and their
 * events are created by the first call in a CUDA context and kept until the
 * process exits; calls in one context share them (their enqueueing is
 * serialised by a lock, and their GPU work runs one call after the other).
 * Heads are independent, so the results equal those of one swa_forward +
 * swa_backward on device copies of the same tensors, bit for bit.
 *   q, k, v, dy   host, p->dtype, shapes and layout as for swa_forward /
 *                 swa_backward; page-locked memory lets the copies overlap
 *   out, softmax_max, softmax_sum, dq, dk, dv
 *                 host, written when `stream` completes
 *   chunks        >= 1, dividing N and N_kv.  Dropout needs dropout_gen = 1
 *                 and chunks = 1: there is no drop_mask argument, and the
 *                 generated keep bits are indexed by the whole problem's heads
 *   device_buffer device, >= swa_step_host_buffer_size bytes, 256-byte aligned
 * All work is enqueued behind the work already on `stream`, and `stream`
 * completes only once every result is in host memory.  Errors: those of
 * swa_forward / swa_backward, SWA_ERR_PARAM_INVALID (chunks), and
 * SWA_ERR_CUDA.  On an error part of the work may already be enqueued;
 * `stream` then still completes only after every copy enqueued by the call
 * has run, so the host buffers may be released once it has. */
SWA_API swa_status_t swa_step_host_buffer_size(const swa_params_t *p, int chunks, size_t *bytes);
SWA_API swa_status_t swa_step_host(const swa_params_t *p, int chunks, const void *q, const void *k,
                                   const void *v, const void *dy, void *out, float *softmax_max,
                                   float *softmax_sum, void *dq, void *dk, void *dv, void *device_buffer,
                                   size_t device_bytes, swa_stream_t stream);
/* swa_workspace_status over every chunk's forward and backward workspace
 * inside a swa_step_host device_buffer. */
SWA_API swa_status_t swa_step_host_status(const swa_params_t *p, int chunks, const void *device_buffer,
                                          swa_stream_t stream);

/* Write the keep mask that p->dropout_seed / p->dropout_offset stand for
 * (see "Dropout" above) in the drop_mask layout: ceil(bits / 8) bytes, bits =
 * sum over sequences of N * Sq_b * Skv_b.  mask is device memory of
 * mask_bytes bytes; bytes past the last element are zero.  It lets a caller
 * keep or inspect the mask a seed-driven call used; the pages' low-level
 * backward takes it as drop_mask.  Errors: the size query's,
 * SWA_ERR_PARAM_NULLPTR, SWA_ERR_WORKSPACE (mask_bytes too small),
 * SWA_ERR_CUDA. */
SWA_API swa_status_t swa_dropout_mask(const swa_params_t *p, uint8_t *mask, size_t mask_bytes,
                                      swa_stream_t stream);

/* ------------------------------------------------------------------------
 * Rotary positions, a paged key/value cache, and attention over it
 * (additions of this library; the pages have no counterpart): what runs
 * beside swa_forward when a model with the BAND window is trained or served.
 *
 * Rotation.  The first rotary_dim = R elements of every head row are R/2
 * pairs.  Pair i of the row at integer positions pos[0..n_axes) is turned by
 * the angle t = pos[pair_axis[i]] * inv_freq[i] (radians):
 *   (a, b) -> (a cos t - b sin t, b cos t + a sin t)
 * Pair i is elements (i, i + R/2), or (2i, 2i + 1) when interleaved = 1.
 * Elements past R are copied.  The backward turns by -t (the transpose of the
 * rotation).  The angle is formed as pos * inv_freq / 2 pi modulo 1 in 64-bit
 * fixed point, with inv_freq / 2 pi modulo 1 rounded once to 2^-64, so positions
 * anywhere in the int32 range keep the accuracy of small ones (within 2^-34
 * turns, for the inv_freq that is given); the products are fp32 and rounded once
 * to the element type.
 *
 * Every tensor may be strided: a swa_strides_t gives the distances, in
 * elements, between batches, rows (tokens) and heads; a NULL stands for the
 * dense layout.  The D elements of a head row are contiguous; tensors start
 * on 16 bytes and strides are multiples of 8 elements (q and k may so be
 * slices of one fused projection).  Inputs may repeat rows (stride 0); the
 * strides of a result, in ascending order, are each past all that the smaller
 * ones span. */
typedef struct {
  int64_t batch, row, head; /* elements; batch is unused for TND */
} swa_strides_t;

typedef struct {
  int32_t layout;           /* swa_layout_t: BNSD [B,N,S,D], or TND [B*S,N,D] */
  int64_t B, S;             /* batch, rows; positions are [n_axes, B*S] */
  int64_t N, D;             /* heads of q, head dim (8..128, a multiple of 8) */
  int64_t N_kv;             /* heads of k; 0 (the default) means N_kv = N */
  int64_t rotary_dim;       /* R, a multiple of 8 up to D; 0 (the default) means D */
  int32_t n_axes;           /* 1..4, default 1 */
  const int32_t *pair_axis; /* host, R/2 axis indices, or NULL: every pair on axis 0 */
  const double *inv_freq;   /* host, R/2 angles per position (radians, finite, |.| <= 2^20), or NULL:
                               base^(-2i/R) for pair i */
  double base;              /* default 10000; > 0 and finite */
  int32_t interleaved;      /* 0 (default): pairs (i, i + R/2); 1: pairs (2i, 2i + 1) */
  int32_t dtype;            /* swa_dtype_t of q, k and the results */
} swa_rope_params_t;

/* Fill `p` with the defaults named above; everything else zero / NULL. */
SWA_API void swa_rope_params_default(swa_rope_params_t *p);

/* Rotate q and k (either may be NULL, with its result; not both).
 *   q, k          device, p->dtype, N and N_kv heads
 *   positions     device, int32 [n_axes, B*S], row b*S + s of a BNSD batch
 *   q_out, k_out  device, p->dtype; may be q and k themselves with the same
 *                 strides (in place), must not overlap them otherwise
 * swa_rope_backward takes the gradients of q_out and k_out and writes those of
 * q and k.  Neither needs a workspace.
 * Errors: SWA_ERR_PARAM_NULLPTR, SWA_ERR_PARAM_INVALID, SWA_ERR_UNSUPPORTED,
 * SWA_ERR_CUDA; nothing is enqueued when a status other than SWA_OK is
 * returned. */
SWA_API swa_status_t swa_rope_forward(const swa_rope_params_t *p, const void *q, const swa_strides_t *q_strides,
                                      const void *k, const swa_strides_t *k_strides, const int32_t *positions,
                                      void *q_out, const swa_strides_t *q_out_strides, void *k_out,
                                      const swa_strides_t *k_out_strides, swa_stream_t stream);
SWA_API swa_status_t swa_rope_backward(const swa_rope_params_t *p, const void *dq_out,
                                       const swa_strides_t *dq_out_strides, const void *dk_out,
                                       const swa_strides_t *dk_out_strides, const int32_t *positions, void *dq,
                                       const swa_strides_t *dq_strides, void *dk, const swa_strides_t *dk_strides,
                                       swa_stream_t stream);

/* Paged cache.  Keys and values of all sequences live in pages of page_size
 * tokens.  Token j of sequence b is slot j mod page_size of page
 * block_table[b][j / page_size].  A page is laid out as its batch entry would
 * be: cache_layout BNSD [num_pages, N_kv, page_size, D], TND
 * [num_pages, page_size, N_kv, D]; other strides by a swa_page_strides_t
 * (NULL: dense): multiples of 8 elements, and in ascending order each a
 * multiple of the one before and past all its entries (as a tensor map
 * needs), so K and V may share one allocation.  Page offsets are 64-bit.
 *
 * The new tokens ("chunk") of all sequences are packed TND: q [T_q, N, D] with
 * the host array cu_seqlens_q as for swa_forward (length-0 sequences and a
 * trailing run of zeros allowed).  kv_lens[b] (device, so that a captured graph
 * can be replayed as the sequences grow) is the length of sequence b with its
 * chunk, q_len_b: chunk token i has position kv_lens[b] - q_len_b + i.  A
 * token whose position is negative does not exist in the cache (a padded
 * batch may so give an unused sequence kv_lens[b] = 0): it is not stored, and
 * its attention follows the formula, the BAND around its position.
 *
 * kv_lens and block_table are read on the device.  A length outside
 * [0, min(max_kv_len, max_pages * page_size)] counts as 0, and a page number
 * outside [0, num_pages) is never followed: its tokens are not stored, and
 * read as zero keys and values.  Both are reported by the status calls as
 * SWA_ERR_PAGE.  Only entries of pages that hold a token of the chunk (append)
 * or a key that some query of the chunk sees (attention) are looked at: pages
 * that fell out of the BAND window may be freed and their entries hold
 * anything.  What a page holds at slots no query of the call sees (past a
 * sequence's length, before its window) is ignored, NaN and infinity included.
 * A non-finite key or value that one query of a chunk sees may reach every
 * query of that chunk. */
typedef struct {
  int64_t page, head, slot; /* elements between pages, heads and slots */
} swa_page_strides_t;

typedef struct {
  int64_t B, N, D;             /* sequences, query heads, head dim (8..128, a multiple of 8) */
  int64_t N_kv;                /* key/value heads; 0 (the default) means N_kv = N; N a multiple of N_kv */
  int64_t T_q;                 /* rows of the packed chunk */
  const int64_t *cu_seqlens_q; /* host, length B, cumulative ends as in swa_params_t */
  int32_t cache_layout;        /* swa_layout_t of a page */
  int64_t num_pages;           /* pages of the cache, 1..2^31 - 1 */
  int64_t page_size;           /* tokens per page, a multiple of 16 up to 65536 */
  int64_t max_pages;           /* block table columns, 1..2^24 */
  int64_t max_kv_len;          /* largest kv_lens[b] of any (re)play of this call, up to 2^28; 0 (the
                                  default): max_pages * page_size.  How the keys are split over the GPU
                                  follows from it, whatever the lengths are: without a window, up to 16
                                  query rows of a sequence and key/value head take a CTA, and up to 8 KB
                                  of workspace, per 16384 keys of this bound (1536 with an 8-bit cache,
                                  where a bound far above the lengths costs time too: 64 sequences of 100
                                  to 16384 keys, 32 / 8 heads of 128, take 199 us with a bound of 16384
                                  keys, 294 with 131072 and 1066 with 2^20) */
  double scale;                /* score scale, default 1.0 */
  int64_t pre_tokens;          /* BAND, around each token's position; defaults 2147483647 */
  int64_t next_tokens;
  int32_t sparse_mode;         /* 0 (every cached token is visible) or 4 (BAND) */
  int32_t dtype;               /* SWA_DTYPE_BF16 (0, default) or SWA_DTYPE_FP16: q, k, v, out and the
                                  pages (unless cache_dtype says otherwise).  fp32 is not built
                                  (SWA_ERR_UNSUPPORTED) */
  int64_t sink_tokens;         /* BAND: the first sink_tokens tokens of a sequence stay visible behind the
                                  window, as in swa_params_t; default 0, no effect without BAND */
  int32_t cache_dtype;         /* swa_cache_t: what the pages hold, SWA_CACHE_SAME (0, default) or
                                  SWA_CACHE_E4M3 (1), see "8-bit cache" */
} swa_paged_params_t;

typedef enum { SWA_CACHE_SAME = 0, SWA_CACHE_E4M3 = 1 } swa_cache_t;

/* 8-bit cache (cache_dtype SWA_CACHE_E4M3).  The pages hold e4m3 codes (a sign,
 * 4 exponent bits of bias 7, 3 mantissa bits; one byte each, page strides in
 * bytes, still multiples of 8), and two arrays int8 [num_pages, N_kv, page_size],
 * dense whatever the layout of the pages and starting on 16 bytes, hold an
 * exponent per token and key/value head: the row stands for code * 2^exponent,
 * which dtype holds exactly.
 * swa_paged_append_ext quantises: exponent = the least integer e with
 * max |x| <= 448 * 2^e over the row (after the rotation, in fp32), held within
 * [-100, 7] (bf16) or [-15, 7] (fp16); code = x * 2^-e rounded once to nearest
 * even.  Infinities and values past 448 * 2^7 = 57344 saturate there, and so may
 * only cost their own precision and that of what is 2^-15 of them; a row with a
 * NaN gets exponent 127.
 * Readers take an exponent above 7 for a row of NaN, one below the least for
 * the least; what the NaN codes (0x7F, 0xFF) stand for under another exponent
 * is not defined (NaN or 480 * 2^e).
 * A slot that no query of a call sees is ignored, its exponent included.
 * Attention of up to 16 query rows per sequence and key/value head rounds the
 * weight of a value with its exponent, P * 2^exponent, to fp16 relative to the
 * largest that the query row has: to 11 bits down to 2^-20 of it, and to 2^-31 of it
 * below; q (bf16) loses what is below 2^-39 of its row's largest.  With more rows
 * the keys and values are exact and the weights as without the cache. */

SWA_API void swa_paged_params_default(swa_paged_params_t *p);

/* Store a chunk's keys and values in the cache.
 *   k, v          device, p->dtype, [T_q, N_kv, D]
 *   k_pages, v_pages
 *                 device; only the chunk's slots are written.  Two chunk
 *                 tokens must not map to one slot
 *   block_table   device, int32 [B, max_pages], rows table_stride entries
 *                 apart (0: max_pages)
 *   kv_lens       device, int32 [B], lengths with the chunk
 *   rope          NULL, or a rotation applied to k on its way into the cache
 *                 (layout TND, B*S = T_q, the same N, N_kv, D and dtype); v is
 *                 never rotated
 *   positions     device, int32 [n_axes, T_q], or NULL: every axis at the
 *                 token's position in its sequence (0 where that is negative)
 *   q, q_out      NULL, or (with rope only) queries [T_q, N, D] rotated along
 *                 with k into q_out, in the same launch; q_out may be q itself
 *                 with the same strides
 *   workspace     device, >= swa_paged_append_workspace_size bytes, 256-byte
 *                 aligned; holds the status only
 * Errors: as swa_rope_forward, plus SWA_ERR_WORKSPACE. */
SWA_API swa_status_t swa_paged_append_workspace_size(const swa_paged_params_t *p, size_t *bytes);
SWA_API swa_status_t swa_paged_append(const swa_paged_params_t *p, const void *k, const swa_strides_t *k_strides,
                                      const void *v, const swa_strides_t *v_strides, void *k_pages,
                                      const swa_page_strides_t *k_page_strides, void *v_pages,
                                      const swa_page_strides_t *v_page_strides, const int32_t *block_table,
                                      int64_t table_stride, const int32_t *kv_lens, const swa_rope_params_t *rope,
                                      const int32_t *positions, const void *q, const swa_strides_t *q_strides,
                                      void *q_out, const swa_strides_t *q_out_strides, void *workspace,
                                      size_t workspace_bytes, swa_stream_t stream);

/* swa_paged_append with an 8-bit cache too.
 *   k_exponents, v_exponents
 *                 device, int8 [num_pages, N_kv, page_size], 16-byte aligned;
 *                 only the chunk's slots are written.  NULL iff the cache is
 *                 not 8-bit (swa_paged_append refuses an 8-bit cache) */
SWA_API swa_status_t swa_paged_append_ext(const swa_paged_params_t *p, const void *k, const swa_strides_t *k_strides,
                                          const void *v, const swa_strides_t *v_strides, void *k_pages,
                                          const swa_page_strides_t *k_page_strides, void *v_pages,
                                          const swa_page_strides_t *v_page_strides, int8_t *k_exponents,
                                          int8_t *v_exponents, const int32_t *block_table, int64_t table_stride,
                                          const int32_t *kv_lens, const swa_rope_params_t *rope,
                                          const int32_t *positions, const void *q, const swa_strides_t *q_strides,
                                          void *q_out, const swa_strides_t *q_out_strides, void *workspace,
                                          size_t workspace_bytes, swa_stream_t stream);

/* Read a chunk's keys and values back from the cache, 16-bit or 8-bit: what
 * swa_paged_append stored (N, scale, window and sinks are not used).  With
 * chunks as long as the sequences it copies those out whole.
 *   k_pages, v_pages, k_exponents, v_exponents, block_table, table_stride, kv_lens
 *                 as for swa_paged_append_ext; read only
 *   k, v          device, p->dtype, [T_q, N_kv, D]; must not overlap the pages.
 *                 Tokens that do not exist in the cache, and those of a page
 *                 number or length out of range, come back as zeros
 *   workspace     as for swa_paged_append (swa_paged_append_workspace_size;
 *                 swa_paged_append_status reports)
 * Errors: as swa_paged_append. */
SWA_API swa_status_t swa_paged_gather(const swa_paged_params_t *p, const void *k_pages,
                                      const swa_page_strides_t *k_page_strides, const void *v_pages,
                                      const swa_page_strides_t *v_page_strides, const int8_t *k_exponents,
                                      const int8_t *v_exponents, const int32_t *block_table, int64_t table_stride,
                                      const int32_t *kv_lens, void *k, const swa_strides_t *k_strides, void *v,
                                      const swa_strides_t *v_strides, void *workspace, size_t workspace_bytes,
                                      swa_stream_t stream);

/* Attention of a chunk over the cache (which holds the chunk's own tokens
 * too): swa_forward's formula with query i of sequence b at position
 * p = kv_lens[b] - q_len_b + i, which sees key j iff p - pre_tokens <= j <=
 * p + next_tokens and 0 <= j < kv_lens[b] (mode 4; with sink_tokens also the
 * keys j < sink_tokens up to p + next_tokens), or every key (mode 0).  A
 * row that sees no key gets out = 0, softmax_max = -inf, softmax_sum = 0.
 * Scores (q.k before the scale too), statistics and sums are fp32; exp(scale q.k -
 * maximum) is rounded to p->dtype before the product with V, as in swa_forward,
 * and out once more.
 *   q             device, p->dtype, [T_q, N, D], may be strided, its rows and
 *                 heads apart (no stride 0)
 *   k_pages, v_pages, block_table, table_stride, kv_lens
 *                 as for swa_paged_append; read only
 *   out           device, p->dtype, dense [T_q, N, D]
 *   softmax_max, softmax_sum
 *                 device, fp32 [T_q, N]; either may be NULL
 *   workspace     device, >= swa_paged_forward_workspace_size bytes, 256-byte
 *                 aligned: status, and the partial results of keys split over
 *                 several CTAs.  Needs no initialisation; a workspace may be
 *                 reused by later calls on the same stream, but not by calls
 *                 (or replays of graphs) running concurrently, nor by calls that
 *                 several threads make at once, on one stream either (a call is
 *                 several launches)
 * Errors: as swa_forward.  The results do not depend on how the keys were
 * split beyond fp32 rounding, and are the same bits from run to run. */
SWA_API swa_status_t swa_paged_forward_workspace_size(const swa_paged_params_t *p, size_t *bytes);
SWA_API swa_status_t swa_paged_forward(const swa_paged_params_t *p, const void *q, const swa_strides_t *q_strides,
                                       const void *k_pages, const swa_page_strides_t *k_page_strides,
                                       const void *v_pages, const swa_page_strides_t *v_page_strides,
                                       const int32_t *block_table, int64_t table_stride, const int32_t *kv_lens,
                                       void *out, float *softmax_max, float *softmax_sum, void *workspace,
                                       size_t workspace_bytes, swa_stream_t stream);

/* The same with an 8-bit cache, and of a chunk that is a tree of drafted tokens
 * (speculative decoding: several continuations in one call).
 *
 * Tree.  Row t of `tree` has bit c (bit c mod 32 of word c / 32) set iff chunk
 * token t of its sequence sees token c of the same chunk: its ancestors and
 * itself, or whatever the caller chooses; bits from the chunk's length on are
 * ignored, and a row may be empty.  Of the keys before the chunk a token sees
 * those that swa_paged_forward's formula gives for position kv_lens[b] - q_len_b +
 * depth, depth[t] being its distance from the root (held within [0, q_len_b - 1]);
 * with next_tokens >= 0, as a tree needs, that is its window and the sinks (a
 * negative pre_tokens leaves the sinks).  The tree alone decides on the chunk's
 * own keys.  The slots hold the chunk in its order, whatever the depths: its
 * tokens are appended as they come, rotated by `positions` of
 * kv_lens[b] - q_len_b + depth.  What is read: pages of keys from the root's window
 * on, the sinks' and the chunk's, every slot of the chunk counting as seen.
 * Afterwards the accepted tokens are appended again in their order, over the
 * chunk.
 *   extra         NULL, or host; the pointers in it are device memory:
 *     k_exponents, v_exponents
 *                 as for swa_paged_append_ext; NULL iff the cache is not 8-bit.
 *                 What sequences of more than 16 query rows per key/value head see
 *                 of an 8-bit cache is first written out as 16-bit pages in the
 *                 workspace: 4 N_kv D bytes per key that such a sequence may see
 *                 (max_kv_len, or its window, chunk and sinks; to 128 keys), for
 *                 as many sequences at a time as fit 1 GB, and 4 B bytes per 128
 *                 keys of max_kv_len.  That is once a chunk for a prompt's, but all
 *                 of the context at every call for a few drafted tokens: 64 sequences
 *                 of 100 to 16384 keys, 32 / 8 heads of 128, take 286 us with 4 tokens
 *                 each (16 rows) and 1060 with 5 to 8 (367 over a 16-bit cache)
 *     tree        uint32 [T_q, words], rows tree_stride words apart (0: the words
 *                 of the longest chunk, ceil(q_len / 32)); NULL: no tree
 *     depth       int32 [T_q], or NULL: the token's place in its chunk */
typedef struct {
  const int8_t *k_exponents, *v_exponents;
  const uint32_t *tree;
  int64_t tree_stride;
  const int32_t *depth;
} swa_paged_extra_t;
SWA_API swa_status_t swa_paged_forward_ext(const swa_paged_params_t *p, const void *q, const swa_strides_t *q_strides,
                                           const void *k_pages, const swa_page_strides_t *k_page_strides,
                                           const void *v_pages, const swa_page_strides_t *v_page_strides,
                                           const swa_paged_extra_t *extra, const int32_t *block_table,
                                           int64_t table_stride, const int32_t *kv_lens, void *out,
                                           float *softmax_max, float *softmax_sum, void *workspace,
                                           size_t workspace_bytes, swa_stream_t stream);

/* Wait for `stream`, then report what the last paged call that used
 * `workspace` met on the device: SWA_OK, SWA_ERR_PAGE (a length or page number
 * out of range, see above), SWA_ERR_TIMEOUT, or SWA_ERR_BOUNDS (bounds-checked
 * build).  `p` as in that call, with the same device current. */
SWA_API swa_status_t swa_paged_append_status(const swa_paged_params_t *p, const void *workspace,
                                             swa_stream_t stream);
SWA_API swa_status_t swa_paged_forward_status(const swa_paged_params_t *p, const void *workspace,
                                              swa_stream_t stream);

/* Wait for `stream`, then report whether any kernel of the last call that
 * used `workspace` gave up a bounded wait: SWA_OK or SWA_ERR_TIMEOUT
 * (SWA_ERR_CUDA if the stream itself failed).  In the bounds-checked build
 * (compiled with SWA_CHECKS = 1; its kernels test every global load and
 * store against the extent of its tensor and skip it when outside) a
 * skipped access reports SWA_ERR_BOUNDS. */
SWA_API swa_status_t swa_workspace_status(const void *workspace, swa_stream_t stream);

/* Measurement support.  `events` is NULL (stop recording) or an array of
 * eight cudaEvent_t handles owned by the caller: {forward start, forward
 * stop, dK/dV start, dK/dV stop, dQ start, dQ stop, preprocess start,
 * preprocess stop}.  Later calls on this thread record each pair on their
 * stream immediately around the corresponding kernel launch (swa_forward's
 * forward kernel; swa_backward's key-major dK/dV kernel, with sink_tokens and
 * the sum of its pieces, query-major dQ kernel and D / lse2 preprocess).  No
 * other effect. */
SWA_API void swa_set_timing_events(void *const *events);

/* Test and inspection support (additions of this library; the pages have no
 * counterpart).
 *
 * swa_debug_schedule: the work items that the band / varlen tile scheduler
 * hands to the kernels of one pass, computed on the host by the same code
 * the kernels run (no GPU needed).  The window is the BAND inequality of the
 * FlashAttentionVarLenScore doc (preTokens / nextTokens as the left and right
 * edges): a 128-row query tile touches one run of 128-row key tiles and a
 * key tile one run of query tiles; tiles outside the runs are skipped.
 *   pass 0   query-major dQ pass (and the forward one CTA per query tile):
 *            one item per query tile of each (batch, query head); partners
 *            are key tiles
 *   pass 1   key-major dK / dV pass: one item per key tile of each (batch,
 *            key/value head); partners are query tiles, walked for every
 *            query head of the group
 *   pass 2   the forward one CTA per pair of query tiles (D <= 64, when the
 *            pairs fill every SM): one item per pair p (query tiles 2p and
 *            2p + 1) of each (batch, query head); partners are the key tiles
 *            from the first start to the last end of the two tiles' runs
 *   items    host, 6 int32 per item in launch order: launch index, batch,
 *            head, tile, first partner tile, partner tile count; at most
 *            `capacity` items are written (items may be NULL to count).
 *            With sink_tokens, an item that also visits sink tiles before its
 *            run has a row for those, before the run's; a key tile whose steps
 *            are split over several CTAs (pass 1) has its row once per CTA
 *   count    host, receives the number of items
 * Errors: the size query's, SWA_ERR_PARAM_NULLPTR (count), and
 * SWA_ERR_PARAM_INVALID (pass).
 *
 * swa_debug_stall: while `kernels` is non-zero, every later call makes the
 * compute warps of the selected kernels (bit 0 forward, bit 1 key-major
 * dK / dV, bit 2 query-major dQ, bit 3 swa_paged_forward's kernel for more
 * than 16 query rows per sequence and key/value head) first wait on a barrier that nothing
 * completes.  That wait gives up after its 2 s limit like any other, the
 * kernel drains its copies and tensor-core work in flight, frees its tensor
 * memory and returns, and swa_workspace_status then reports
 * SWA_ERR_TIMEOUT: it exercises the bounded-wait failure path without a
 * fault.  The outputs of such a call are undefined.  Process-wide; 0 turns
 * it off.
 *
 * swa_debug_forward_pairs: how later forward calls with D <= 64 pick their
 * kernel.  0 (the default): one CTA per pair of query tiles when the pairs
 * fill every SM at least once, else one CTA per query tile; 1: always pairs;
 * 2: never.  Both kernels compute the same results; the switch lets tests
 * reach each on small problems.  Process-wide.
 *
 * swa_debug_extent_slack: every later call takes `elems` (>= 0; negative
 * values count as 0) off each tensor extent that the bounds-checked build
 * (libswa_checked.so, see swa_workspace_status) tests the kernels' global
 * loads and stores against, so that accesses at the end of q / out / dQ,
 * k / dK / dV, the statistics and a stored keep mask count as outside their
 * tensor: they are skipped and the call's status word reports
 * SWA_ERR_BOUNDS.  It exercises that path with accesses that are all in
 * range.  The release build has no such checks and ignores it; the
 * outputs of a call it affects are undefined.  Process-wide; 0 turns it off. */
SWA_API swa_status_t swa_debug_schedule(const swa_params_t *p, int32_t pass, int32_t *items, int64_t capacity,
                                        int64_t *count);
SWA_API void swa_debug_stall(int32_t kernels);
SWA_API void swa_debug_forward_pairs(int32_t mode);
SWA_API void swa_debug_extent_slack(int64_t elems);

/* Text describing the last non-OK status returned on this thread. */
SWA_API const char *swa_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SWA_H */
