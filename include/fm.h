/*
 * fm.h — C ABI of the GB300 (sm_103a) FlashMask-style masked attention library.
 *
 * The method (FlashMask, arXiv 2410.01359, abstract): attention masks are
 * carried as O(N) column-wise bounds instead of a dense N x N matrix, and the
 * kernels use them to skip (Q-tile, KV-tile) blocks that are fully masked,
 * run fully visible blocks without any mask arithmetic, and apply the
 * per-element mask only on the remaining boundary blocks (blog post
 * "FlashMask技术", §2.2, three-way block decision).  The result is plain
 * masked softmax attention, exactly (blog §2.2, "mathematically
 * equivalent"; abstract, "without sacrificing computational accuracy").
 *
 * Mask encoding used throughout: for batch b, mask head hm and key column j,
 *     lower masked rows [lts_j, lte_j)   and   upper masked rows [uts_j, ute_j)
 * (half-open; start >= end is an empty range; all values in [0, N]).
 * Element (i, j) is masked when query row i lies in either range.  The
 * arrays are int32 [B, Hm, N], row-major; Hm is 1 (one mask for all heads)
 * or H (one mask per head).  Head h reads mask head (Hm == 1 ? 0 : h).
 *
 * Tensors: Q, K, V, dO are bf16 [B, H, N, d] contiguous (d = 64 or 128);
 * lse is fp32 [B, H, N] (natural log); outputs are bf16 or fp32 [B, H, N, d].
 *
 * Conventions
 *  - Memory: every buffer is allocated by the caller.  The library allocates
 *    no device memory and keeps no pointer after a call returns.
 *  - Device calls are asynchronous on the given stream (NULL = legacy
 *    default stream).  Argument errors are returned before anything is
 *    launched.  Errors the device detects (a bound outside [0, N], a plan
 *    that does not match the call, a pipeline wait that ran out) are written
 *    to the caller's int32 dev_status (zero it first; the first error wins)
 *    and read by the caller after synchronising.
 *  - Device pointers must be 16-byte aligned.
 *  - Thread safety: calls may be made from several host threads.
 */
#ifndef FM_H_
#define FM_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FM_API __attribute__((visibility("default")))
#else
#define FM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FM_OK = 0,
    FM_ERR_INVALID_ARG = 1,      /* null / misaligned pointer, bad size or dtype          */
    FM_ERR_UNSUPPORTED = 2,      /* head dim, tile size or device not supported          */
    FM_ERR_UNREPRESENTABLE = 3,  /* row-form mask with > 2 masked ranges in some column  */
    FM_ERR_BAD_BOUNDS = 4,       /* a bound outside [0, N] (host or device detected)     */
    FM_ERR_PLAN_MISMATCH = 5,    /* plan built for other shapes or tile sizes            */
    FM_ERR_WORKSPACE = 6,        /* workspace missing or too small                       */
    FM_ERR_CUDA = 7,             /* a CUDA runtime / driver call failed                  */
    FM_ERR_TIMEOUT = 8,          /* a bounded device-side wait ran out (kernel returned) */
    FM_ERR_DEBUG_CHECK = 9,      /* a device-side check of an FM_DEBUG build failed      */
    FM_ERR_LENGTHS = 10,         /* request lengths outside the sizes of the step        */
    FM_ERR_PAGES = 11,           /* too few free pages, or a page or slot out of range   */
    FM_ERR_PROBS = 12            /* a drafted token or a row of probabilities that cannot be used */
} fm_status;

enum { FM_TILE_SKIP = 0, FM_TILE_FULL = 1, FM_TILE_PARTIAL = 2 };
enum { FM_DT_BF16 = 0, FM_DT_F32 = 1, FM_DT_E4M3 = 2 /* paged caches only */ };

/* Flags of fm_attn_fwd / fm_attn_bwd.
 * FM_FLAG_PRECISE: the softmax probabilities P (forward and backward) and dS
 * (backward) enter the tensor-core products as two bf16 terms, x = hi + lo
 * with hi = bf16(x), lo = bf16(x - hi), instead of one bf16 rounding.  The
 * products keep ~16 significant bits of P and dS (more tensor-core work:
 * 1.5x the forward PV product, 1.6x the backward products).  Without it the
 * kernels use the usual FlashAttention arithmetic (bf16 P and dS operands,
 * fp32 accumulation).  Use it when gradients are large (|dQ| of tens), where
 * one bf16 rounding of dS and of O (through D) shows in the result. */
enum { FM_FLAG_PRECISE = 1 };

/* Same type as cudaStream_t, so a cudaStream_t can be passed directly. */
typedef struct CUstream_st *fm_stream_t;

/* Column-bound mask; the four pointers are DEVICE arrays int32 [B, Hm, N]. */
typedef struct {
    const int32_t *lts, *lte, *uts, *ute;
    int32_t B, Hm, N;
} fm_bounds;

/* Human-readable name of a status code (static storage). */
FM_API const char *fm_status_string(fm_status st);

/* Library ABI version (incremented when a signature changes). */
FM_API int fm_abi_version(void);

/*
 * fm_mask_from_rows — HOST, synchronous.
 * Passage: blog "FlashMask技术" §2.1 (causal example) and §3.3 (document
 * packing): one inclusive attend interval [cs_i, ce_i] per query row.
 * cs, ce: host int32 [B, Hm, N]; cs_i > ce_i is an empty row; otherwise
 * 0 <= cs_i <= ce_i < N is required (else FM_ERR_BAD_BOUNDS).
 * Writes the column form to host arrays lts, lte, uts, ute [B, Hm, N]:
 * for each column the rows that do NOT attend it must form at most two
 * ranges (else FM_ERR_UNREPRESENTABLE, outputs then undefined).  A masked
 * range that starts at row 0 is stored as the upper range, any other (or the
 * second of two) as the lower range; empty ranges are written canonically,
 * lower (N, N) and upper (0, 0).  Runs in O(N) per (b, hm).
 */
FM_API fm_status fm_mask_from_rows(const int32_t *cs, const int32_t *ce, int B, int Hm, int N,
                            int32_t *lts, int32_t *lte, int32_t *uts, int32_t *ute);

/*
 * fm_mask_from_row_intervals — HOST, synchronous.
 * Passage: blog "FlashMask技术" §6.1 item 1 (multi-interval extension:
 * several disjoint attend intervals per row, printed as row 0 -> (0, 100),
 * (200, 300) and row 1 -> (0, 50), (150, 250)), read with the inclusive
 * interval convention of §3.3.  The window-with-sink-tokens mask of the §5
 * streaming-inference example (row i attends [0, sink) and (i - window, i])
 * is such a two-interval row form.
 * starts, ends: host int32 [B, Hm, N, K], K >= 1 interval slots per row;
 * slot (s, e) with s > e is unused; otherwise 0 <= s <= e < N is required
 * (else FM_ERR_BAD_BOUNDS).  Row i attends the union of its intervals, which
 * may overlap, touch or come in any order.  Output and errors as for
 * fm_mask_from_rows (which is the K = 1 case, with identical results): each
 * column's non-attending rows must form at most two ranges, else
 * FM_ERR_UNREPRESENTABLE.  Runs in O(N K log K) per (b, hm).
 */
FM_API fm_status fm_mask_from_row_intervals(const int32_t *starts, const int32_t *ends, int K, int B,
                                     int Hm, int N, int32_t *lts, int32_t *lte, int32_t *uts,
                                     int32_t *ute);

/*
 * Compressed column bounds.  Passage: blog "FlashMask技术" §6.2 item 2
 * (memory compression, next step: differential encoding of the interval
 * vectors and 8-bit integers for the offsets).  Per 128-column block of each
 * of the four bound arrays of each (b, hm): the block's first value as int32
 * and the 127 column-to-column differences as int8 when all fit in
 * [-128, 127], else the block's int32 values; a directory of per-block
 * offsets lets every block decode on its own.  Causal, window, prefix and
 * document masks compress about 3.7x (16 bytes per column to about 4.3).
 *
 * fm_bounds_compressed_bytes — HOST: the exact size of the compressed form of
 *   these host bounds (int32 [B, Hm, N] each), 0 on bad arguments.
 * fm_bounds_compress — HOST, synchronous: writes it into out (out_bytes at
 *   least that size, else FM_ERR_WORKSPACE; bad arguments FM_ERR_INVALID_ARG).
 *   Bounds are stored as given (validated when classified).
 * fm_bounds_decompress — DEVICE, async: expands a compressed buffer (device,
 *   16-byte aligned, `bytes` long) into the caller's device arrays `out`
 *   (whose B, Hm, N must be those it was compressed with).  A buffer whose
 *   header or directory does not match (wrong magic or shape, an entry beyond
 *   the payload) writes FM_ERR_INVALID_ARG to dev_status and nothing is read
 *   beyond `bytes`.  B * Hm <= 65535.
 */
FM_API size_t fm_bounds_compressed_bytes(const int32_t *lts, const int32_t *lte, const int32_t *uts,
                                         const int32_t *ute, int B, int Hm, int N);
FM_API fm_status fm_bounds_compress(const int32_t *lts, const int32_t *lte, const int32_t *uts,
                                    const int32_t *ute, int B, int Hm, int N, void *out, size_t out_bytes);
FM_API fm_status fm_bounds_decompress(const void *cbounds, size_t bytes, fm_bounds out, int32_t *dev_status,
                                      fm_stream_t stream);

/*
 * Plan = tile labels plus, per Q tile, the ordered list of non-skip KV tiles
 * and, per KV tile, the list of non-skip Q tiles (blog §4.1 item 2: decide
 * before a KV block is loaded whether it is needed at all), plus the order in
 * which the attention kernels take their tiles: longest list first, in
 * half-octave length buckets, so that a tile with a long list (sink columns,
 * the first tiles of a long document) starts in the first wave.  Opaque
 * device buffer of fm_plan_bytes() bytes, 256-byte aligned, written by
 * fm_tile_classify and read by fm_attn_fwd / fm_attn_bwd.
 * bq, bk in {64, 128}; the attention kernels need bq = bk = 128.
 * Returns 0 for invalid sizes.
 */
FM_API size_t fm_plan_bytes(int B, int Hm, int N, int bq, int bk);

/*
 * fm_tile_classify — DEVICE, async.
 * Passage: blog §2.2 (skip / full GEMM / masked GEMM per block pair).  The
 * printed test is garbled; the decision implemented is: per KV tile take the
 * min and max of each canonicalised bound (empty lower -> (N, N), empty
 * upper -> (0, 0)) over its columns; for Q rows [qb, qe) the pair is
 *   SKIP    if all columns' lower ranges cover [qb, qe) or all upper ones do,
 *   FULL    if not SKIP and every lower and every upper range misses [qb, qe),
 *   PARTIAL otherwise (tile ends clipped to N).
 * labels (nullable): device uint8 [B, Hm, n_q, n_k] copy of the labels.
 * dev_status: device int32 (required).  Bounds outside [0, N] set
 * FM_ERR_BAD_BOUNDS there.  Three launches on the stream: per-tile bound
 * min/max, labels and lists, work order.
 */
FM_API fm_status fm_tile_classify(fm_bounds m, int bq, int bk, void *plan, size_t plan_bytes,
                           uint8_t *labels, int32_t *dev_status, fm_stream_t stream);

/* Workspace of fm_attn_fwd in bytes (may be 0: then ws may be NULL). */
FM_API size_t fm_fwd_workspace_bytes(int B, int H, int N, int d);

/*
 * fm_attn_fwd — DEVICE, async.
 * Passages: FlashAttention article §二.1-二.3 (tiling, max-subtracted
 * softmax, QK^T and PV fused on tensor cores), blog §2.2 and §4.1 items 2-3
 * (skip blocks before loading them, mask fused into the softmax on boundary
 * blocks only).  Computes, per (b, h),
 *     O = softmax(scale * Q K^T with masked entries removed) V,
 *     lse_i = ln sum_{j attended} exp(scale q_i.k_j)
 * with O_i = 0 and lse_i = -inf for a row that attends nothing.
 * q, k, v: device bf16 [B, H, N, d]; plan from fm_tile_classify(m, 128, 128);
 * o: device [B, H, N, d] of o_dtype (FM_DT_BF16 / FM_DT_F32);
 * lse: device fp32 [B, H, N]; ws: fm_fwd_workspace_bytes() bytes or NULL;
 * flags: 0 or FM_FLAG_PRECISE.
 */
FM_API fm_status fm_attn_fwd(const void *q, const void *k, const void *v, fm_bounds m, const void *plan,
                      int B, int H, int N, int d, float scale, void *o, int o_dtype, float *lse,
                      void *ws, size_t ws_bytes, int flags, int32_t *dev_status,
                      fm_stream_t stream);

/* Workspace of fm_attn_bwd in bytes: fp32 dQ accumulator [B,H,N,d] plus
 * fp32 D = rowsum(dO * O) [B,H,N].  (With fp32 gradients the kernels
 * accumulate dQ in the caller's dq buffer directly and the accumulator
 * part of the workspace is left untouched; the size is the same for both
 * gradient dtypes.) */
FM_API size_t fm_bwd_workspace_bytes(int B, int H, int N, int d);

/*
 * fm_attn_bwd — DEVICE, async.
 * Exact gradient of fm_attn_fwd's O with upstream dO (lse has no upstream
 * gradient); the pages use the method for training (abstract: SFT, LoRA,
 * DPO, RM), which needs these.  With P_ij = exp(scale q_i.k_j - lse_i) on
 * attended pairs (0 elsewhere), D_i = sum_k dO_ik O_ik:
 *     dV = P^T dO,  dP = dO V^T,  dS = P o (dP - D),
 *     dQ = scale dS K,  dK = scale dS^T Q.
 * Same tile skipping as the forward.  o, lse: the forward's outputs (o of
 * o_dtype); dq, dk, dv: device [B, H, N, d] of grad_dtype; flags: 0 or
 * FM_FLAG_PRECISE (with a precise backward, compute O with a precise forward
 * too: D is taken from O); ws: fm_bwd_workspace_bytes() bytes (overwritten).
 */
FM_API fm_status fm_attn_bwd(const void *q, const void *k, const void *v, const void *o, int o_dtype,
                      const float *lse, const void *dO, fm_bounds m, const void *plan, int B,
                      int H, int N, int d, float scale, void *dq, void *dk, void *dv,
                      int grad_dtype, int flags, void *ws, size_t ws_bytes, int32_t *dev_status,
                      fm_stream_t stream);

/*
 * fm_attn_bwd_noalloc — DEVICE, async.  No counterpart in the paper: this
 * entry point exists for callers that may not allocate device memory (code
 * running under another framework's allocator, latency-critical loops that
 * must not call cudaMalloc after start-up, plugins handed only their input
 * and output buffers).  Same contract and results as fm_attn_bwd, but the
 * workspace comes from a fixed array inside the library instead of the
 * caller, so nothing is allocated.
 * Limit: fm_bwd_workspace_bytes(B, H, N, d) <= FM_NOALLOC_SCRATCH_BYTES
 * (64 MiB: about 130,000 rows B*H*N at d = 128); larger sizes return
 * FM_ERR_WORKSPACE before anything is launched.
 * The first call made in a CUDA context (the device's primary context, or a
 * context the caller made current) looks up the array's device address in
 * that context; make that first call before any stream capture.  The lookup
 * is cached per context id, so a context created later (after
 * cudaDeviceReset, for example) gets a fresh lookup on its first call.
 * A device that has loaded the array keeps it until the process exits.
 * Shape errors return the same codes as fm_attn_bwd.
 * Every call uses the same array: calls whose work overlaps on the GPU (for
 * example on two streams) race and give wrong results; calls ordered on one
 * stream are safe.  Each call clears what it needs; nothing carries over.
 */
#define FM_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)
FM_API fm_status fm_attn_bwd_noalloc(const void *q, const void *k, const void *v, const void *o,
                                     int o_dtype, const float *lse, const void *dO, fm_bounds m,
                                     const void *plan, int B, int H, int N, int d, float scale,
                                     void *dq, void *dk, void *dv, int grad_dtype, int flags,
                                     int32_t *dev_status, fm_stream_t stream);

/*
 * Row windows — the same three calls for the Q rows [q_row0, q_row0 + Nq) of
 * the N x N mask against all N key columns: one rank's share of a sequence
 * split over several GPUs (blog §4.3, sequence-parallel integration: the
 * column intervals all-gathered, each rank computing the rows it holds;
 * key/value shards a window's rows never attend are skipped whole by the
 * tile labels).  q_row0 must be a multiple of 128 (of bq for
 * fm_tile_classify_rows), 1 <= Nq, q_row0 + Nq <= N; else FM_ERR_INVALID_ARG.
 * The bounds keep the whole mask ([B, Hm, N], global row numbers).
 *   Q, dO, O: [B, H, Nq, d]; lse: [B, H, Nq]; K, V: [B, H, N, d].
 *   fm_attn_bwd_rows: dQ [B, H, Nq, d] is complete; dK, dV [B, H, N, d]
 *   receive this window's contribution only (zero where it attends nothing):
 *   the contributions of all windows add up to the full gradients.  The
 *   workspace is fm_bwd_workspace_bytes(B, H, Nq, d).
 * The plan of a window is fm_plan_bytes_rows(...) bytes and is built by
 * fm_tile_classify_rows with the same window.  Whole mask: q_row0 = 0, Nq = N
 * (what fm_plan_bytes, fm_tile_classify, fm_attn_fwd and fm_attn_bwd do).
 */
FM_API size_t fm_plan_bytes_rows(int B, int Hm, int N, int q_row0, int Nq, int bq, int bk);
FM_API fm_status fm_tile_classify_rows(fm_bounds m, int q_row0, int Nq, int bq, int bk, void *plan,
                                size_t plan_bytes, uint8_t *labels, int32_t *dev_status,
                                fm_stream_t stream);
FM_API fm_status fm_attn_fwd_rows(const void *q, const void *k, const void *v, fm_bounds m,
                           const void *plan, int B, int H, int N, int q_row0, int Nq, int d,
                           float scale, void *o, int o_dtype, float *lse, void *ws, size_t ws_bytes,
                           int flags, int32_t *dev_status, fm_stream_t stream);
FM_API fm_status fm_attn_bwd_rows(const void *q, const void *k, const void *v, const void *o,
                           int o_dtype, const float *lse, const void *dO, fm_bounds m,
                           const void *plan, int B, int H, int N, int q_row0, int Nq, int d,
                           float scale, void *dq, void *dk, void *dv, int grad_dtype, int flags,
                           void *ws, size_t ws_bytes, int32_t *dev_status, fm_stream_t stream);

/*
 * FP8 forward — DEVICE, async.  Passage: blog "FlashMask技术" §4.2 (the
 * H100 path computes in FP8); per-tensor scaling is the plainest reading.
 * fm_quantize_fp8: e4m3 codes of a bf16 [B, H, N, d] tensor with one scale,
 *   descale = amax / 448 (1 if amax = 0), code = e4m3(x / descale) (fp32
 *   division, round to nearest even, saturating at +-448; inputs finite).
 *   transpose = 0: x8 is [B, H, N, d]; 1: x8 is [B, H, d, N] (N a multiple
 *   of 16, else FM_ERR_UNSUPPORTED) — the layout fm_attn_fwd_fp8 wants for V.
 *   descale: device float, written.  d = 64 or 128.
 * fm_attn_fwd_fp8: fm_attn_fwd (whole mask, standard mode, d = 128) on e4m3
 *   q8, k8 [B, H, N, d] and vt8 [B, H, d, N] with descale = device float[3]
 *   (Q, K, V): S = scale * dq * dk * Q8 K8^T, P rounded to e4m3 for the P V
 *   product (P <= 256 under the lazy rescale), O = dv * (P V) / sum P.  N a
 *   multiple of 16; d != 128 -> FM_ERR_UNSUPPORTED.  Same plan, bounds and
 *   outputs as fm_attn_fwd.
 */
FM_API fm_status fm_quantize_fp8(const void *x, int B, int H, int N, int d, int transpose, uint8_t *x8,
                          float *descale, fm_stream_t stream);
FM_API fm_status fm_attn_fwd_fp8(const uint8_t *q8, const uint8_t *k8, const uint8_t *vt8,
                          const float *descale, fm_bounds m, const void *plan, int B, int H, int N,
                          int d, float scale, void *o, int o_dtype, float *lse, int32_t *dev_status,
                          fm_stream_t stream);

/*
 * Attention over a paged cache — DEVICE, async (fm_paged_plan_bytes: HOST).
 * The serving form of the forward: requests of ragged lengths whose keys and
 * values lie in fixed-size pages of one pool, each request with a row of page
 * numbers (its block table), and per step a chunk of new tokens per request,
 * from a single one (decoding) to thousands (a prompt).
 *
 * A step has `requests` requests; request r has ctx_lens[r] tokens in the cache
 * and q_lens[r] new ones (0 or more).  The new tokens' rows (of q, of k and v to
 * append, of o and lse) stand one behind the other in the order of the requests: rows
 * [cu_q[r], cu_q[r + 1]).  New token i of request r has position ctx_lens[r] + i
 * and attends, of its request's ctx_lens[r] + q_lens[r] keys (the new ones
 * included, which therefore are appended first), key j if
 *     j <= position  and  (window = 0  or  j > position - window  or  j < sink):
 * causal, or a causal window with the first `sink` keys kept (blog §5,
 * window_size and sink_tokens).  Query head h reads KV head h / (Hq / Hkv).
 *
 * fm_paged_plan: the step's bookkeeping, from lengths on the device.
 *   Pages: a request needs ceil(len / page_size) of them.  With free_pages (int32
 *   [n_free], device) the pages that the new tokens need are taken from it, from
 *   index *free_head on, in the order of the requests and of their positions, and
 *   entered into block_table (int32 [requests, max_pages]); *free_next becomes
 *   the index behind the last one taken.  Without (NULL; n_free, free_head and
 *   free_next unused) block_table has to hold every page already.  Entries of pages
 *   already held are read, all others are left as they were.
 *   Writes seq_lens[r] = ctx_lens[r] + q_lens[r]; cu_q (int32 [requests + 1]); per
 *   row t < cu_q[requests] slots[t] = page * page_size + offset (int64
 *   [max_tokens]) and positions[t] (int32 [max_tokens], may be NULL), -1 in both
 *   behind; and the plan that fm_attn_paged walks.
 *   seq_lens may be ctx_lens and free_next may be free_head: they are advanced in
 *   place (a captured step can be replayed); no other two arrays may overlap.
 *   Lengths that do not fit the step's sizes (negative, a chunk over max_q, more than
 *   max_tokens rows, more than max_pages pages, or 2^31 tiles of 128 keys and more over
 *   the KV heads of the requests of at most 32 rows) give FM_ERR_LENGTHS, too few free
 *   pages FM_ERR_PAGES, in dev_status; the plan is then empty: no page is taken,
 *   cu_q is 0, every slot -1, seq_lens = ctx_lens, and fm_attn_paged does
 *   nothing.  A page number outside [0, num_pages) gives FM_ERR_PAGES and slot -1 for
 *   its rows alone.
 * fm_paged_append: writes row t of k and v (bf16, [T, Hkv, d], strides of tokens and
 *   heads in elements) to the cache's slot slots[t]; slots below 0 are skipped,
 *   slots at or behind num_pages * page_size are skipped with FM_ERR_PAGES.  e4m3
 *   caches get e4m3(x / descale) as fm_quantize_fp8 rounds.  Two rows with the same
 *   slot: which one's values are left there, or parts of both, is not defined.
 * fm_attn_paged: q bf16 [rows, Hq, d] (strides of tokens and heads in elements, the
 *   last dimension contiguous), o [rows, Hq, d] and lse fp32 [rows, Hq] contiguous,
 *   with rows at least cu_q[requests] (else FM_ERR_LENGTHS in dev_status and nothing
 *   is written); rows at or behind cu_q[requests] are left as they were, so that what a
 *   fresh allocation held there (NaN too) is still there, as in all rows after a plan that
 *   failed.  `step` has to be the plan's (else FM_ERR_PLAN_MISMATCH in dev_status),
 *   block_table the one it was built from.  Pages that no row of their request
 *   attends are not read, so their table entries may be stale (behind a window),
 *   and what a page holds behind the request's last token may be NaN.  The
 *   request's own tokens are expected to be finite: a value that is not may reach
 *   rows of the same request whose mask excludes it.  A page number outside
 *   [0, num_pages) among the attended gives FM_ERR_PAGES and its keys read as zeros.
 *   Scores, maxima, sums and products are fp32 (fp32 accumulation).  P enters the
 *   second product with 24 bits (o fp32, at most 32 rows of new tokens times Hq / Hkv per
 *   request), 16 bits (otherwise where o is fp32 or the rows are as few) or 8 bits
 *   (bf16 o, more rows); over an e4m3 cache with 22 (o fp32, or at most 8 rows) or 11 bits, but in
 *   steps of 2^-31 of the row's largest weight at the finest (a weight is off by at most
 *   2^-32 of the largest), and Q, where the rows are more, as two e4m3 terms (exact for
 *   elements of 2^-9 of the row's largest or more, off by at most 2^-17 of it for smaller
 *   ones).  o is rounded once.
 *   The plan holds the workspace as well, whatever the number of requests: 5 MB (d = 128),
 *   and 40 MB more where a request may have more than 32 rows (half of both for d = 64).
 *   Calls that share a plan (any number of layers per step) have to follow one another on
 *   the GPU, and so have replays of graphs that share one.  After a status other than 0,
 *   plan again.
 *
 * Sizes: d = 64 or 128; page_size a multiple of 16, 65536 at most; Hq / Hkv whole and at
 * most 32, Hq at most 4096; at most 8192 requests and 2^24 rows; max_pages * page_size
 * below 2^31 - 2^17; without a window a sink changes nothing.  Caches: token (p, h, t) of k
 * begins at element p * k_page + h * k_head + t * k_tok, its d elements contiguous; strides and
 * pointers are multiples of 16 bytes.  Values are code * descale for e4m3 (device float each,
 * positive; ignored for bf16).
 */
typedef struct {
    int32_t requests, max_tokens, max_q, max_pages;
    int32_t num_pages, page_size;
    int32_t Hq, Hkv, d;
    int32_t window, sink;           /* 0: none */
} fm_paged_step;
typedef struct {
    void *k, *v;
    int64_t k_page, k_head, k_tok, v_page, v_head, v_tok;   /* strides, elements */
    const float *k_descale, *v_descale;
    int32_t num_pages, page_size, Hkv, d;
    int32_t dtype;                  /* FM_DT_BF16 or FM_DT_E4M3 */
} fm_paged_cache;
FM_API size_t fm_paged_plan_bytes(const fm_paged_step *step);
FM_API fm_status fm_paged_plan(const fm_paged_step *step, const int32_t *ctx_lens, const int32_t *q_lens,
                               int32_t *block_table, const int32_t *free_pages, int n_free,
                               const int32_t *free_head, int32_t *free_next, int32_t *seq_lens,
                               int32_t *cu_q, int64_t *slots, int32_t *positions, void *plan,
                               size_t plan_bytes, int32_t *dev_status, fm_stream_t stream);
FM_API fm_status fm_paged_append(const void *k, int64_t k_tok, int64_t k_head, const void *v,
                                 int64_t v_tok, int64_t v_head, const int64_t *slots, int T,
                                 const fm_paged_cache *cache, int32_t *dev_status, fm_stream_t stream);
FM_API fm_status fm_attn_paged(const fm_paged_step *step, const void *q, int64_t q_tok, int64_t q_head,
                               int rows, const fm_paged_cache *cache, const int32_t *block_table,
                               void *plan, size_t plan_bytes, float scale, void *o, int o_dtype,
                               float *lse, int32_t *dev_status, fm_stream_t stream);

/*
 * Rotary positions — DEVICE, async (fm_rotary_table: HOST).
 * Element pairs (a, b) of a head turn by an angle that grows with the row's position p:
 *     a' = m (a cos p theta_i - b sin p theta_i),   b' = m (b cos p theta_i + a sin p theta_i),
 * so that the product of a query and a key depends on their distance.  The first `rot`
 * elements of the head are turned, the others are copied; pair i is (x_i, x_(i + rot/2)), or
 * (x_2i, x_(2i+1)) if `interleaved`.
 *
 * fm_rotary_table: the frequencies, as 64-bit fractions of a turn per position (so that an
 *   angle is off by less than 2^-30 turns at any position below 2^24; int32 positions
 *   all work), into host turns[rot / 2], and m.  theta_i = base^(-2 i / rot), and for contexts `factor` s >= 1 times
 *   as long as those that the model was trained on:
 *     FM_ROPE_LINEAR: theta_i / s;
 *     FM_ROPE_NTK:    base s^(rot / (rot - 2)) in place of base (rot > 2);
 *     FM_ROPE_YARN:   theta_i (g + (1 - g) / s), g = clamp((original theta_i / 2 pi - slow) /
 *                     (fast - slow), 0, 1): pairs that turn more than `fast` times within the
 *                     `original` positions are left, those that turn less than `slow` times are
 *                     stretched; m = 0.1 ln s + 1.  (The ramp g is linear in the turns, as in the method's formula.  Programs
 *                     whose ramp is linear in the pair's index, between those that turn `fast` and `slow` times, have other
 *                     frequencies in between, by up to a factor of 2.3 at s = 8: their models need a table of their own.)
 *   m = 1 otherwise.  rot even, 2 to 128; base > 1; 0 <= slow < fast and original > 0 for YARN; all finite (else
 *   FM_ERR_INVALID_ARG).
 * fm_rope: y = the turned x.  x of x_dtype, y of y_dtype (bf16 or fp32): element (b, h, n, c) at b * batch +
 *   h * head + n * tok + c (strides in elements, multiples of 16 bytes); positions int32, of row (b, n) at b *
 *   pos_batch + n.  inverse != 0 turns back, with the same m: the gradient with respect
 *   to x from the one with respect to y (the transposed map).  Rows whose position is
 *   negative are left as they were in y.  y may be x (same strides and type), and may not
 *   overlap it otherwise.  Sine and cosine are fp32, from an angle reduced in 64-bit
 *   integers; products are fp32; y is rounded once.
 * rotary: `turns` (device, 16-byte aligned) holds fm_rotary_table's values, or others: theta_i / 2 pi modulo 1,
 *   times 2^64; rot a multiple of 8, at most d (else FM_ERR_UNSUPPORTED); d = 64 or 128.
 */
enum { FM_ROPE_PLAIN = 0, FM_ROPE_LINEAR = 1, FM_ROPE_NTK = 2, FM_ROPE_YARN = 3 };
typedef struct {
    int32_t rot, scaling;
    double base, factor, original, slow, fast;
} fm_rotary_spec;
typedef struct {
    const uint64_t *turns;          /* device [rot / 2] */
    int32_t rot, interleaved;
    float magnitude;                /* m */
} fm_rotary;
typedef struct {
    int64_t batch, head, tok;       /* strides, elements */
} fm_strides;
FM_API fm_status fm_rotary_table(const fm_rotary_spec *spec, uint64_t *turns, float *magnitude);
FM_API fm_status fm_rope(const void *x, int x_dtype, fm_strides xs, const int32_t *positions, int64_t pos_batch,
                         int B, int H, int N, int d, const fm_rotary *rotary, int inverse, void *y, int y_dtype,
                         fm_strides ys, fm_stream_t stream);

/*
 * Long conversations over a paged cache — DEVICE, async: what a program does around
 * fm_attn_paged once per layer (fm_paged_append_rope, fm_paged_weights, fm_paged_evict) or once
 * per step (fm_verify_drafts, fm_paged_release).
 *
 * fm_paged_append_rope: fm_rope of a step's rows and fm_paged_append in one: q_out row t =
 *   q row t turned by positions[t] (bf16 [T, Hq, d], strides of tokens and heads as q's own; q_out may be q);
 *   k row t turned and v row t as it is go to the cache's slot slots[t].  K is rounded once, from the turned fp32
 *   value (bf16, or e4m3 of value / descale).  Where positions[t] is negative nothing of row t
 *   is written; a slot is treated as fm_paged_append treats it, and does not
 *   concern q.  Positions are the caller's: after an eviction they run ahead of the
 *   plan's, which count cached tokens.
 * fm_paged_weights: the attention weight that every cached key of a step's requests receives,
 *     weights[page, h, offset] (+)= sum over rows t and query heads g of KV head h that attend the key
 *                                   of exp(scale q[t, g] . k - lse[t, g]),
 *   fp32 [num_pages, Hkv, page_size], contiguous.  Keys that the step brought (position >= ctx_lens[r]) begin
 *   from zero, the others are added to; keys that no row attends (behind a window) are left as they were.  Same step,
 *   plan, q, cache (its k alone is read), block table and scale as fm_attn_paged, after it, with its lse; `rows` as there.
 *   Scores and sums are fp32; beside an e4m3 cache the q of requests of at most 32 rows enters as two
 *   e4m3 terms, as in fm_attn_paged.  A key's sum is added up in a fixed order, except that several
 *   requests that hold one page add to it in any order.  Every row counts, those of drafted tokens that fm_verify_drafts
 *   refuses among them, and what older keys have from them stays.  A row whose lse is +infinity gives nothing where its score is finite: a program that
 *   wants the kept rows alone calls this after the verification, with the lse of the rows behind (out < 0) at +infinity.
 *   A step for which this is not called leaves the weights of its keys as
 *   that memory was (a page given out again holds another request's).  A row gives nothing to keys that it does not attend, whatever its
 *   lse.  A page number outside [0, num_pages) among the attended
 *   gives FM_ERR_PAGES and its keys are left out.
 * fm_paged_evict: cuts requests of more than `budget` cached tokens down to `budget` in one layer: per KV head the first
 *   `sink` tokens stay, the last `recent` ones, and of those between the budget - sink - recent
 *   with the largest weights (equal ones: the earlier; NaN counts as the largest), in their order, at
 *   places 0 .. budget - 1 of the request: keys, values and weights are moved, in place.  Different heads may keep
 *   different tokens.  lens: int32 [requests] cached tokens; new_lens[r] = min(lens[r], budget) (another array than
 *   lens: every layer of the model reads the same lens); kept: int32 [requests, Hkv, budget], the
 *   places kept, -1 for requests that are not cut.  What lies behind the new length is left as it is.
 *   A request whose length is out of range (FM_ERR_LENGTHS) or that holds a page outside [0, num_pages) among those of its
 *   tokens (FM_ERR_PAGES) is not cut, and new_lens[r] = lens[r].
 *   Places, and with them positions of the next plan and windows, count the tokens that are left; rotary positions are the
 *   caller's to keep.  Pages of a request that is cut may be held by no other request, and none twice.  weights as above; their page and
 *   head sizes are the cache's.  1 <= budget, 0 <= sink, 0 <= recent, sink + recent <= budget.
 * fm_paged_release: gives the pages behind the requests' new lengths back to the free list that fm_paged_plan
 *   takes from: pages ceil(lens[r] / page_size) .. ceil(held[r] / page_size) - 1 of every request, in the order of
 *   the requests and of their places, to free_pages[*free_head - n .. *free_head - 1], and *free_next = *free_head - n;
 *   seq_lens[r] = lens[r].  0 <= lens[r] <= held[r]; lens[r] = 0 ends a request.  The table keeps the
 *   entries (nothing reads behind a length).  seq_lens may be held or lens, and free_next may be
 *   free_head.  Without a free list (free_pages NULL; free_head, free_next unused) only seq_lens is written.
 *   Lengths out of range give FM_ERR_LENGTHS; a page outside [0, num_pages), or more pages than
 *   were taken from the list (n > *free_head, or *free_head outside [0, n_free]), FM_ERR_PAGES: then nothing is given back and
 *   seq_lens[r] = held[r], *free_next = *free_head.
 *   Pages that several requests hold (a common prefix) would be given back several times: only
 *   the last holder's call may include them.
 * fm_verify_drafts: which of the drafted tokens of a step are kept, and the token behind them, so that
 *   they are distributed as the target's own.  Rows of request r: [cu_q[r], cu_q[r + 1]) (the plan's cu_q); row i fed
 *   tokens[i], whose first is the last known token and the others the drafted ones; target row
 *   i: p = the target's probabilities of the token behind it; draft row i: q = those that token i + 1 was drawn
 *   from, or draft NULL: it was taken with certainty (q is 1 there).  Draft t = tokens[i + 1] is kept if
 *   u_accept[i] q(t) < p(t), up to the first that is not, at row a of the request (or its last row, all
 *   kept); then the token is drawn that u_sample[r] in [0, 1) points at, the smallest x with
 *       sum_(y <= x) w(y) > u_sample[r] sum w,   w = max(p - q, 0) of row a where a draft was refused and
 *                                                that is not all zero, else w = max(p, 0).
 *   Sums are held in about 48 bits.  out[row]: the kept drafts, the drawn token, -1 behind (int32 [rows]; rows of
 *   no request are left as they were); n_out[r]: kept drafts + 1 (0 for a request without rows);
 *   new_lens[r] = seq_lens[r] - rows of the request + n_out[r] (may be seq_lens): the tokens whose keys stay in the cache.
 *   target, draft: [rows, V] of dtype (bf16 or fp32), row strides in elements, any alignment of a whole
 *   element.  1 <= V <= 2^24.  A drafted token outside [0, V) is refused, with FM_ERR_PROBS; so is the draw where the
 *   sum of w is zero, infinite or NaN: the token is then -1.  cu_q outside [0, rows] or
 *   decreasing: FM_ERR_LENGTHS, and the request has no rows.  rows = 0 (target, draft, tokens, u_accept and out unused) is a
 *   step without any.  No other two arrays may overlap.
 */
FM_API fm_status fm_paged_append_rope(const void *q, int64_t q_tok, int64_t q_head, int Hq, const void *k, int64_t k_tok,
                                      int64_t k_head, const void *v, int64_t v_tok, int64_t v_head, const int64_t *slots,
                                      const int32_t *positions, int T, const fm_rotary *rotary,
                                      const fm_paged_cache *cache, void *q_out, int64_t qo_tok, int64_t qo_head,
                                      int32_t *dev_status, fm_stream_t stream);
FM_API fm_status fm_paged_weights(const fm_paged_step *step, const void *q, int64_t q_tok, int64_t q_head, int rows,
                                  const fm_paged_cache *cache, const int32_t *block_table, void *plan, size_t plan_bytes,
                                  float scale, const float *lse, float *weights, int32_t *dev_status,
                                  fm_stream_t stream);
FM_API fm_status fm_paged_evict(const fm_paged_cache *cache, int requests, int max_pages, const int32_t *lens,
                                const int32_t *block_table, float *weights, int budget, int recent, int sink,
                                int32_t *kept, int32_t *new_lens, int32_t *dev_status, fm_stream_t stream);
FM_API fm_status fm_paged_release(int requests, int max_pages, int num_pages, int page_size, const int32_t *held,
                                  const int32_t *lens, const int32_t *block_table, int32_t *free_pages, int n_free,
                                  const int32_t *free_head, int32_t *free_next, int32_t *seq_lens,
                                  int32_t *dev_status, fm_stream_t stream);
FM_API fm_status fm_verify_drafts(const void *target, int64_t target_row, const void *draft, int64_t draft_row, int dtype,
                                  int V, int rows, const int32_t *tokens, const float *u_accept, const float *u_sample,
                                  const int32_t *cu_q, const int32_t *seq_lens, int requests, int32_t *out,
                                  int32_t *n_out, int32_t *new_lens, int32_t *dev_status, fm_stream_t stream);

/*
 * Step graphs — create / destroy HOST, synchronous; launch DEVICE, async.
 * One step of the path (fm_tile_classify, fm_attn_fwd and, when dO is given,
 * fm_attn_bwd; 128 x 128 tiles) captured once into a CUDA graph for a fixed
 * set of buffers and replayed with a single launch.  Passages: blog §6.2
 * item 1 (capture the compute pattern in a CUDA Graph) and FlashAttention
 * article §三.3 (CUDA Graphs to cut kernel-launch overhead, which dominates
 * small problems).  Every launch reads the current contents of
 * the buffers in fm_step_args: refill q, k, v, dO and the bounds in place
 * between launches.  The caller keeps every buffer allocated and unmoved until
 * fm_step_graph_destroy, zeroes dev_status before reading it, and does not run
 * two launches on the same buffers concurrently.
 * fm_step_graph_create: argument errors are those of the three calls (the
 * capture is discarded, nothing is allocated); args or graph NULL ->
 * FM_ERR_INVALID_ARG; a failed capture -> FM_ERR_CUDA.  *graph is written on
 * success only (else set to NULL).
 */
typedef struct {
    const void *q, *k, *v;          /* bf16 [B, H, N, d] */
    const void *dO;                 /* bf16 [B, H, N, d], or NULL: forward-only graph */
    fm_bounds mask;
    void *plan;                     /* fm_plan_bytes(B, Hm, N, 128, 128) bytes */
    size_t plan_bytes;
    void *o;                        /* [B, H, N, d] of o_dtype */
    int o_dtype;
    float *lse;                     /* [B, H, N] */
    void *dq, *dk, *dv;             /* [B, H, N, d] of grad_dtype; unused without dO */
    int grad_dtype;
    void *ws;                       /* fm_bwd_workspace_bytes(B, H, N, d); unused without dO */
    size_t ws_bytes;
    int B, H, N, d;
    float scale;
    int flags;                      /* FM_FLAG_PRECISE or 0 */
    int32_t *dev_status;
} fm_step_args;
typedef struct fm_step_graph_st *fm_step_graph;
FM_API fm_status fm_step_graph_create(const fm_step_args *args, fm_step_graph *graph);
FM_API fm_status fm_step_graph_launch(fm_step_graph graph, fm_stream_t stream);
FM_API fm_status fm_step_graph_destroy(fm_step_graph graph);

/*
 * Per-kernel timing (the library's own tracing).  fm_profile_begin starts
 * recording a CUDA event pair around every kernel the library launches
 * (process-wide, up to 4096 launches); fm_profile_end waits for those
 * events, writes up to max_entries (kernel id, milliseconds) records and
 * stops recording.  Returns the number of records written, or -1 on error.
 */
enum { FM_K_CLASSIFY_MINMAX = 0, FM_K_CLASSIFY_LISTS = 1, FM_K_FWD = 2, FM_K_BWD_PRE = 3,
       FM_K_BWD = 4, FM_K_BWD_POST = 5, FM_K_CLASSIFY_ORDER = 6, FM_K_FP8_AMAX = 7,
       FM_K_FP8_CONVERT = 8, FM_K_PAGED_PLAN = 9, FM_K_PAGED_APPEND = 10, FM_K_PAGED_DECODE = 11,
       FM_K_PAGED_CHUNK = 12, FM_K_ROPE = 13, FM_K_PAGED_APPEND_ROPE = 14, FM_K_PAGED_WEIGH_FEW = 15,
       FM_K_PAGED_WEIGH_MANY = 16, FM_K_PAGED_EVICT = 17, FM_K_PAGED_RELEASE = 18, FM_K_VERIFY = 19, FM_K_COUNT = 20 };
typedef struct {
    int32_t kernel;
    float ms;
} fm_kernel_time;
FM_API fm_status fm_profile_begin(void);
FM_API int fm_profile_end(fm_kernel_time *out, int max_entries);

/*
 * fm_debug_wait_test — HOST, test hook; nothing calls it in a product path.
 * Failure detection is tested on the real kernels without faulting the GPU:
 * after this call, the next fm_attn_fwd / fm_attn_fwd_rows launch
 * (kernel = 0), fm_attn_bwd / fm_attn_bwd_rows launch (kernel = 1) or launch of
 * the few-rows or many-rows kernel of fm_attn_paged (FM_K_PAGED_DECODE,
 * FM_K_PAGED_CHUNK) or fm_paged_weights (FM_K_PAGED_WEIGH_FEW, _MANY) made by the process bounds every device-side wait by
 * limit_cycles SM cycles (100,000 .. the default bound of about 3e9) instead of
 * the default, and its first CTA withholds the load of its second K tile (forward),
 * of its second Q/dO half (backward) or of its second tile (few rows; many rows:
 * every CTA expects a byte more of its K tiles than comes, and the bound is that of
 * the waits for K).  The wait for that load runs out: the kernel writes
 * FM_ERR_TIMEOUT to dev_status, raises its abort flag (every other wait of the
 * CTA then gives up), drains the copies and tensor-core products
 * it issued, frees its TMEM and returns; the CUDA context stays usable.
 * The switch is consumed by that one launch; kernel = -1 clears it.
 * Returns FM_ERR_INVALID_ARG for another kernel id or a limit out of range.
 */
FM_API fm_status fm_debug_wait_test(int kernel, long long limit_cycles);

/*
 * Self-test of the bounded wait used by every pipeline barrier: one CTA
 * waits on a barrier that nothing completes, gives up after about
 * limit_cycles SM clock cycles and writes FM_ERR_TIMEOUT to dev_status.
 * Lets failure detection be tested without hanging a GPU.
 */
FM_API fm_status fm_selftest_wait_timeout(long long limit_cycles, int32_t *dev_status,
                                   fm_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* FM_H_ */
