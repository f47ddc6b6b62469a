/*
 * idx.h - C ABI of libidx, the GB300 (sm_103a) sparse-attention prefill indexer.
 *
 * Problem (page "[sglang] logits를 쓰지 않는 top-k: SGLang의 LiteTopK prefill
 * indexer", introduction and section 1): for every query row r and every key j
 * that the row can see, ks[r] <= j < ke[r], the indexer score is
 *
 *     s[r,j] = k_scale[j] * sum_h w[r,h] * max(0, q[r,h,:] . k[j,:])
 *
 * and the row keeps the topk best keys.  This library returns the EXACT top-k:
 * keys ordered by (score descending, key index ascending), the first topk kept,
 * reported as row-relative indices j - ks[r] (page 1, section 1: candidate
 * indices are stored as key - ks[row]) in ascending order, followed by -1 when
 * the row sees fewer than topk keys (page 1, section 3: a consumer skips
 * negative positions).
 *
 * Conventions shared by every entry point
 *  - Tensor arguments are DEVICE pointers owned by the caller; the library
 *    keeps no pointer after the call returns and allocates no device memory.
 *    Scratch memory is the caller's workspace `ws` of at least the size its
 *    *_workspace query returns, 256-byte aligned.
 *  - All layouts are row-major and contiguous:
 *      q [rows, H, D], k [keys, D]  (both bf16 or both fp8 e4m3, see idx_dtype)
 *      k_scale [keys] float32 (> 0), w [rows, H] float32 (>= 0)
 *      ks, ke [rows] int32;  out_idx [rows, topk] int32
 *  - `stream` is a cudaStream_t (NULL is the legacy default stream).  Calls are
 *    asynchronous on that stream; the host never waits on the device.
 *  - Arguments are validated on the host before anything is launched; a bad
 *    argument returns an error and launches nothing.  Errors met on the
 *    device (a visible range outside [0, keys], a wait that timed out) are
 *    OR-ed into the optional device status word options->d_status as
 *    IDX_DEV_* bits; nothing traps.
 *  - Preconditions not checked: scores, q, k, k_scale, w hold no NaN/Inf;
 *    k_scale > 0 and w >= 0 (the score formula relies on it).
 *  - Supported: sm_103a; H in {8, 16, 32, 64}; D in {64, 128};
 *    1 <= topk <= 4096; rows >= 0 (a row count of 0 is a no-op).
 *    Anything else returns IDX_EUNSUPPORTED.
 */
#ifndef IDX_H_
#define IDX_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    IDX_OK = 0,
    IDX_EINVAL = 1,        /* a null pointer, a negative size, topk < 1 ... */
    IDX_EALIGN = 2,        /* a tensor or the workspace is not 16 B (256 B for ws) aligned */
    IDX_EWORKSPACE = 3,    /* ws_bytes smaller than the query returned */
    IDX_EUNSUPPORTED = 4,  /* dtype, H, D, topk or the GPU architecture */
    IDX_ECUDA = 5,         /* a CUDA runtime/driver call failed */
    IDX_ETIMEOUT = 6       /* reserved for host-side reporting of IDX_DEV_TIMEOUT */
} idx_status;

/* bits OR-ed into *options->d_status by device code */
#define IDX_DEV_TIMEOUT 0x1   /* a bounded wait inside a kernel gave up */
#define IDX_DEV_RANGE   0x2   /* a row's [ks, ke) is not inside [0, keys] or exceeds max_len */
#define IDX_DEV_STATE   0x4   /* the exact fallback ran out of its refinement levels */
#define IDX_DEV_PAGES   0x8   /* idx_cache_resize: the free pages did not suffice for every row */

/* IDX_MXFP4 (the OCP MX format): e2m1 elements packed two per byte (element 2i in
 * the low nibble) with one e8m0 scale per 32 consecutive elements along D; only
 * the *_mxfp4 entry points below take it (they also take the scale arrays). */
typedef enum {
    IDX_BF16 = 1,
    IDX_FP8_E4M3 = 2,
    IDX_MXFP4 = 3,
    IDX_FP16 = 4,  /* the serving entry points below only */
    IDX_FP32 = 5   /* idx_add_rmsnorm_quant only */
} idx_dtype;

/* Optional device-side counters (zero them before the call if you read them). */
typedef struct idx_stats {
    int emit_all_rows;   /* rows that see <= cap keys: every key became a candidate */
    int overflow_rows;   /* rows whose candidate count exceeded the slab cap */
    int short_rows;      /* rows with fewer than topk candidates although they see > cap keys */
    int fallback_rows;   /* rows re-selected by the exact full-row rescan */
    int max_count;       /* largest candidate count of any row */
    int split_rows;      /* rows the standalone top-k selected with a multi-block row split */
    int tie_rescan_rows; /* standalone top-k rows that needed the multi-pass path (the
                            one-pass candidate runs missed or overflowed) */
    int reserved;
} idx_stats;

/* Every field 0 selects the default.  Pass NULL for all defaults. */
typedef struct idx_options {
    float cap_factor;     /* candidate slab cap = ceil(cap_factor * topk) when given;
                             default min(max(ceil(3.5 * topk), 4096), 12288) (page 1
                             sizes its slab at about 2.25 x topk; the larger default
                             lets the threshold sample take a wider stride, so the
                             sample pass costs less than the extra candidates add).
                             Caps above 12288 are refused. */
    float target_factor;  /* expected candidates / topk that the sampled threshold aims
                             at; default sqrt(cap/topk).  Test knob to force short or
                             overflowing rows. */
    int sample_stride;    /* odd stride S of the threshold sample; 0 = automatic */
    int row_split;        /* standalone top-k row split, see below;
                             idx_window_attention_mxfp4: 0 the cheaper path, -1 tiles of few
                             rows, 1 the tensor cores' dense path;
                             idx_cache_resize, idx_cache_compact: -1 ranks pages with one
                             CTA, as where a device does not place a cluster of 16 */
    int* d_status;        /* optional device int receiving IDX_DEV_* bits */
    idx_stats* d_stats;   /* optional device counters */
    int relative_rows;    /* idx_topk_from_scores: row r's visible scores start at
                             column 0 of its row (the layout idx_score_materialise
                             writes) instead of column ks[r] */
    int test_stall_us;    /* test only, 0 = off.  n > 0: the TMA producer of every
                             scoring pass issues no copy for key tile 1, and the
                             scoring kernel's waits give up after about n
                             microseconds (instead of about 2 s).  A pass with more
                             than one tile then stops early with IDX_DEV_TIMEOUT in
                             *d_status, leaving no copy or MMA in flight; the call
                             returns and its results are meaningless.  The parts of
                             idx_prefix_attention on the tensor cores' dense path (the
                             prefix's, and private ones that take it) and the dense path of
                             idx_window_attention_mxfp4 do the same with their key tile 1.  It exists to run the timeout unwind on
                             purpose. */
    void* const* stage_events; /* optional array of cudaEvent_t, recorded on `stream`
                             at stage boundaries (NULL entries are skipped).
                             idx_score_topk: [0] start, [1] after the sample and its
                             thresholds, [2] after the scoring/emit pass, [3] after
                             the slab top-k, [4] after the exact rescan (end).
                             The other entry points: [0] start, [1] end. */
} idx_options;

/* row_split: 0 = automatic (page "[sglang] ROCm DSA Indexer Top-K 최적화",
 * row_split function: split a row over g blocks when it is at least 65536 long
 * and g = min(SMs / rows, 32) >= 4), -1 or 1 = never split, g >= 2 = force
 * g blocks (at most 64).  Grids with more than 65535 rows never split.  A
 * split row is streamed once by g blocks, each over a contiguous slice; one
 * more block per row selects from what they kept, or re-selects the whole row
 * exactly when a slice kept more than it can hand over. */

/* ------------------------------------------------------------------------
 * idx_score_topk - fused score + exact top-k, without writing [rows, keys]
 * logits (page 1, "Sampled Threshold" and section 1).
 *
 * Per row: a threshold T_r is taken from an odd-stride single-key sample of
 * the row's own scores (page 1, section 2); one scoring pass emits only
 * (score, key) pairs with score >= T_r into a per-row candidate slab of `cap`
 * entries together with the exact count (page 1, section 1 parameter list);
 * an exact radix top-k then selects from the slab.  Rows whose count ended
 * below topk or above cap are re-selected exactly by a full-row rescan, so the
 * result never depends on the sample (the page's own kernel stays lossy here;
 * this library does not).
 *
 *   q, k, k_scale, w, ks, ke : inputs as in the conventions above
 *   rows, keys, H, D, topk   : sizes; keys < 2^31 - 256 and rows * H < 2^31 - 256
 *   max_len                  : an upper bound on ke[r] - ks[r] (0 = keys); it
 *                              sizes the workspace
 *   dt                       : element type of q and k
 *   out_idx                  : [rows, topk] int32 result
 *   ws, ws_bytes             : workspace, >= idx_score_topk_workspace(...)
 * Returns IDX_OK or an error from the list above.
 * ------------------------------------------------------------------------ */
size_t idx_score_topk_workspace(int rows, long long keys, long long max_len, int H, int D,
                                int topk, idx_dtype dt, const idx_options* opt);
idx_status idx_score_topk(const void* q, const void* k, const float* k_scale, const float* w,
                          const int* ks, const int* ke, int rows, long long keys,
                          long long max_len, int H, int D, int topk, idx_dtype dt,
                          int* out_idx, void* ws, size_t ws_bytes, const idx_options* opt,
                          void* stream);

/* ------------------------------------------------------------------------
 * idx_score_topk_host - idx_score_topk on inputs and output in HOST memory:
 * the call a host that holds q, k, ... (and wants the indices back) makes.
 * Page-locked host memory lets the copies run asynchronously and overlap the
 * compute; pageable memory gives the same result without the overlap.
 *
 * The rows are taken in two chunks (whole row blocks each).  k and
 * k_scale go up first, then each chunk's q, w, ks and ke on a copy stream;
 * chunk c is scored and selected on `stream` once its inputs are up, while
 * chunk c + 1 goes up and chunk c - 1's indices come back on a second copy
 * stream.  The call returns with everything enqueued and `stream` waiting
 * for the last copy back: once `stream` is synchronised, out_idx is
 * complete.  The copy streams and their events are the library's, one pair
 * per device; calls on one device are serialised on the host.
 *
 *   q, k, k_scale, w, ks, ke, out_idx : HOST pointers, shapes as for
 *                              idx_score_topk (no alignment needed)
 *   ws, ws_bytes             : DEVICE workspace (256-byte aligned), at least
 *                              idx_score_topk_host_workspace(...): the device
 *                              copies of the inputs and of out_idx, and the
 *                              fused workspace of one chunk
 *   opt                      : as for idx_score_topk; stage_events [0] start
 *                              and [1] end on `stream`
 * Returns IDX_OK or an error from the list above (arguments are checked
 * before anything is copied).
 * ------------------------------------------------------------------------ */
size_t idx_score_topk_host_workspace(int rows, long long keys, long long max_len, int H, int D,
                                     int topk, idx_dtype dt, const idx_options* opt);
idx_status idx_score_topk_host(const void* q, const void* k, const float* k_scale,
                               const float* w, const int* ks, const int* ke, int rows,
                               long long keys, long long max_len, int H, int D, int topk,
                               idx_dtype dt, int* out_idx, void* ws, size_t ws_bytes,
                               const idx_options* opt, void* stream);

/* ------------------------------------------------------------------------
 * idx_topk_from_scores - exact top-k of given fp32 scores (page "[sglang] ROCm
 * DSA Indexer Top-K 최적화": fp32 12-bit coarse histogram, radix tie
 * refinement, full-row rescan when the threshold bin overflows the tie
 * buffer, multi-block row split for long rows at low batch).
 *
 *   scores [rows, row_stride] fp32; row r's visible scores are
 *          scores[r*row_stride + j] for ks[r] <= j < ke[r]
 *          (or scores[r*row_stride + j - ks[r]] with options->relative_rows)
 *   ks may be NULL (all rows start at 0).
 *   out_idx [rows, topk]: ascending j - ks[r], then -1.
 * The result is bit-exact: ties at equal fp32 values (+0 == -0) go to the
 * lower index.  NaN scores are a precondition violation.
 * ws: idx_topk_workspace(...) bytes, 256-byte aligned (IDX_EWORKSPACE if
 * smaller, IDX_EALIGN if misaligned); 0 bytes, and ws may be NULL, unless
 * rows are split (row_split above): then 2 * 8192 * 4 + 8 bytes per block of
 * a split row, 8 bytes per row and 256.  The call allocates nothing, and the
 * workspace needs no clearing between calls.
 * ------------------------------------------------------------------------ */
size_t idx_topk_workspace(int rows, long long row_stride, int topk, const idx_options* opt);
idx_status idx_topk_from_scores(const float* scores, long long row_stride, const int* ks,
                                const int* ke, int rows, int topk, int* out_idx, void* ws,
                                size_t ws_bytes, const idx_options* opt, void* stream);

/* ------------------------------------------------------------------------
 * idx_score_materialise - the two-pass baseline's first pass (page 1,
 * introduction: the full [rows, keys] logits written to global memory).
 * Writes s[r,j] for ks[r] <= j < ke[r] to scores[r*row_stride + (j - ks[r])]
 * (row_stride >= the longest visible range); other entries are not touched.
 * Bit-identical to the scores the fused path compares against its threshold.
 * Feed the result to idx_topk_from_scores with options->relative_rows = 1.
 * ------------------------------------------------------------------------ */
idx_status idx_score_materialise(const void* q, const void* k, const float* k_scale,
                                 const float* w, const int* ks, const int* ke, int rows,
                                 long long keys, int H, int D, idx_dtype dt, float* scores,
                                 long long row_stride, const idx_options* opt, void* stream);

/* ------------------------------------------------------------------------
 * idx_score_topk_noalloc - idx_score_topk for callers that cannot allocate.
 * The paper has no counterpart to this entry point.
 *
 * Some callers only hold pointers to memory that someone else owns (a plugin
 * in a host framework that gives its extensions no allocator, or a serving
 * loop that must not call cudaMalloc, which can synchronize the device) and so
 * cannot pass a workspace.  This call takes the same arguments as
 * idx_score_topk without ws/ws_bytes and runs the same kernels on a scratch
 * array compiled into the library; it allocates no memory.
 *
 *  - Limit: the problem's idx_score_topk_workspace(...) must not exceed
 *    IDX_NOALLOC_SCRATCH_BYTES (32 MiB); larger problems return
 *    IDX_EWORKSPACE and launch nothing.  At topk 2048 with 64K-key rows that
 *    is about 480 query rows per call.
 *  - Every GPU that loads the library holds the 32 MiB array until the
 *    process exits.
 *  - The first call on a device looks up the array's device address (with
 *    that device current) and caches it; make that first call before any
 *    stream capture.
 *  - All calls share the one array, and each call leaves its contents behind
 *    (the kernels write every word they later read, so nothing needs
 *    clearing).  Calls whose executions overlap on the GPU, on any stream or
 *    from any thread, race on it: serialize them.
 * ------------------------------------------------------------------------ */
#define IDX_NOALLOC_SCRATCH_BYTES (32ull << 20)
idx_status idx_score_topk_noalloc(const void* q, const void* k, const float* k_scale,
                                  const float* w, const int* ks, const int* ke, int rows,
                                  long long keys, long long max_len, int H, int D, int topk,
                                  idx_dtype dt, int* out_idx, const idx_options* opt,
                                  void* stream);

/* ------------------------------------------------------------------------
 * idx_score_topk_routed - the same result as idx_score_topk, by the faster
 * path for the call's longest row (page "[sglang] logits를 쓰지 않는 top-k",
 * section 4: the fused path is used only when the longest row sees enough
 * keys; below that the filter passes most keys and the dense path is
 * faster).
 *
 * idx_route_fused(rows, max_len, topk) is the gate.  1 (the fused path)
 * when max_len <= max(ceil(2.25 topk), 4096) (every row fits the default
 * candidate slab: all keys are emitted, no sampling); else 0 (the two-pass
 * path: idx_score_materialise into the workspace, then idx_topk_from_scores)
 * for few rows, rows <= SMs / 4 with rows x max_len <= 2^25 (the logits are
 * small and the top-k splits each long row over >= 4 blocks, while the fused
 * path pays its sample, threshold and slab launches: at 8-32 rows x 1M keys,
 * H 32, the two-pass path is 1.36-1.02x faster); else 1 when max_len >= 24576
 * keys and 0 below.  24576 is the crossover measured on GB300 for e4m3
 * q/k with H = 32 and 64 and topk 512 and 2048 (4096 causal rows): the
 * two-pass path is faster from 6144 to 16384 keys, the two are within 1 % at
 * 24576 and 32768 (where the fused path needs no logits workspace), and the
 * fused one is faster at 65536; the page's own rule (8 x topk keys, 16384 at
 * topk 2048) sits below it.  Both
 * paths select exactly the same keys (they compare the same fp32 scores).
 * Arguments as idx_score_topk; max_len 0 = keys.  The workspace of the
 * two-pass route holds the [rows, max_len] fp32 logits.
 * ------------------------------------------------------------------------ */
int idx_route_fused(int rows, long long max_len, int topk);
size_t idx_score_topk_routed_workspace(int rows, long long keys, long long max_len, int H,
                                       int D, int topk, idx_dtype dt, const idx_options* opt);
idx_status idx_score_topk_routed(const void* q, const void* k, const float* k_scale,
                                 const float* w, const int* ks, const int* ke, int rows,
                                 long long keys, long long max_len, int H, int D, int topk,
                                 idx_dtype dt, int* out_idx, void* ws, size_t ws_bytes,
                                 const idx_options* opt, void* stream);

/* ------------------------------------------------------------------------
 * idx_page_table_transform - row-relative top-k positions to physical KV
 * slots of a paged cache (page "[sglang] logits를 쓰지 않는 top-k", section 3:
 * the page-table transform for paged output, page size 64).
 *
 *   idx   [rows, topk] int32, device, rewritten in place: every p >= 0
 *         becomes table[t, p / page_size] * page_size + p % page_size, with
 *         t = row_map[r] (or r when row_map is NULL); negative entries (the
 *         -1 padding) are left as they are.
 *   table [table_rows, table_stride] int32, device: physical page of each
 *         logical page of a table row.
 *   row_map [rows] int32, device, optional: the table row of each query row
 *         (all query rows of one request share its row).
 * A page past table_stride, or a table row outside [0, table_rows), gives -1
 * and raises IDX_DEV_RANGE in options->d_status.  The physical slot must fit
 * in int32 (a precondition, not checked).  Four entries per thread with one
 * 16-byte load and store when topk % 4 == 0 and idx is 16-byte aligned, one
 * otherwise.  No workspace; asynchronous on `stream`.
 * ------------------------------------------------------------------------ */
idx_status idx_page_table_transform(int* idx, int rows, int topk, const int* table,
                                    int table_rows, long long table_stride, const int* row_map,
                                    int page_size, const idx_options* opt, void* stream);

/* ------------------------------------------------------------------------
 * MXFP4 inputs (page "[sglang] logits를 쓰지 않는 top-k", section 1: an fp4
 * indexer whose 128-element keys are 64 bytes).
 *
 * idx_mxfp4_to_e4m3 - n rows of D MXFP4 elements to e4m3, exactly.
 *   x   [n, D/2] bytes, device, 16-byte aligned: two e2m1 elements per byte,
 *       element 2i in the low nibble
 *   sf  [n, D/32] bytes, device: the e8m0 scale (2^(sf - 127)) of each block of
 *       32 consecutive elements
 *   out [n, D] e4m3 bytes, device, 16-byte aligned
 * An e2m1 value (0, ±0.5 ... ±6) times 2^e is an e4m3 value when e lies in
 * [-8, 6] (the OCP recipe e = floor(log2 max|x|) - 2 gives that range for
 * |x| in [2^-6, 2^8)); such elements are converted exactly.  Others (and the
 * NaN scale 255) are saturated to ±448 or flushed to zero and raise
 * IDX_DEV_RANGE.  D % 32 == 0 (IDX_EINVAL); misaligned x or out: IDX_EALIGN.
 *
 * idx_score_topk_mxfp4 / idx_score_materialise_mxfp4 - idx_score_topk and
 * idx_score_materialise on MXFP4 q [rows, H, D/2] + q_sf [rows, H, D/32] and
 * k [keys, D/2] + k_sf [keys, D/32]: q and k are expanded to e4m3 into the
 * workspace and scored by the e4m3 tensor-core path, so the scores are those of
 * the MXFP4 values (bit-identical to the e4m3 path on the same values).  Other
 * arguments as there; the workspaces are the e4m3 path's plus rows*H*D +
 * keys*D bytes (256-byte aligned regions).
 * ------------------------------------------------------------------------ */
idx_status idx_mxfp4_to_e4m3(const uint8_t* x, const uint8_t* sf, long long n, int D,
                             uint8_t* out, const idx_options* opt, void* stream);
size_t idx_score_topk_mxfp4_workspace(int rows, long long keys, long long max_len, int H,
                                      int D, int topk, const idx_options* opt);
idx_status idx_score_topk_mxfp4(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k,
                                const uint8_t* k_sf, const float* k_scale, const float* w,
                                const int* ks, const int* ke, int rows, long long keys,
                                long long max_len, int H, int D, int topk, int* out_idx,
                                void* ws, size_t ws_bytes, const idx_options* opt,
                                void* stream);
size_t idx_score_materialise_mxfp4_workspace(int rows, long long keys, int H, int D);
idx_status idx_score_materialise_mxfp4(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k,
                                       const uint8_t* k_sf, const float* k_scale,
                                       const float* w, const int* ks, const int* ke, int rows,
                                       long long keys, int H, int D, float* scores,
                                       long long row_stride, void* ws, size_t ws_bytes,
                                       const idx_options* opt, void* stream);

/* ------------------------------------------------------------------------
 * Serving operators around the indexer: the norm that makes its 8-bit rows, the
 * attention of a decode batch over a paged cache, and the eviction that keeps
 * such a cache within a budget.
 *
 * idx_add_rmsnorm_quant - per row of x [rows, N] (bf16, fp16 or fp32):
 *     h = x + residual (h = x when residual is NULL)
 *     y = h * rsqrt(mean(h^2) + eps) * weight
 *     scale = max(max|y| / 448, 2^-100),   out = e4m3(y / scale)
 * with one scale per row (group 0: scale [rows]; for N = D these are k and
 * k_scale as idx_score_topk reads them) or per `group` consecutive columns
 * (group 32, 64 or 128, N % group == 0: scale [rows, N / group]).  h is kept in
 * fp32 up to the codes and is rounded to x's type only in residual_out.  All of it
 * is fp32: a scale is within 64 units of 2^-24, and a code is the one nearest to
 * 448 h weight / max|h weight|, which is y / scale up to such roundings: a quotient
 * halfway between two codes may get either (|h weight| 3/4 of the largest, say; up
 * to 150 codes in 10^6 of 16-bit rows of 128).
 *   x            rows of N elements, x_stride elements apart (x_stride >= N, so x
 *                may be a column slice of a wider projection)
 *   residual     [rows, N] or NULL, residual_out [rows, N] or NULL (may be
 *                `residual` itself, not x); weight [N]; all of x's type
 *   out [rows, N] e4m3 bytes, scale fp32
 * 1 <= N <= 32768 (IDX_EUNSUPPORTED above).  Pointers are aligned to their
 * element (IDX_EALIGN); rows on 16-byte boundaries (out: 8) with N % 8 == 0 take
 * the vector path, and with a group they have to.  Scales and codes are NaN where the
 * fp32 sum of the row's squares is not finite (a NaN or infinite h, or |h| from about
 * 2^63 on), where mean(h^2) + eps is below 2^-126 (a row of zeros with eps 0), and where a
 * NaN weight enters; other rows are not affected.  No workspace.
 * ------------------------------------------------------------------------ */
idx_status idx_add_rmsnorm_quant(const void* x, long long x_stride, const void* residual,
                                 const void* weight, int rows, int N, float eps, int group,
                                 idx_dtype dt, void* residual_out, uint8_t* out, float* scale,
                                 const idx_options* opt, void* stream);

/* ------------------------------------------------------------------------
 * idx_prefix_attention - attention of B requests with Q new tokens each over a
 * prefix that all of them share and a private part of each one's own, both in
 * one paged cache.  The prefix is read once for the whole batch.
 *
 * Row (b, t, head) sees the prefix's slots 0 .. prefix_len - 1 and the private
 * slots 0 .. lens[b] - (Q - 1 - t) - 1: the newest Q private slots are the new
 * tokens in order, and a token does not see those after it.  With key head
 * head / (Hq / Hkv), z_j = scale * q . k_j:
 *     out = sum_j exp(z_j) v_j / sum_j exp(z_j),   lse = log sum_j exp(z_j)
 * A row that sees nothing gets out 0 and lse -inf; one that sees a NaN logit or one of +inf
 * gets NaN, and so do the weights of its request and key head.
 * Sums of weights times v are fp32 before they are divided, and weights reach 2^8: bf16 values of
 * 2^89 and more may leave it.
 *
 *   q   [B, Q, Hq, D];  k_cache, v_cache [pages, Hkv, page_size, D]; bf16 or fp16
 *   prefix_table [ceil(prefix_len / page_size)] int32: the prefix's pages in order
 *                (may be NULL when prefix_len is 0)
 *   table [B, table_stride] int32: each request's own pages; lens [B] int32
 *   max_len  an upper bound on lens (0 = table_stride * page_size)
 *   w, w_out [B, Hkv, slots] fp32, both NULL or both given (w_out may be w),
 *            slots >= max_len: the weight each private slot has gathered,
 *                w_out[b,h,j] = w[b,h,j] + sum over h's rows of exp(z_j - lse)
 *            for j < lens[b]; the newest Q slots start from 0 whatever w holds.
 *            Slots from lens[b] on are not written.
 *   out [B, Q, Hq, D] of q's type;  lse [B, Q, Hq] fp32 or NULL
 *   ws  idx_prefix_attention_workspace(...) bytes for the same max_len (the
 *       table's width where the call says 0), 256-byte aligned; needs no
 *       clearing between calls.  The size does not shrink when B, Q, Hq, D,
 *       prefix_len, max_len or weights grows: one for the largest serves all.
 * Supported: D 64 or 128; page_size 16, 32, 64 or 128; 1 <= Q <= 16; Hq a
 * multiple of Hkv with Hq / Hkv <= 128; B * Hkv <= 65535; prefix_len, max_len < 2^30; pages >= 1
 * with keys.  The workspace query gives 0 for sizes that the call refuses.  Device errors
 * (IDX_DEV_RANGE): lens[b] outside [0, max_len] is clamped; a page outside
 * [0, pages) reads as zeros, and the results of its request (of all of them,
 * for a page of the prefix) are meaningless.
 * ------------------------------------------------------------------------ */
size_t idx_prefix_attention_workspace(int B, int Q, int Hq, int Hkv, int D, int prefix_len,
                                      int max_len, int weights);
/* The parts that such a call is cut into on the current device: plan[0] parts of the prefix of plan[1]
 * keys each, plan[2] private parts of plan[3] keys, plan[4] 1 when the private parts take the tensor
 * cores' dense path.  Nothing is launched. */
idx_status idx_prefix_attention_plan(int B, int Q, int Hq, int Hkv, int D, int prefix_len, int max_len,
                                     int weights, int* plan);
idx_status idx_prefix_attention(const void* q, const void* k_cache, const void* v_cache,
                                const int* prefix_table, const int* table, const int* lens,
                                const float* w, int B, int Q, int Hq, int Hkv, int D, int pages,
                                int page_size, int prefix_len, long long table_stride,
                                int max_len, long long slots, float scale, idx_dtype dt,
                                void* out, float* lse, float* w_out, void* ws, size_t ws_bytes,
                                const idx_options* opt, void* stream);

/* ------------------------------------------------------------------------
 * idx_cache_evict - keeps at most `budget` of the lens[b] cached slots of each
 * (request, key head), by the weights idx_prefix_attention gathers.
 *
 * Slots are ranked protected first (position < sink, or position >=
 * next_pos[b] - recent), then by weight (a NaN counts as -inf), ties to the lower
 * slot; the first `budget` stay.  Kept slots below `budget` do not move; the i-th hole among
 * them (ascending) takes the K and V rows, weight and position of the i-th kept
 * slot from `budget` on (ascending).  The heads of a request may keep different
 * tokens.  A request of at most `budget` slots keeps everything.
 *
 *   k_cache, v_cache [pages, Hkv, page_size, D] bf16 or fp16, moved in place
 *   table [B, table_stride], lens [B], next_pos [B] int32 (next_pos: tokens the
 *         request has seen, one past the largest position)
 *   w fp32, positions int32 [B, Hkv, slots]; w_out, positions_out likewise: the
 *         first min(lens[b], budget) entries are written (each may be its input,
 *         then only the filled holes are)
 *   lens_out [B] int32 = min(lens[b], budget); not lens itself
 *   max_len  an upper bound on lens (0 = table_stride * page_size)
 *   ws  idx_cache_evict_workspace(...) bytes for the same max_len (the table's
 *       width where the call says 0), 256-byte aligned; the size grows with B, Hkv
 *       and max_len, but not with budget
 * No two requests may share a private page.  budget >= 1, recent, sink >= 0 and
 * recent + sink <= budget (IDX_EINVAL); D 64 or 128; page_size 16, 32, 64 or 128;
 * B * Hkv < 2^28 and pages * Hkv * page_size < 2^32 - 16 (IDX_EUNSUPPORTED).
 * Device errors (IDX_DEV_RANGE): lens[b] outside [0, max_len] is clamped; a K/V
 * row in a page outside [0, pages) is not moved.
 * ------------------------------------------------------------------------ */
size_t idx_cache_evict_workspace(int B, int Hkv, int budget, int max_len);
idx_status idx_cache_evict(void* k_cache, void* v_cache, const int* table, const int* lens,
                           const float* w, const int* positions, const int* next_pos, int B,
                           int Hkv, int D, int pages, int page_size, long long table_stride,
                           int max_len, long long slots, int budget, int recent, int sink,
                           idx_dtype dt, int* lens_out, float* w_out, int* positions_out,
                           void* ws, size_t ws_bytes, const idx_options* opt, void* stream);

/* ------------------------------------------------------------------------
 * A paged K/V cache in 4 bits: the append that writes it and the attention that
 * reads it.  K and V are MXFP4 (see idx_mxfp4_to_e4m3 for the format):
 *   k_codes, v_codes [pages, Hkv, page_size, D / 2] bytes, 16-byte aligned
 *   k_sf, v_sf       [pages, Hkv, page_size, D / 32] bytes, 16-byte aligned
 *   table [B, table_stride] int32: each request's pages; lens [B] int32: its slots
 *         in the cache, the call's new tokens among them (the last ones)
 *   q_start [B + 1] int32: tokens q_start[b] .. q_start[b + 1] - 1 of the call's T
 *         are request b's new ones, in order; NULL: T / B each (T % B == 0).
 * Token i of request b's n new ones has position lens[b] - n + i.
 * Supported: D 64 or 128; page_size 16, 32, 64 or 128; B <= 65535;
 * pages * Hkv * page_size < 2^31 - 256 (IDX_EUNSUPPORTED).
 *
 * idx_cache_append_mxfp4 - writes the new tokens' keys and values at their
 * positions.  Per block of 32 elements: e = floor(log2 max|x|) - 2, at least -127
 * (0 for a block of zeros), scale byte e + 127, and the e2m1 code nearest to
 * x / 2^e, ties to even, saturated at 6: exact in every bit.  A block with an
 * element that is not finite gets the NaN scale 255 and zero codes.
 *   k, v  [T, Hkv, D] bf16 or fp16, tokens k_stride, v_stride elements apart (at least
 *         Hkv * D, so both may be slices of one projection); rows on 16-byte boundaries
 *         are read with wide loads, others element by element
 * A token whose page is negative is not kept.  A request's last slots are written whatever they hold, so lens has to
 * count its new tokens (after an idx_cache_resize: that served the row, see there).  Tokens outside every request are not
 * read.  No two requests may share the page of a new token.  Device errors
 * (IDX_DEV_RANGE): a position outside [0, table_stride * page_size), a page from `pages` on or a request that
 * ends behind token T: the token is not written.  No workspace.
 *
 * idx_window_attention_mxfp4 - attention of every request's new tokens (one for a decode
 * step, a chunk of a prompt, a few drafted ones) over its cache, causal, with a sliding
 * window and first tokens that stay visible.  The token at position p sees slots j <= p
 * with j < sink or j > p - window (all j <= p when window is 0, and sink does not count).
 * With key head head / (Hq / Hkv), z_j = scale * q . k_j over those slots:
 *     out = sum_j exp(z_j) v_j / sum_j exp(z_j),   lse = log sum_j exp(z_j).
 * A row that sees nothing gets out 0 and lse -inf.  A row that sees a slot with a NaN scale
 * (255, in K or V) or a logit that is NaN or +inf gets NaN, and no other row does.  Weights below 2^-31
 * of a row's largest count as 0.  Values 2^120 and more below the largest in their 32 columns, of a slot that
 * a row of the same request sees, lose bits.  Where many rows of a request share a key head (a prompt),
 * values may be taken in q's type: in fp16 those below 2^-23 are then rounded to multiples of 2^-24 and scales above
 * 2^13 count as NaN scales; in bf16 scales above 2^125 do, and values below 2^-60 lose bits beside scales of V
 * above 2^87 that a row of the same request sees.  q . k itself, before scale, is fp32 there.
 *   q    [T, Hq, D] bf16 or fp16, tokens q_stride elements apart, rows on 16-byte boundaries
 *   max_q   an upper bound on a request's new tokens (0 = T)
 *   max_len an upper bound on lens (0 = table_stride * page_size)
 *   out  [T, Hq, D] of q's type, contiguous, apart from q; lse [T, Hq] fp32 or NULL.  Rows of
 *        tokens outside every request are not written.
 *   ws   idx_window_attention_mxfp4_workspace(...) bytes for the same arguments (max_q and
 *        max_len as the call counts them), 256-byte aligned; needs no clearing between calls.
 *        The size does not shrink when an argument grows (a window of 0 is the largest).
 * Pages without a slot that a row of the request sees are not read and need not exist (table entries of any
 * value).  Other slots of the pages that are read may be read too, and change no bit of a result, whatever they
 * hold.  Further limits: Hq a multiple of Hkv with Hq / Hkv <= 128; T * Hq < 2^31 - 256; max_len, window,
 * sink < 2^30.  Device errors (IDX_DEV_RANGE): lens[b] outside [0, max_len] is clamped; where q_start is not in
 * order, a request has more than max_q tokens or a row sees a page outside [0, pages), the request's results
 * are meaningless.
 * ------------------------------------------------------------------------ */
idx_status idx_cache_append_mxfp4(const void* k, long long k_stride, const void* v,
                                  long long v_stride, uint8_t* k_codes, uint8_t* k_sf,
                                  uint8_t* v_codes, uint8_t* v_sf, const int* table,
                                  const int* lens, const int* q_start, int B, int T, int Hkv,
                                  int D, int pages, int page_size, long long table_stride,
                                  idx_dtype dt, const idx_options* opt, void* stream);
size_t idx_window_attention_mxfp4_workspace(int B, int T, int max_q, int Hq, int Hkv, int D,
                                            int max_len, int window, int sink);
/* How such a call is cut on the current device: plan[0] splits of the keys that a tile of rows sees, plan[1]
 * keys each, plan[2] 1 when the rows take the tensor cores' dense path (many rows per request and key head),
 * plan[3] the most rows of a tile.  Nothing is launched. */
idx_status idx_window_attention_mxfp4_plan(int B, int T, int max_q, int Hq, int Hkv, int D, int max_len, int window,
                                           int sink, int* plan);
idx_status idx_window_attention_mxfp4(const void* q, long long q_stride, const uint8_t* k_codes,
                                      const uint8_t* k_sf, const uint8_t* v_codes,
                                      const uint8_t* v_sf, const int* table, const int* lens,
                                      const int* q_start, int B, int T, int max_q, int Hq, int Hkv,
                                      int D, int pages, int page_size, long long table_stride,
                                      int max_len, int window, int sink, float scale, idx_dtype dt,
                                      void* out, float* lse, void* ws, size_t ws_bytes,
                                      const idx_options* opt, void* stream);

/* ------------------------------------------------------------------------
 * The pages of a cache (of any element type): which rows of a page table hold
 * them.  refs[p] is the number of table entries, over all rows and within their
 * lengths, that name page p; a page is free when it is 0 (or less).
 *   table [B, table_stride], lens [B] (in slots), refs [pages] int32
 *   refs_out, table_out, lens_out: the same after the call; each may be its input.  Of a row of
 *         table_out the first ceil(lens_out / page_size) entries are written (in place: those
 *         that change).
 *   caches [n_caches] HOST array of device arrays whose pages move or are copied, page_bytes
 *         [n_caches] bytes of a page in each (HOST): K and V, codes and scales, the indexer's
 *         keys ...  Bases 16-byte aligned and page_bytes a multiple of 16 (IDX_EALIGN);
 *         n_caches <= 8.
 * page_size 16, 32, 64 or 128; table_stride * page_size < 2^31; B <= 2^24; pages <= 2^31 - 256
 * (IDX_EUNSUPPORTED).  Results do not depend on the order in which threads run.  Device errors
 * (IDX_DEV_RANGE): a length outside [0, table_stride * page_size] counts as 0 in a fork and leaves its row
 * as it is otherwise; a table entry outside [0, pages) within a row's length is kept and not counted.
 *
 * idx_cache_fork - row i takes over the pages and the length of row parent[i] as they were
 * before the call and gives its own back; all rows at once (the next step of a beam search).
 * parent[i] = i leaves the row, -1 ends it (length 0).  Nothing is copied: rows share pages
 * until one of them grows (idx_cache_resize).  Other parents outside [0, B): IDX_DEV_RANGE, the
 * row is left.  lens_out must not be parent (IDX_EINVAL).  ws: idx_cache_fork_workspace(...)
 * bytes, 256-byte aligned, when table_out is table or lens_out is lens; NULL and 0 otherwise.
 *
 * idx_cache_resize - row i goes from lens[i] to new_lens[i] slots.  First the rows that shrink
 * give back the pages that they no longer need.  Then the rows that grow take free pages, the
 * lowest free page first, in the order of rows and within a row of its slots.  A row that grows
 * into a partly filled last page which other entries name too (refs above 1 once the rows have
 * shrunk) takes a page for a copy of it first and gives the shared one back; every such row
 * copies, also when all that hold the page grow (it is free from the next call on).  From the
 * first row on for which the free pages do not suffice, rows that want pages keep their pages
 * and length, and IDX_DEV_PAGES is raised; lens_out tells.  A new length outside [0, table_stride
 * * page_size]: IDX_DEV_RANGE, the row is left.  A row whose lens_out is not its new length has no slots for the
 * tokens that it was to grow by: an append with that length would write them over its newest slots, and over other
 * rows' where it shares their page.  Until it is served the append and the attention get 0 as its length
 * (lens_out[i] == new_lens[i] ? lens_out[i] : 0, on the device): its tokens are not kept, and its rows see nothing.
 * ws: idx_cache_resize_workspace(...) bytes, 256-byte aligned.
 *
 * idx_cache_compact - moves the live pages to the front: with `live` pages whose count is above
 * 0, the i-th free page below `live` takes the contents and count of the i-th live page from there on,
 * and the tables follow.  live [1] int32 is written.  Counts of all other pages become 0.
 * ws: idx_cache_compact_workspace(...) bytes, 256-byte aligned.
 * ------------------------------------------------------------------------ */
size_t idx_cache_fork_workspace(int B, long long table_stride);
idx_status idx_cache_fork(const int* refs, const int* table, const int* lens, const int* parent,
                          int B, int pages, int page_size, long long table_stride, int* refs_out,
                          int* table_out, int* lens_out, void* ws, size_t ws_bytes,
                          const idx_options* opt, void* stream);
size_t idx_cache_resize_workspace(int B, int pages, long long table_stride);
idx_status idx_cache_resize(void* const* caches, const long long* page_bytes, int n_caches,
                            const int* refs, const int* table, const int* lens,
                            const int* new_lens, int B, int pages, int page_size,
                            long long table_stride, int* refs_out, int* table_out, int* lens_out,
                            void* ws, size_t ws_bytes, const idx_options* opt, void* stream);
size_t idx_cache_compact_workspace(int B, int pages);
idx_status idx_cache_compact(void* const* caches, const long long* page_bytes, int n_caches,
                             const int* refs, const int* table, const int* lens, int B, int pages,
                             int page_size, long long table_stride, int* refs_out, int* table_out,
                             int* live, void* ws, size_t ws_bytes, const idx_options* opt,
                             void* stream);

/* Static text for a status code. */
const char* idx_status_string(idx_status s);

/* Library version, (major << 16) | minor. */
int idx_version(void);

/* Text of the CUDA error behind the calling thread's last IDX_ECUDA or
 * IDX_EUNSUPPORTED that came from a CUDA call ("" when there was none). */
const char* idx_last_cuda_error(void);

/* Number of kernels this library has launched in this process (all devices,
 * all threads); a diagnostic for benchmarks. */
unsigned long long idx_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* IDX_H_ */
