/*
 * ds_sparse_mla.h -- C ABI of the GB300 (sm_103a) deterministic sparse top-k
 * and sparse MLA attention library (libds_sparse_mla.so).
 *
 * What the library computes
 * -------------------------
 * The two steps of DeepSeek-V4-style sparse MLA described on the pages
 * "[DeepSeek-V4][Preview][DO NOT MERGE] Batch-invariant kernels for 0-diff
 * RL" (vllm-project/vllm PR 54955), sections "Deterministic sparse top-k" and
 * "Sparse MLA and FlashMLA", and "[Bugfix] Make DSV4 sparse MLA work
 * end-to-end for plain decode, MTP, and DSpark" (vllm-project/vllm PR 51538),
 * section "What is fixed":
 *
 *   1. ds_topk_per_row: for every row, the k positions with the largest
 *      indexer scores under the total order (score descending, position
 *      ascending), written in ascending position order, -1 in unused slots.
 *   2. ds_sparse_mla_decode / ds_sparse_mla_prefill: gather the selected
 *      entries of a paged latent KV cache (64 entries per page, 576 = 512
 *      latent + 64 rope dims, one latent row shared by every head) and
 *      compute out = softmax(scale * q K^T) V with V = the first 512 dims of
 *      the same rows, plus lse = ln(sum exp(scale * q K^T)).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every pointer argument is a DEVICE pointer (cudaMalloc'd or otherwise
 *    device-accessible) unless stated otherwise. Nothing is allocated or
 *    freed inside; outputs and workspaces are owned by the caller, as in the
 *    caller-owned-output contract of "[JJ] Preallocate DeepSeek V4
 *    padded-query output" (local-inference-lab/vllm PR 671, section
 *    "Operation contract").
 *  - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *    stream). Every call only enqueues work on it and never synchronises the
 *    host, so calls may be captured into a CUDA graph.
 *  - Arguments are validated on the host before anything is launched.
 *    Unsupported shapes are a hard error (PR 54955: "missing kernel support
 *    is a hard error rather than a silent fallback"); ds_last_error() names
 *    the offending parameter and the allowed set (PR 51538, "SM120 gate").
 *  - Row lengths are computed signed and clamped at 0 before any decision,
 *    so a negative length from a padded request is an empty row, never a
 *    huge unsigned value (PR 51538, "What is fixed").
 *  - Offsets inside the kernels are 64-bit: tensors may exceed 2^31
 *    elements (PR 54955, the 64-bit offset fix).
 *  - Results never depend on the rest of the batch: every row's output is
 *    bit-identical whether it runs alone or inside any batch, because each
 *    row's work is split and reduced in an order fixed by k alone.
 *  - Return value: DS_OK, or a ds_status error code. Any code other than
 *    DS_OK or DS_ERR_CUDA means nothing was launched; DS_ERR_CUDA means a
 *    launch failed (cudaGetLastError() reported an error).
 */
#ifndef DS_SPARSE_MLA_H
#define DS_SPARSE_MLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DS_OK = 0,
  DS_ERR_NULL = 1,         /* a required pointer is NULL                      */
  DS_ERR_SHAPE = 2,        /* a size is negative or inconsistent              */
  DS_ERR_UNSUPPORTED = 3,  /* a size is outside the supported set             */
  DS_ERR_DTYPE = 4,        /* unknown kv_dtype                                */
  DS_ERR_ALIGN = 5,        /* a pointer is not aligned as required            */
  DS_ERR_WORKSPACE = 6,    /* workspace missing or smaller than required      */
  DS_ERR_CUDA = 7          /* the CUDA runtime reported an error at launch    */
} ds_status;

typedef enum {
  DS_KV_BF16 = 0,          /* kv row = 576 bfloat16 (1152 bytes)              */
  DS_KV_FP8_E4M3 = 1       /* kv row = 656 bytes, layout below                */
} ds_kv_dtype;

/*
 * FP8 KV row layout (656 bytes, 16-byte aligned): bytes [0, 512) are the
 * 512 latent dims as OCP FP8 E4M3 codes; bytes [512, 528) are four
 * little-endian float32 scales, one per 128-dim group (dims 0-127, 128-255,
 * 256-383, 384-511), kept contiguous as in the FP8 KV cache of
 * "MooreThreads/vllm-musa PR 178" (optimisation table, contiguous FP32 scale
 * groups); bytes [528, 656) are the 64 rope dims as bfloat16. A latent value
 * is code * scale of its group.
 */
#define DS_PAGE_BLOCK_SIZE 64
#define DS_D_QK 576
#define DS_D_V 512
#define DS_KV_ROW_BYTES_BF16 1152
#define DS_KV_ROW_BYTES_FP8 656
#define DS_INDEXER_HEAD_DIM 128

/* Device-side error bits ORed into *err_flag (when err_flag != NULL). */
#define DS_DEVERR_IDX 1      /* an idx entry other than -1 outside [0, lens[row]) */
#define DS_DEVERR_PAGE 2     /* a block-table slot beyond bt_stride, or a page id
                                outside [0, num_pages)                            */
#define DS_DEVERR_ROWREQ 4   /* prefill: row_req[t] outside [0, num_requests)     */
#define DS_DEVERR_TIMEOUT 8  /* an internal pipeline wait gave up (library bug)   */
#define DS_DEVERR_NOPAGE 16  /* pages: the pool has too few free pages            */
#define DS_DEVERR_LEN 32     /* a length that the operation cannot take           */
#define DS_DEVERR_SHARED 64  /* a page to be rewritten that other rows hold too   */

/*
 * Message of the last error on the calling host thread ("" if none). The
 * string is thread-local and stays valid until the next call on this thread.
 */
const char* ds_last_error(void);

/*
 * 1 if (num_heads, topk, page_block_size, d_qk, d_v, kv_dtype) is a shape the
 * attention entry points accept, else 0 with ds_last_error() naming the first
 * parameter that missed and the values that are available. Lets a caller
 * validate a model configuration at init time instead of at its first decode
 * (PR 51538, "SM120 gate"). Supported: num_heads in {16, 32, 64, 128}; topk a
 * multiple of 64 in [64, 2048]; page_block_size 64; d_qk 576; d_v 512;
 * kv_dtype DS_KV_BF16 or DS_KV_FP8_E4M3.
 */
int ds_supported_config(int num_heads, int topk, int page_block_size, int d_qk, int d_v,
                        int kv_dtype);

/*
 * Workspace bytes that let ds_topk_per_row spread every row of this shape
 * over the whole GPU (the grid kernel), or 0 for shapes that another kernel
 * serves without one. Nonzero for batches of at most 256 rows of at most
 * 131072 scores (8192 to 2^24 scores in all) that are neither 16 or more rows
 * of at most 32768 nor 256 or more rows of at most 65536: 256 header bytes,
 * then 64 KiB of candidate list and 8 bytes of bookkeeping for each of the
 * ceil((row_stride + 255) / 8192) segments a row may have, per row. k does
 * not change it.
 */
size_t ds_topk_workspace_size(int64_t num_rows, int64_t row_stride, int k);

/*
 * Workspace bytes ds_sparse_mla_decode / ds_sparse_mla_prefill need for
 * num_rows query rows (decode requests or prefill tokens), num_heads heads
 * and top-k width k: the per-split partial results (the unnormalised output
 * rounded to bfloat16, the running maximum and sum in float32). The number
 * of splits is a function of k alone. Returns 0 for an unsupported shape.
 */
size_t ds_sparse_mla_workspace_size(int64_t num_rows, int num_heads, int k);

/*
 * Deterministic per-row top-k ("Deterministic sparse top-k", PR 54955; length
 * clamp and -1 padding from PR 51538, "What is fixed").
 *
 *  scores      float32, row-major [num_rows, row_stride]; 4-byte aligned.
 *  row_stride  elements between consecutive rows, 1 <= row_stride <= 2^28.
 *  num_rows    >= 0 (0 launches nothing).
 *  row_starts  int32 [num_rows]; row_ends int32 [num_rows]. Row b ranks the
 *              scores at positions [row_starts[b], row_starts[b] + L_b) with
 *              L_b = clamp(row_ends[b] - row_starts[b], 0,
 *                          row_stride - row_starts[b]),
 *              computed signed; a row_starts[b] outside [0, row_stride] gives
 *              L_b = 0.
 *  k           1 <= k <= 16384.
 *  idx_out     int32 [num_rows, k], written fully: the selected positions
 *              RELATIVE to row_starts[b], ascending, then -1 in slots
 *              [min(k, L_b), k). Rows with L_b <= k select every position.
 *
 * Order: larger score first; equal scores (-0.0 equals +0.0) by lower
 * position; NaN ranks below -inf and NaNs tie with one another. The selected
 * set is therefore unique and the output is bit-exact and independent of the
 * batch.
 *
 *  workspace   NULL, or 256-byte aligned device memory of workspace_bytes.
 *              With at least ds_topk_workspace_size() bytes (when that is
 *              nonzero) and scores 16-byte aligned, the grid kernel runs:
 *              one cooperative launch whose CTAs are all resident, preceded
 *              by a zero fill of the workspace's first 256 bytes (so its
 *              contents need no initialisation); otherwise a kernel that
 *              needs no workspace runs. The output is identical either way.
 *              After the grid kernel, the int32 at byte offset 8 of the
 *              workspace is 0; a nonzero value means one of its bounded
 *              waits gave up (not expected: the launch keeps every CTA
 *              resident) and idx_out is unspecified. Concurrent calls need
 *              separate workspaces.
 */
int ds_topk_per_row(const float* scores, int64_t row_stride, int64_t num_rows,
                    const int32_t* row_starts, const int32_t* row_ends, int k,
                    int32_t* idx_out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Sparse MLA decode over a paged latent KV cache ("Sparse MLA and FlashMLA",
 * PR 54955: decode gathers the selected KV and runs sparse attention; slot
 * arithmetic slot = block_id * block_size + offset from PR 51538).
 *
 *  q            bfloat16 [num_rows, num_heads, 576], 16-byte aligned.
 *  kv_pages     DS_KV_BF16: bfloat16 [num_pages, 64, 576];
 *               DS_KV_FP8_E4M3: uint8 [num_pages, 64, 656]. 16-byte aligned.
 *  num_pages    >= 1.
 *  block_table  int32 [num_rows, bt_stride]: page id of each 64-position
 *               block of row b's context.
 *  idx          int32 [num_rows, k]: context positions to attend to (the
 *               output of ds_topk_per_row); -1 entries are skipped.
 *  lens         int32 [num_rows]: context length of each row.
 *  scale        softmax scale applied to q.K (e.g. 1/sqrt(576)).
 *  out          bfloat16 [num_rows, num_heads, 512], 16-byte aligned.
 *  lse          float32 [num_rows, num_heads]: natural-log sum of
 *               exp(scale * q.K) over the valid entries (-inf if none).
 *  workspace    >= ds_sparse_mla_workspace_size(num_rows, num_heads, k)
 *               bytes, 256-byte aligned; contents need no initialisation.
 *  err_flag     optional int32 device word (NULL = no report). Entries with
 *               an idx outside [0, lens[b]) (other than -1), or whose page
 *               lookup misses, are skipped and a DS_DEVERR_* bit is ORed in;
 *               the kernels never trap.
 *
 * Entry j of row b is valid iff 0 <= idx[b,j] < lens[b], idx[b,j]/64 <
 * bt_stride and the page id lies in [0, num_pages). A row with no valid entry
 * gives out = 0 and lse = -inf.
 */
int ds_sparse_mla_decode(const void* q, const void* kv_pages, int kv_dtype, int64_t num_pages,
                         const int32_t* block_table, int64_t bt_stride,
                         const int32_t* idx, const int32_t* lens,
                         int64_t num_rows, int num_heads, int k, float scale,
                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                         int32_t* err_flag, void* stream);

/*
 * Sparse MLA prefill: as decode, with one query row per token. Token t reads
 * block-table row row_req[t] (int32 [num_tokens], in [0, num_requests)) and
 * is computed on its own, never through a batch-level plan ("Batch-invariant
 * prefill chunks each request independently", PR 54955). block_table is
 * int32 [num_requests, bt_stride]; idx, lens, q, out and lse are indexed by
 * token. A row_req outside [0, num_requests) gives out = 0, lse = -inf and
 * sets DS_DEVERR_ROWREQ.
 */
int ds_sparse_mla_prefill(const void* q, const void* kv_pages, int kv_dtype, int64_t num_pages,
                          const int32_t* block_table, int64_t bt_stride, int64_t num_requests,
                          const int32_t* row_req, const int32_t* idx, const int32_t* lens,
                          int64_t num_tokens, int num_heads, int k, float scale,
                          void* out, float* lse, void* workspace, size_t workspace_bytes,
                          int32_t* err_flag, void* stream);

/*
 * Allocation-free variant of ds_sparse_mla_decode. The pages have no
 * counterpart to this entry point; it exists for callers that cannot provide
 * device scratch memory: code running under a memory manager that owns all
 * device memory, code in the middle of recording a CUDA graph (where a plain
 * cudaMalloc is not allowed), and loops that cannot afford cudaMalloc's
 * implicit device synchronisation.
 *
 * Arguments, results and errors are those of ds_sparse_mla_decode, minus the
 * workspace. The scratch is a built-in 32 MiB device array of this library
 * (each GPU holds it from the time the library's module is first loaded there
 * until the process exits). Calls whose ds_sparse_mla_workspace_size() exceeds
 * 32 MiB return DS_ERR_WORKSPACE with a message; nothing is launched. The call
 * itself performs no cudaMalloc/cudaFree or other allocation.
 *
 * The first call on each device looks up the array's device address (with
 * that device current); make that first call before any stream capture. A
 * lookup that fails returns DS_ERR_CUDA and is not remembered: the next call
 * tries again.
 * Every call shares the one array, and each call overwrites what the
 * previous one left there: calls that can overlap on the GPU (on different
 * streams without ordering between them) race on it and must not be issued.
 */
int ds_sparse_mla_decode_noalloc(const void* q, const void* kv_pages, int kv_dtype,
                                 int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                                 const int32_t* idx, const int32_t* lens, int64_t num_rows,
                                 int num_heads, int k, float scale, void* out, float* lse,
                                 int32_t* err_flag, void* stream);

/*
 * Sparse MLA decode over the concatenation [top-k entries of the compressed
 * KV || sliding-window entries of the window KV], with per-head attention
 * sinks ("[DeepSeek-V4][Preview][DO NOT MERGE] Batch-invariant kernels for
 * 0-diff RL", section "Sparse MLA and FlashMLA": decode gathers compressed
 * and sliding-window KV and runs one sparse attention over both; attention
 * sinks keep -inf padding. "[Bugfix] Make DSV4 sparse MLA work end-to-end
 * ...", section "What is fixed": the window index list is padded to a
 * multiple of 64 entries).
 *
 * The first ten arguments and q, out, lse, workspace, err_flag and stream
 * are those of ds_sparse_mla_decode (k is the top-k width). The window:
 *  swa_pages        the window pool, same row format and kv_dtype as
 *                   kv_pages, 16-byte aligned; swa_num_pages >= 1.
 *  swa_block_table  int32 [num_rows, swa_bt_stride]: page id of each
 *                   64-position block of the row's window context.
 *  swa_idx          int32 [num_rows, swa_width]: window positions (-1 =
 *                   padding); an entry is valid iff 0 <= swa_idx < swa_lens[row]
 *                   and its page lookup hits, like a top-k entry.
 *  swa_lens         int32 [num_rows].
 *  swa_width        0 (no window; the window arguments may be NULL) or a
 *                   multiple of 64 in [64, 512].
 *  attn_sink        optional float32 [num_heads] (NULL = no sinks): the sink
 *                   logit of each head, in the units of scale * q.K (natural
 *                   log). It joins the softmax denominator with no value row:
 *                   out = sum_j exp(S_j) V_j / (sum_j exp(S_j) + exp(sink)),
 *                   lse = log(sum_j exp(S_j) + exp(sink)); -inf = no sink.
 *                   A head with no valid entry gives out = 0 and lse = sink.
 *  workspace        >= ds_sparse_mla_swa_workspace_size(num_rows, num_heads,
 *                   k, swa_width) bytes, 256-byte aligned.
 *
 * The concatenated list is cut into 64-entry tiles spread evenly over
 * max(ceil(k / 512), ceil((k + swa_width) / 768)) splits, so the reduction
 * order depends on k and swa_width only, never on the batch.
 */
int ds_sparse_mla_decode_swa(const void* q, const void* kv_pages, int kv_dtype, int64_t num_pages,
                             const int32_t* block_table, int64_t bt_stride, const int32_t* idx,
                             const int32_t* lens, int k, const void* swa_pages,
                             int64_t swa_num_pages, const int32_t* swa_block_table,
                             int64_t swa_bt_stride, const int32_t* swa_idx,
                             const int32_t* swa_lens, int swa_width, const float* attn_sink,
                             int64_t num_rows, int num_heads, float scale, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, int32_t* err_flag,
                             void* stream);

/* Workspace bytes of ds_sparse_mla_decode_swa (0 for an unsupported shape). */
size_t ds_sparse_mla_swa_workspace_size(int64_t num_rows, int num_heads, int k, int swa_width);

/*
 * Indexer scores (the "MQA logits" that the top-k selects from). "[SM120]
 * Sync DS4 with upstream main + validated perf backports" routes these
 * logits through their own kernel and sizes a paged-MQA warm-up; "[Bugfix]
 * Make DSV4 sparse MLA work end-to-end ...", section "What is fixed", gives
 * the indexer one signed context length per query token. The pages give no
 * formula; this library computes the lightning indexer of the
 * DeepSeek-V3.2-Exp technical report: for query row r and position s,
 *
 *   logits[r, s] = sum_j weights[r, j] * max(0, q[r, j, :] . k[s, :])
 *
 * (multi-head queries, one shared key per position), with fp32 accumulation
 * and the heads summed in order j = 0, 1, ...
 *
 *  q              bfloat16 [num_rows, num_heads, 128], 16-byte aligned.
 *  weights        float32 [num_rows, num_heads].
 *  k_pages        bfloat16 [num_pages, 64, 128] key cache, 16-byte aligned;
 *                 the key of position s of a row is
 *                 k_pages[block_table[req, s / 64], s % 64].
 *  block_table    int32 [num_requests, bt_stride]; req = row_req[r], or r
 *                 when row_req is NULL (then num_requests >= num_rows).
 *  lens           int32 [num_rows]: row r scores positions 0 .. L_r - 1 with
 *                 L_r = clamp(lens[r], 0, 64 * bt_stride), computed signed.
 *  logits         float32 [num_rows, logits_stride], logits_stride >=
 *                 64 * bt_stride; positions at or beyond L_r are not written.
 *                 Feed it to ds_topk_per_row with row_starts = 0 and
 *                 row_ends = lens (the same clamp applies there).
 *  err_flag       optional int32 device word: DS_DEVERR_PAGE for a page id
 *                 outside [0, num_pages) (its 64 positions score -inf),
 *                 DS_DEVERR_ROWREQ for a row_req outside [0, num_requests)
 *                 (the row scores nothing).
 *
 * Supported: num_heads 16, 32 or 64; head dim 128. A row's scores depend on
 * that row's q, weights and keys alone (bitwise the same in any batch).
 * Asynchronous on `stream`; allocates nothing.
 */
int ds_indexer_logits(const void* q, const float* weights, const void* k_pages,
                      int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                      int64_t num_requests, const int32_t* row_req, const int32_t* lens,
                      int64_t num_rows, int num_heads, int head_dim, float* logits,
                      int64_t logits_stride, int32_t* err_flag, void* stream);

/*
 * KV cache write: new latent rows into the paged cache, as bf16 rows or
 * quantised to the FP8 layout above (MooreThreads/vllm-musa PR 178,
 * optimisation table: the FP8 attention cache write, with each row's FP32
 * scale groups kept contiguous).
 *
 *  latent     bfloat16 [num_rows, 576] (512 latent dims, then 64 rope dims),
 *             16-byte aligned.
 *  slots      int64 [num_rows], 8-byte aligned: row i goes to slot
 *             page * 64 + offset ("[Bugfix] Make DSV4 sparse MLA work
 *             end-to-end ...", section "What is fixed": slot =
 *             block_id * block_size + offset). A negative slot is a padding
 *             row and writes nothing (never into page 0); a slot at or past
 *             num_pages * 64 writes nothing and ORs DS_DEVERR_PAGE into
 *             err_flag.
 *  kv_dtype   DS_KV_BF16: the row is copied. DS_KV_FP8_E4M3: per group of
 *             128 latent dims, scale = amax / 448 (1 for an all-zero group),
 *             code = E4M3(x / scale) rounded to nearest, ties to even,
 *             saturating at +-448 (float32 division); the four float32
 *             scales and the 64 bf16 rope dims follow the codes.
 *  kv_pages   the pool (layout as for ds_sparse_mla_decode), 16-byte aligned;
 *             only the written slots change.
 *  err_flag   optional int32 device word (NULL = no report).
 *
 * Rows are independent: a row's bytes depend on that row alone. num_rows = 0
 * is a no-op. Slots that repeat are written in an unspecified order.
 */
int ds_kv_cache_write(const void* latent, int64_t num_rows, const int64_t* slots, int kv_dtype,
                      void* kv_pages, int64_t num_pages, int32_t* err_flag, void* stream);

/*
 * Block-scaled 8-bit cache ("kv8"): the paged cache of layers that keep keys
 * and values per head (draft layers and the dense layers beside the sparse
 * ones), held as OCP FP8 E4M3 codes with one float32 scale for each page of
 * 64 positions, side (key or value) and head:
 *
 *  kv_pages     uint8 [num_pages, 2, num_kv_heads, 64, head_dim], 16-byte
 *               aligned; index 0 of the second axis holds keys, 1 values.
 *  kv_scales    float32 [num_pages, 2, num_kv_heads].
 *               value = code * scale of its page, side and head. Scales are
 *               positive and finite; ds_kv8_append writes powers of two.
 *               (A row whose largest score passes 2^22 in magnitude, where
 *               float32 cannot tell weights apart any more, can give NaN;
 *               a score below float32's range counts as not seen.
 *               Where value scales of one request differ by a
 *               factor of 2^100 or more, a page of the small ones can drop
 *               out of a row's softmax.)
 *
 * It uses the block tables and the page size of the latent cache: position s
 * of a request lies in slot s % 64 of page block_table[request, s / 64]. What
 * a page holds behind the request's last position is never used, whatever it
 * is (NaN codes included).
 *
 * head_dim is 64 or 128; num_heads is a multiple of num_kv_heads (query head
 * h reads key/value head h / (num_heads / num_kv_heads)), both at most 1024,
 * bt_stride is at most 2^24, num_requests at most 2^20, num_tokens (of append
 * and prefill) at most 2^24, and the product num_pages * 2 * num_kv_heads * 64
 * below 2^31.
 *
 * Ragged calls give each request's tokens by token_starts, int32
 * [num_requests + 1] in device memory, never decreasing: request r owns rows
 * token_starts[r] .. token_starts[r + 1] - 1 of the token-indexed arrays (the
 * values are clamped to [0, num_tokens]). lens[r] counts the positions of
 * request r INCLUDING these n tokens, which are its last n positions.
 *
 *
 * ds_kv8_append: the keys and values of new tokens into the cache.
 *
 *  k, v         bfloat16, row t at k + t * k_stride (v + t * v_stride)
 *               elements, each row [num_kv_heads, head_dim] contiguous;
 *               16-byte aligned, strides multiples of 8 and at least
 *               num_kv_heads * head_dim (slices of a fused projection).
 *  block_table  int32 [num_requests, bt_stride].
 *  err_flag     optional: DS_DEVERR_LEN for a request with lens[r] < n (it
 *               writes nothing), DS_DEVERR_PAGE for a page beyond bt_stride
 *               or outside the pool (its tokens are not written).
 *
 * Scale of a touched (page, side, head): a = max |x| of the new tokens in the
 * page; need = the smallest power of two with a <= 448 * need, its exponent
 * limited to [-60, 120] (0 if a = 0); old = the present scale if the page
 * holds earlier positions of the request, else 0; scale = max(old, need), or
 * 2^-60 if both are 0. Earlier codes become E4M3(code * (old / scale)) when
 * the scale grew, new ones are E4M3(x / scale), rounded to nearest with ties
 * to even, saturating at +-448; a quotient or product that float32 does not
 * hold (the scale before the call was no power of two) is rounded to float32
 * first. A NaN becomes the NaN code and does not enter
 * a. With power-of-two scales a growing scale changes earlier values only
 * where their codes leave E4M3's normal range.
 *
 * A page that is written belongs to one request of the call (pages shared
 * after ds_pages_fork are full ones, which are never written again). Calls
 * that repeat a page give unspecified bytes in it.
 */
int ds_kv8_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                  int64_t num_tokens, const int32_t* token_starts, int64_t num_requests,
                  const int32_t* block_table, int64_t bt_stride, const int32_t* lens,
                  int num_kv_heads, int head_dim, void* kv_pages, float* kv_scales,
                  int64_t num_pages, int32_t* err_flag, void* stream);

/*
 * ds_kv8_decode: attention of next_n new tokens per request (1, or target and
 * draft tokens under multi-token prediction) over the kv8 cache. Token j of
 * request r sees the first clamp(lens[r] - next_n + 1 + j, 0, 64 * bt_stride)
 * positions: s_i = scale * q . k_i, out = sum_i softmax(s)_i v_i, lse =
 * ln sum_i exp(s_i); a token that sees nothing gives out = 0, lse = -inf.
 * (A weight times its page's value scale is held in 11 bits down to 2^-17 of
 * the row's largest and in fewer below; under 2^-27 of it, it adds nothing to
 * out. lse and the weights' sum are fp32. The form in which q is multiplied
 * moves a score by at most 2^-14, whatever q holds.)
 *
 *  q            bfloat16, token (r, j) at q + (r * next_n + j) * q_stride
 *               elements, [num_heads, head_dim] contiguous; 16-byte aligned,
 *               q_stride a multiple of 8 and at least num_heads * head_dim.
 *               A non-finite value makes its head's outputs NaN.
 *  next_n       1 .. 64.
 *  out          bfloat16 [num_requests, next_n, num_heads, head_dim], 16-byte
 *               aligned; lse float32 [num_requests, next_n, num_heads].
 *  workspace    >= ds_kv8_decode_workspace_size() bytes, 256-byte aligned;
 *               contents need no initialisation.
 *  err_flag     optional: DS_DEVERR_PAGE for a page outside the pool (its
 *               positions are left out of the softmax).
 *
 * num_requests * next_n * num_heads is below 2^31. A request's outputs depend
 * on its own q, length and cache alone, bit for bit: contexts are cut at fixed
 * positions, whatever else the batch holds.
 */
int ds_kv8_decode(const void* q, int64_t q_stride, const void* kv_pages, const float* kv_scales,
                  int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                  const int32_t* lens, int64_t num_requests, int next_n, int num_heads,
                  int num_kv_heads, int head_dim, float scale, void* out, float* lse,
                  void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream);

/*
 * Workspace bytes of ds_kv8_decode (0 for an unsupported shape). They follow
 * the table's width, not the lengths: up to 32 spans for each row of q to
 * 131072 positions, one for each 4096 above.
 */
size_t ds_kv8_decode_workspace_size(int64_t num_requests, int next_n, int num_heads,
                                    int num_kv_heads, int head_dim, int64_t bt_stride);

/*
 * ds_kv8_tree_decode: the same for a tree of drafts: the next_n tokens of request
 * r are nodes, node i at position lens[r] - next_n + i of the cache. Node j sees
 * every position before lens[r] - next_n, and node i where bit i of masks[r, j]
 * is set (its ancestors and itself, in a tree; any set is taken, also one with no
 * bit). Positions below 0 do not exist, those past the table are not seen; bits
 * from next_n on are ignored.
 *
 *  masks        uint64 [num_requests, next_n], 8-byte aligned.
 *
 * All else as for ds_kv8_decode, but bt_stride is at most 2^20, and the workspace
 * has ds_kv8_tree_decode_workspace_size() bytes. Trees of up to 80 rows (next_n *
 * num_heads / num_kv_heads) are computed as by ds_kv8_decode, and with masks of a
 * chain (bit i set for i <= j) the results are then the same, bit for bit; larger
 * ones by tiles of 256 rows as in ds_kv8_prefill (q as precise as there), over spans
 * of the context that follow from the request's length alone.
 */
int ds_kv8_tree_decode(const void* q, int64_t q_stride, const uint64_t* masks,
                       const void* kv_pages, const float* kv_scales, int64_t num_pages,
                       const int32_t* block_table, int64_t bt_stride, const int32_t* lens,
                       int64_t num_requests, int next_n, int num_heads, int num_kv_heads,
                       int head_dim, float scale, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, int32_t* err_flag, void* stream);

/* Workspace bytes of ds_kv8_tree_decode (0 for an unsupported shape): up to 8
 * spans for each row of q, or as for ds_kv8_decode. */
size_t ds_kv8_tree_decode_workspace_size(int64_t num_requests, int next_n, int num_heads,
                                         int num_kv_heads, int head_dim, int64_t bt_stride);

/*
 * ds_kv8_prefill: the same attention for ragged prompts (or prompt chunks):
 * token i of a request with n tokens sees the first
 * clamp(lens[r] - n + 1 + i, 0, 64 * bt_stride) positions (causal). Rows of
 * out and lse that belong to no request are left as they are. Arguments as
 * for ds_kv8_decode; q, out and lse are indexed by token. The workspace has
 * ds_kv8_prefill_workspace_size() bytes, 256-byte aligned; its contents need
 * no initialisation. num_tokens * num_heads / num_kv_heads is below 2^31 - 256
 * and bt_stride at most 2^20 (a request's context is walked in order, and waits
 * have a limit). An element of q below 2^-28 of its head's largest is taken
 * with an error of up to 2^-39 of that one.
 *
 * A token's outputs depend on its own request alone, bit for bit, and not on
 * how the request's tokens are spread over calls.
 */
int ds_kv8_prefill(const void* q, int64_t q_stride, int64_t num_tokens,
                   const int32_t* token_starts, int64_t num_requests, const void* kv_pages,
                   const float* kv_scales, int64_t num_pages, const int32_t* block_table,
                   int64_t bt_stride, const int32_t* lens, int num_heads, int num_kv_heads,
                   int head_dim, float scale, void* out, float* lse, void* workspace,
                   size_t workspace_bytes, int32_t* err_flag, void* stream);

/* Workspace bytes of ds_kv8_prefill. */
size_t ds_kv8_prefill_workspace_size(int64_t num_tokens, int64_t num_requests, int num_heads,
                                     int num_kv_heads, int head_dim);

/*
 * ds_qk_norm_rope: norms of queries and keys per head and the rotation by
 * position, in one pass, in front of ds_kv8_append and the attention (and, with
 * 576 dims, of ds_kv_cache_write and the sparse attention).
 *
 * A head's row x of head_dim values becomes
 *   y_d = x_d * w_d / sqrt(mean over d < norm_dim of x_d^2 + eps), d < norm_dim,
 *   y_d = x_d behind (and everywhere on a side without weights),
 * and then the rot_dim values from rot_start on are turned in pairs (u, v) by
 * a_i = position * inv_freq_i: (u cos a_i - v sin a_i, v cos a_i + u sin a_i).
 * Pair i is (i, i + rot_dim / 2), or (2 i, 2 i + 1) with interleaved != 0. All
 * in float32 (squares of values above 2^63 overflow there), rounded to bfloat16
 * once; the angle is exact to 2^-22 turns at any position, for frequencies up to
 * 1024 in magnitude.
 *
 *  q, k         bfloat16, row t at q + t * q_stride (k + t * k_stride)
 *               elements, [heads, head_dim] contiguous; 16-byte aligned, strides
 *               multiples of 8 and at least heads * head_dim. k may be NULL with
 *               num_k_heads = 0.
 *  q_weight,    bfloat16 [norm_dim], 16-byte aligned, or NULL: no norm on that
 *  k_weight     side.
 *  positions    int32 [num_tokens], any value (a negative one turns the other
 *               way); inv_freq float32 [rot_dim / 2]. Both unused with rot_dim 0.
 *  q_out,       as q and k, with strides of their own. Either may be its input
 *  k_out        with the same stride; other overlaps give unspecified results.
 *
 * head_dim is a multiple of 16 up to 1024, norm_dim one of 8 in [0, head_dim],
 * rot_dim one of 16, rot_start one of 8; at most 1024 heads a side and 2^24
 * tokens. A row's result depends on that row alone, bit for bit.
 */
int ds_qk_norm_rope(const void* q, int64_t q_stride, int num_q_heads, const void* q_weight,
                    const void* k, int64_t k_stride, int num_k_heads, const void* k_weight,
                    int64_t num_tokens, int head_dim, int norm_dim, float eps,
                    const int32_t* positions, const float* inv_freq, int rot_start, int rot_dim,
                    int interleaved, void* q_out, int64_t q_out_stride, void* k_out,
                    int64_t k_out_stride, void* stream);

/*
 * ds_kv8_accept: after the drafts of a tree were verified, the accepted ones
 * move to the places behind the positions that were there before them, in all
 * layers by one launch.
 *
 *  layers       array in HOST memory, read during the call: the caches that the
 *               block table indexes, all of num_pages pages, num_kv_heads and
 *               head_dim. At most DS_MAX_KV8_LAYERS, each listed once.
 *  lens         int32 [num_requests], the next_n drafts of each request included
 *               (draft i lies at position lens[r] - next_n + i). Not changed.
 *  accepted     int32 [num_requests, width], width <= next_n <= 64: the accepted
 *               drafts' numbers, ascending, -1 behind them. Drafts that are not
 *               listed are dropped.
 *  new_lens     int32 [num_requests]: lens[r] - next_n + the number accepted. Not
 *               lens itself: hand it to ds_pages_shrink, which gives the pages
 *               behind back and sets the length.
 *  err_flag     optional: DS_DEVERR_IDX for a list that is not ascending, holds a
 *               number past next_n or one behind a -1; DS_DEVERR_LEN for a
 *               length in (0, next_n) or above 64 * bt_stride; DS_DEVERR_PAGE
 *               for a page outside the pool. Such a request stays as it is, its
 *               new length is its length. So does one of length <= 0, without
 *               an error.
 *
 * Scales: a page that gets positions has the largest scale of the pages that its
 * positions come from (itself among them where it keeps any); a code whose page
 * had a smaller one becomes E4M3(code * (old / scale)) as in ds_kv8_append, and
 * all others are copied as they are. Slots behind the new length keep their bytes.
 * The pages that hold the drafts belong to one request each (as ds_kv8_append
 * asks); others are not written.
 */
#define DS_MAX_KV8_LAYERS 128
typedef struct {
  void* kv_pages;
  float* kv_scales;
} ds_kv8_layer;

int ds_kv8_accept(const ds_kv8_layer* layers, int num_layers, int64_t num_pages,
                  const int32_t* block_table, int64_t bt_stride, const int32_t* lens,
                  int64_t num_requests, int num_kv_heads, int head_dim, int next_n,
                  const int32_t* accepted, int width, int32_t* new_lens, int32_t* err_flag,
                  void* stream);

/*
 * ds_kv8_mass: adds up the attention weight that cached positions get from new
 * tokens, for ds_kv8_evict. With the lse that ds_kv8_prefill, ds_kv8_decode or
 * ds_kv8_tree_decode gave for the same q and cache,
 *   mass[r, g, p] += sum over request r's tokens that see p (as in
 *   ds_kv8_prefill) and the heads h of kv head g of exp(scale * q . k_p - lse).
 * The positions of the call's own tokens, the last n of each request, start at
 * 0: they are set, whatever mass held there, and a fresh page needs no clearing.
 *
 *  q, token_starts, kv_pages, kv_scales, block_table, lens, scale   as for
 *               ds_kv8_prefill (decode: one token a request).
 *  lse          float32 [num_tokens, num_heads]; -inf: the row adds nothing, whatever
 *               its q holds (a padding token).
 *  mass         float32 [num_requests, num_kv_heads, mass_stride], mass_stride at
 *               least 64 * bt_stride. Rows of requests without tokens and
 *               entries at and past lens[r] keep their values. A fork's row is a
 *               copy that the caller makes.
 *  err_flag     optional: DS_DEVERR_PAGE for a page outside the pool: its
 *               positions get nothing (0 where they are the call's own).
 *
 * Scores are products of bfloat16 q and the codes with fp32 sums (about 2^-20 of
 * the largest partial sum), exponentials and sums are fp32. Up to 24 rows a kv head
 * (tokens times heads of the group) take q as three E4M3 pieces: exact down to 2^-19
 * of the row's largest |q|, and below that off by at most 2^-27 of it. A NaN key makes its
 * own position NaN where a row sees it, a non-finite q or a NaN lse the positions that the
 * row sees (rows of lse -inf aside).
 * num_tokens * num_heads / num_kv_heads is below 2^31 - 256 and bt_stride at most
 * 2^20. A request's mass depends on that request alone, bit for bit; it does
 * depend, in the last bits, on how its tokens are spread over calls. Needs no
 * workspace.
 */
int ds_kv8_mass(const void* q, int64_t q_stride, const float* lse, int64_t num_tokens,
                const int32_t* token_starts, int64_t num_requests, const void* kv_pages,
                const float* kv_scales, int64_t num_pages, const int32_t* block_table,
                int64_t bt_stride, const int32_t* lens, int num_heads, int num_kv_heads,
                int head_dim, float scale, float* mass, int64_t mass_stride, int32_t* err_flag,
                void* stream);

/*
 * ds_kv8_evict: holds every request of one layer's cache to `budget` positions.
 * Each kv head of a request with more keeps its first `first` positions, its
 * last `recent` ones, and of those between the budget - first - recent with the
 * most mass (equal mass: the lower position; NaN below everything), in their
 * order: they move to positions 0 .. budget - 1, codes, scales and mass alike.
 * Heads keep positions of their own; what a head's position stands for is the
 * caller's affair (keys hold their rotation already).
 *
 *  mass         float32 [num_requests, num_kv_heads, mass_stride], 16-byte
 *               aligned, mass_stride a multiple of 4 up to 2^28: the attention
 *               weight that each position got (ds_kv8_mass). Entries from budget
 *               on keep their values.
 *  budget       >= first + recent; budget - first - recent at most 16384.
 *  refcounts    optional int32 [num_pages]: a request whose first
 *               ceil(budget / 64) pages, which are rewritten, include one with a
 *               count above 1 stays as it is and sets DS_DEVERR_SHARED. Without
 *               it the caller answers for that.
 *  new_lens     int32 [num_requests]: the length afterwards. lens is not changed:
 *               it is the same for all layers, and ds_pages_shrink sets it once
 *               they are done.
 *  workspace    >= ds_kv8_evict_workspace_size() bytes, 256-byte aligned, no
 *               initialisation. Concurrent calls need separate ones.
 *  err_flag     optional: DS_DEVERR_LEN for a length above 64 * bt_stride or
 *               mass_stride, DS_DEVERR_PAGE for a page outside the pool; such a
 *               request stays as it is.
 *
 * Scales as for ds_kv8_accept: over many calls a page's scale tends to the largest that
 * its head had, and a value is off by one rounding and, in E4M3's subnormal range, half a
 * step of each scale it went through (with powers of two together less than 2^-9 of the
 * present scale). All positions behind the first dropped one move, also where few are
 * dropped. num_requests * num_kv_heads is at most 2^26. A request's result depends on that
 * request alone, bit for bit.
 */
int ds_kv8_evict(float* mass, int64_t mass_stride, int budget, int first, int recent,
                 void* kv_pages, float* kv_scales, int64_t num_pages, const int32_t* refcounts,
                 const int32_t* block_table, int64_t bt_stride, const int32_t* lens,
                 int64_t num_requests, int num_kv_heads, int head_dim, int32_t* new_lens,
                 void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream);

/* Workspace bytes of ds_kv8_evict (0 for an unsupported shape). */
size_t ds_kv8_evict_workspace_size(int64_t num_requests, int num_kv_heads, int64_t mass_stride,
                                   int budget, int first, int recent);

/*
 * Pages of a paged cache: who holds them, and moving them.
 *
 * The state is three device arrays of the caller:
 *  refcounts    int32 [num_pages]: how many block-table entries hold the
 *               page; a page is free when its count is not positive.
 *  block_table  int32 [num_rows, bt_stride]: row r holds its first
 *               ceil(lens[r] / 64) entries (lens clamped to
 *               [0, 64 * bt_stride]); the rest holds nothing.
 *  lens         int32 [num_rows].
 * Lengths are lowered by ds_pages_shrink. A caller that lowers one itself stays
 * within the row's last page: entries behind ceil(lens[r] / 64) count as empty,
 * so that their pages would be lost. Either way a page that ds_pages_fork shares
 * must not become one that is appended to.
 * Pages are handed out lowest number first, in the order of the call's list,
 * so the state after a call follows from the state before it.
 *
 * The caches that the pages index (any number of layers, codes, scales,
 * latent rows, indexer keys) are given as pools, an array in HOST memory that
 * is read during the call: pool i holds num_pages pages of page_bytes bytes
 * each, back to back, from data (4-byte aligned; page_bytes a multiple of 4).
 * At most DS_MAX_POOLS pools, 2^22 pages and 2^24 rows; lists of at most 65535
 * entries; the pools' page_bytes sum to at most 2^28.
 *
 * Common to these calls: a negative list entry is padding; a row outside
 * [0, num_rows) is skipped and sets DS_DEVERR_ROWREQ; workspaces have
 * ds_pages_workspace_size() bytes, 256-byte aligned, and need no
 * initialisation. Concurrent calls need separate workspaces, and calls on the
 * same state need an order between them.
 */
#define DS_MAX_POOLS 128
typedef struct {
  void* data;
  int64_t page_bytes;
} ds_page_pool;

/* Workspace bytes of the page calls for a pool and a list of n entries. */
size_t ds_pages_workspace_size(int64_t num_pages, int64_t n);

/*
 * Page src[i] to page dst[i] in every pool, i < n (int32 lists). An i with a
 * negative src or dst is padding; a page at or past num_pages sets
 * DS_DEVERR_PAGE and copies nothing. No dst may repeat or be a src of the
 * same call (the copies run at once).
 */
int ds_pages_copy(const ds_page_pool* pools, int num_pools, int64_t num_pages, const int32_t* src,
                  const int32_t* dst, int64_t n, int32_t* err_flag, void* stream);

/*
 * Gives up everything the listed rows hold: each held page loses one count,
 * the entries become -1 and the length 0. A row that is listed twice is freed
 * once. A held entry of -1 counts for nothing; one outside the pool, or of a
 * page whose count is not positive, sets DS_DEVERR_PAGE and changes no count.
 */
int ds_pages_free(int32_t* refcounts, int64_t num_pages, int32_t* block_table, int64_t bt_stride,
                  int32_t* lens, int64_t num_rows, const int32_t* rows, int64_t n,
                  int32_t* err_flag, void* stream);

/*
 * Makes row children[i] a copy of row parents[i]: full pages are shared (one
 * count more each), a partly filled last page is copied in every pool to a
 * free page of its own (so both rows may append), the length is taken over.
 * Parents are read as they were before the call. A child has to be empty
 * (length <= 0) and listed once: otherwise the later entry is skipped and
 * DS_DEVERR_ROWREQ set. The i-th copied page takes the i-th free page; a
 * child for which none is left stays empty and sets DS_DEVERR_NOPAGE. A page
 * outside the pool is taken over as it is, also where it is a partly filled
 * last one, and sets DS_DEVERR_PAGE.
 */
int ds_pages_fork(const ds_page_pool* pools, int num_pools, int32_t* refcounts, int64_t num_pages,
                  int32_t* block_table, int64_t bt_stride, int32_t* lens, int64_t num_rows,
                  const int32_t* parents, const int32_t* children, int64_t n, void* workspace,
                  size_t workspace_bytes, int32_t* err_flag, void* stream);

/*
 * Grows row rows[i] to new_lens[i] positions: the entries it holds more get
 * free pages (count 1). A new length below the present one or above
 * 64 * bt_stride sets DS_DEVERR_LEN, a row listed before sets
 * DS_DEVERR_ROWREQ; both are skipped. Entry i takes the free pages after
 * those that the entries before it ask for; where that passes the last free
 * page the row stays as it is and DS_DEVERR_NOPAGE is set.
 */
int ds_pages_extend(int32_t* refcounts, int64_t num_pages, int32_t* block_table,
                    int64_t bt_stride, int32_t* lens, int64_t num_rows, const int32_t* rows,
                    const int32_t* new_lens, int64_t n, void* workspace, size_t workspace_bytes,
                    int32_t* err_flag, void* stream);

/*
 * Lowers row rows[i] to new_lens[i] positions: the pages that it no longer needs
 * lose one count and their entries become -1. A new length above the present
 * one or below 0 sets DS_DEVERR_LEN and a row listed before DS_DEVERR_ROWREQ;
 * both are skipped. A new length equal to lens[r] changes nothing, whatever it
 * is. Entries that are no pages of the row's count as for ds_pages_free.
 */
int ds_pages_shrink(int32_t* refcounts, int64_t num_pages, int32_t* block_table,
                    int64_t bt_stride, int32_t* lens, int64_t num_rows, const int32_t* rows,
                    const int32_t* new_lens, int64_t n, int32_t* err_flag, void* stream);

/*
 * Moves the live pages to the front of the pool: with num_live pages live,
 * the i-th live page at or past num_live goes to the i-th free page below it,
 * in every pool, and the tables follow. Results go to block_table_out
 * (entries that no row holds are copied as they are), refcounts_out and
 * num_live_out (int32); block_table_out may be block_table and refcounts_out
 * may be refcounts. The pools change in place; pages at and past num_live
 * keep their bytes. A held entry outside the pool or of a free page stays and
 * sets DS_DEVERR_PAGE. Workspace: ds_pages_workspace_size(num_pages, 0).
 */
int ds_pages_compact(const ds_page_pool* pools, int num_pools, const int32_t* refcounts,
                     int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                     const int32_t* lens, int64_t num_rows, int32_t* refcounts_out,
                     int32_t* block_table_out, int32_t* num_live_out, void* workspace,
                     size_t workspace_bytes, int32_t* err_flag, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DS_SPARSE_MLA_H */
