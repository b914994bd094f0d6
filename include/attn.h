/*
 * attn.h -- C ABI of libattn.so: batched GQA attention with a per-head sink
 * logit over a paged KV cache, for one NVIDIA GB300 GPU (sm_103a).
 *
 * What is computed.  "GPT-OSS on day 0" (Perplexity), section "Sink
 * Attention": every query head h owns one learned sink logit that takes part
 * in the softmax.  It enters the denominator only (its value vector is zero)
 * and is not multiplied by sm_scale:
 *
 *   out[i,h] = sum_j exp(s_ij - m) v_j / (sum_j exp(s_ij - m) + exp(sink_h - m))
 *   s_ij     = sm_scale * q[i,h] . k_j            (k, v of KV head h / (Hq/Hkv))
 *   lse[i,h] = m + ln(sum_j exp(s_ij - m) + exp(sink_h - m))   (natural log)
 *
 * The same section describes the kernels as parallel over heads and over the
 * KV length, with the softmax computed online (running max and scale) and
 * the sink placed in the first part of a KV split only; this library does
 * exactly that (split-KV decode with a log-sum-exp merge).
 *
 * Request model, "Disaggregated prefill and decode" (Perplexity), section
 * "Prefill vs decode performance": request b forwards qo_len_b query tokens
 * and reads kv_len_b tokens from the KV cache; decode has qo_len = 1.  Query
 * i of request b sits at absolute position kv_len_b - qo_len_b + i, so with
 * causal masking it sees keys j <= kv_len_b - qo_len_b + i.
 *
 * KV cache layout, "Hosting Qwen on Blackwell" (Perplexity), section
 * "Deploying on GB200 NVL72", and "Disaggregated prefill and decode", section
 * "Sharded KV transfer": HND pages, heads outer and each page's tokens
 * contiguous.  Concretely one pool, bf16, row-major:
 *
 *   kv_cache[num_pages][2][Hkv][page_size][head_dim]      ([.][0] = K, [.][1] = V)
 *
 * Tensors (all caller-owned device memory, row-major, contiguous):
 *   q, out   bf16  [total_qo_rows][Hq][head_dim]   total_qo_rows = qo_indptr[batch]
 *   lse      fp32  [total_qo_rows][Hq]             natural log; may be NULL
 *   sinks    fp32  [Hq]                            may be NULL (no sink, i.e. -inf)
 *
 * Threading and streams: every launch is asynchronous on the caller's
 * cudaStream_t, passed as void* (NULL = legacy default stream).  A plan may be
 * used from one host thread at a time.  Launches that share a plan's
 * workspace must not overlap on the GPU (issue them on one stream).
 *
 * Errors: functions return attn_status and never abort or throw.  Argument
 * and shape checks happen on the host before anything is launched.  Kernels
 * never trap: a page id outside the pool or a wait that runs out is recorded
 * in a device error word of the plan's workspace (read it with
 * attn_plan_device_error) and the offending load is skipped.
 */
#ifndef ATTN_H
#define ATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define ATTN_API __attribute__((visibility("default")))
#else
#define ATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1,          /* malformed pointer, size or index array */
    ATTN_ERR_UNSUPPORTED = 2,          /* well-formed but outside the supported shapes */
    ATTN_ERR_WORKSPACE_TOO_SMALL = 3,  /* bound workspace smaller than required */
    ATTN_ERR_CUDA = 4,                 /* a CUDA runtime/driver call failed */
    ATTN_ERR_NOT_BOUND = 5,            /* launch before attn_plan_bind_workspace */
    ATTN_ERR_DEVICE = 6                /* a kernel recorded an error (see device error bits) */
} attn_status;

/* Bits of the device error word (attn_plan_device_error). */
#define ATTN_DEVICE_ERR_PAGE_ID 1      /* page id outside [0, num_pages_in_pool) */
#define ATTN_DEVICE_ERR_TIMEOUT 2      /* a bounded wait inside a kernel ran out */
#define ATTN_DEVICE_ERR_PLAN 4         /* attn_decode_graph: malformed request metadata or
                                          work beyond the graph plan's capacity;
                                          attn_pages_fork: malformed parents, or more
                                          entries than fit */
#define ATTN_DEVICE_ERR_PAGES 8        /* attn_pages_*: no free page was left, or a page was
                                          given up that nothing held */

/* Opaque plan; owned by the library, freed with attn_plan_destroy. */
typedef struct attn_plan_s* attn_plan_t;

/* Summary of a plan (host-side copy, for callers and tests). */
typedef struct {
    int32_t batch;
    int32_t total_qo_rows;
    int32_t num_decode_requests;     /* requests with qo_len == 1 */
    int32_t num_prefill_requests;    /* requests with qo_len > 1 */
    int32_t num_decode_units;        /* CTAs of one attn_decode launch */
    int32_t num_decode_groups_split; /* (request, kv head, head slice) groups split over >1 chunk */
    int32_t num_decode_partials;     /* partial states held in the workspace */
    int32_t decode_chunk_blocks;     /* target split-KV chunk, in 16-token blocks */
    int32_t num_prefill_items;       /* CTAs of one attn_prefill launch */
    int32_t num_sms;                 /* SM count the plan was balanced for */
    int64_t decode_kv_tokens;        /* sum of kv_len over decode requests */
    int64_t prefill_pairs;           /* visible (query, key) pairs over prefill rows, per query head */
    size_t workspace_bytes;
} attn_plan_info;

/*
 * attn_plan -- build the work list of one batch (host only; launches nothing).
 *
 * The split of the work over heads and over the KV length follows "GPT-OSS on
 * day 0", section "Sink Attention"; the qo_len / kv_len request model follows
 * "Disaggregated prefill and decode", section "Prefill vs decode performance".
 * Requests with qo_len == 1 are decode requests (attn_decode), requests with
 * qo_len > 1 are prefill requests (attn_prefill); qo_len == 0 contributes no
 * rows.  Long decode sequences are split into chunks of whole 16-token blocks
 * so that the number of CTAs fills num_sms SMs; chunk 0 of each split carries
 * the sink and the chunks are merged by log-sum-exp inside the same launch.
 *
 *   qo_indptr      host int32 [batch+1]; qo_indptr[0] = 0, non-decreasing
 *   kv_indptr      host int32 [batch+1]; CSR offsets of each request's pages in
 *                  page_table; kv_indptr[0] = 0, non-decreasing
 *   page_table     DEVICE int32 [kv_indptr[batch]]; page ids into the pool.
 *                  Borrowed: it must stay valid, unchanged, for every launch
 *                  made with this plan.  Not read by attn_plan.
 *   last_page_len  host int32 [batch]; tokens used in the request's last page,
 *                  1..page_size (ignored for a request with no pages);
 *                  kv_len = (n_pages - 1) * page_size + last_page_len
 *   batch >= 0; num_qo_heads % num_kv_heads == 0 (query head h reads KV head
 *   h / (num_qo_heads / num_kv_heads)); head_dim in {64, 128}; page_size in
 *   {16, 32, 64, 128}; qo_len <= kv_len for every request; causal in {0, 1};
 *   sm_scale finite; num_pages_in_pool > 0 when any request has pages;
 *   num_sms > 0, or 0 to query the current CUDA device.
 *
 * On success *plan_out owns host memory only and *workspace_bytes_out is the
 * size of the device workspace the plan needs.  Nothing is written on error.
 */
ATTN_API attn_status attn_plan(const int32_t* qo_indptr, const int32_t* kv_indptr,
                      const int32_t* page_table, const int32_t* last_page_len,
                      int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
                      int32_t head_dim, int32_t page_size, int32_t causal, float sm_scale,
                      int32_t num_pages_in_pool, int32_t num_sms, attn_plan_t* plan_out,
                      size_t* workspace_bytes_out);

/*
 * attn_plan_bind_workspace -- attach caller-owned device memory to the plan
 * and upload the work list into it (asynchronous copy on `stream`; the host
 * copy stays valid).  `workspace` must be 256-byte aligned and hold at least
 * the plan's workspace_bytes; it is used by every later launch of the plan
 * and must outlive them.  Clears the device error word and the split-merge
 * counters.  May be called again (e.g. with other memory).
 */
ATTN_API attn_status attn_plan_bind_workspace(attn_plan_t plan, void* workspace, size_t bytes,
                                     void* stream);

/*
 * attn_decode -- sink attention for the plan's decode rows (qo_len == 1):
 * one CTA per (request, KV head, head slice, KV chunk); the GQA group's query
 * heads share every K/V tile read from HBM.  Writes out and lse rows of
 * decode requests only.  Pointers as in the file comment.
 */
ATTN_API attn_status attn_decode(attn_plan_t plan, const void* q, const void* kv_cache,
                        const float* sinks, void* out, float* lse, void* stream);

/*
 * attn_prefill -- sink attention for the plan's prefill rows (qo_len > 1),
 * causal or not as planned: one CTA per (128-row query tile, pair of query
 * heads of one GQA group), QK^T and PV on the tensor cores.  Writes out and
 * lse rows of prefill requests only.  For a mixed batch call attn_prefill
 * and attn_decode with the same plan, in either order, on one stream.
 */
ATTN_API attn_status attn_prefill(attn_plan_t plan, const void* q, const void* kv_cache,
                         const float* sinks, void* out, float* lse, void* stream);

/*
 * attn_plan_ragged / attn_prefill_ragged -- the same sink attention over
 * contiguous, unpadded K and V with no KV cache, for embedding-style serving
 * ("Fast embeddings on GPUs" (Perplexity), section "ROSE": with no KV cache
 * the attention kernels take ragged inputs so that nothing is padded).
 *
 *   qo_indptr  host int32 [batch + 1]: request b's query rows
 *   kv_indptr  host int32 [batch + 1]: request b's rows of k and v (tokens,
 *              not pages); qo_len <= kv_len, queries aligned to the end of
 *              the keys for the causal mask as in attn_plan
 *   q, out     bf16 [qo_indptr[batch]][Hq][head_dim]
 *   k, v       bf16 [kv_indptr[batch]][Hkv][head_dim] (16-byte aligned)
 *   sinks, lse as in attn_prefill
 * Every request (qo_len = 1 included) runs on the tcgen05 prefill kernel; the
 * plan has no decode work (attn_decode on it does nothing) and cannot be used
 * with attn_prefill or attn_append_kv (ATTN_ERR_INVALID_ARG).  Workspace and
 * error word as for attn_plan.
 */
ATTN_API attn_status attn_plan_ragged(const int32_t* qo_indptr, const int32_t* kv_indptr, int32_t batch,
                                      int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                                      int32_t causal, float sm_scale, int32_t num_sms, attn_plan_t* plan_out,
                                      size_t* workspace_bytes_out);
ATTN_API attn_status attn_prefill_ragged(attn_plan_t plan, const void* q, const void* k, const void* v,
                                         const float* sinks, void* out, float* lse, void* stream);

/*
 * attn_plan_cross / attn_cross -- cross attention: the query rows of each sequence
 * (its decoder's) over all of an encoder's states, which have a length of their
 * own, longer or shorter than the rows; nothing is causal.  No source describes it:
 * an interface addition.  Rows that look at the same states belong to one
 * sequence: a prompt's tokens, the beams, samples or draft tokens of a step.  They
 * then share every read of K and V.
 *
 *   qo_indptr  host int32 [batch + 1]: sequence b's query rows, any number
 *   kv_start, kv_len  host int32 [batch]: sequence b's states are rows
 *              [kv_start, kv_start + kv_len) of k and v, 0 <= kv_start,
 *              kv_start + kv_len <= kv_rows.  So k and v may be packed, padded to
 *              one length, or a store from which sequences come and go; sequences
 *              may share rows.  Rows that no sequence has are not used (they may
 *              hold NaN).  kv_len = 0: out = 0, lse = the sink's (-inf without).
 *   q, out     bf16 [qo_indptr[batch]][Hq][head_dim];  sinks, lse as in attn_prefill
 *   k, v       bf16 [kv_rows][Hkv][head_dim], rows k_stride / v_stride elements apart
 *              (multiples of 8, at least Hkv * head_dim), 16-byte aligned: the two
 *              halves of a fused projection are taken as they are.  Not read, and
 *              may be NULL, where kv_rows = 0.
 *   head_dim in {64, 128}; num_qo_heads % num_kv_heads == 0; rows * Hq and kv_rows
 *   below 2^30 (else ATTN_ERR_UNSUPPORTED)
 * Workspace, binding and error word as for attn_plan (attn_plan_info: num_decode_units
 * counts the work of few rows, num_prefill_items that of many); every other launch
 * refuses such a plan (ATTN_ERR_INVALID_ARG).  attn_cross writes all rows of out and lse,
 * but for those of work that recorded ATTN_DEVICE_ERR_TIMEOUT and, until
 * attn_plan_device_error has read that, of all sequences whose keys are split.
 * The order of every sum is fixed.  Async on `stream`; capturable (after one
 * uncaptured call with these pointers has built the TMA descriptors).
 */
ATTN_API attn_status attn_plan_cross(const int32_t* qo_indptr, const int32_t* kv_start, const int32_t* kv_len,
                                     int32_t batch, int32_t kv_rows, int32_t num_qo_heads, int32_t num_kv_heads,
                                     int32_t head_dim, float sm_scale, int32_t num_sms, attn_plan_t* plan_out,
                                     size_t* workspace_bytes_out);
ATTN_API attn_status attn_cross(attn_plan_t plan, const void* q, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, const float* sinks, void* out, float* lse, void* stream);

/*
 * attn_merge_states -- combine two attention states over disjoint key sets
 * into the state over their union, by the log-sum-exp rule implied by the
 * split along the KV length in "GPT-OSS on day 0", section "Sink Attention"
 * (the pages do not print it):
 *   L = max(lse_a, lse_b);  w_x = exp(lse_x - L)
 *   v_out = (w_a v_a + w_b v_b) / (w_a + w_b);  lse_out = L + ln(w_a + w_b)
 * A state with lse = -inf (no keys, no sink) is the identity.  The sink must
 * be counted in exactly one of the two inputs.
 *
 *   va, vb, vout   bf16 [n_tokens][n_heads][head_dim]  (vout may alias va or vb)
 *   lsea, lseb     fp32 [n_tokens][n_heads], natural log
 *   lseout         fp32 [n_tokens][n_heads] or NULL
 *   head_dim a multiple of 4, at most 256.  Device pointers, async on stream.
 */
ATTN_API attn_status attn_merge_states(const void* va, const float* lsea, const void* vb,
                              const float* lseb, void* vout, float* lseout, int32_t n_tokens,
                              int32_t n_heads, int32_t head_dim, void* stream);

/*
 * attn_merge_states_f32 -- the same log-sum-exp merge for fp32 value states:
 * partial states kept unrounded (a KV sequence split across calls or
 * devices, the sink counted in one part only, as in "GPT-OSS on day 0",
 * section "Sink Attention") merge without rounding each part to bf16 first.
 *   va, vb         fp32 [n_tokens][n_heads][head_dim], 16-byte aligned
 *   lsea, lseb     fp32 [n_tokens][n_heads], natural log
 *   vout           fp32 (vout_bf16 = 0; 16-byte aligned, may alias va or vb)
 *                  or bf16 (vout_bf16 != 0; 8-byte aligned), [n_tokens][n_heads][head_dim]
 *   lseout         fp32 [n_tokens][n_heads] or NULL
 * head_dim a multiple of 4, at most 256.  Device pointers, async on stream;
 * ATTN_ERR_INVALID_ARG for bad sizes, NULL or misaligned pointers.
 */
ATTN_API attn_status attn_merge_states_f32(const float* va, const float* lsea, const float* vb,
                                           const float* lseb, void* vout, int32_t vout_bf16, float* lseout,
                                           int32_t n_tokens, int32_t n_heads, int32_t head_dim, void* stream);

/*
 * attn_decode_noalloc -- attn_decode for callers that cannot allocate device
 * memory when they run attention: an engine that reserves its whole memory
 * budget up front and forbids cudaMalloc while it serves (cudaMalloc may also
 * synchronise the device and so stall every other stream).  No source
 * describes such a call: this is an interface addition.
 *
 * Same arguments and results as attn_decode (host-planned paged plans; a
 * graph plan is refused with ATTN_ERR_INVALID_ARG), but the plan needs no
 * bound workspace: the work list, split-KV partial states, merge counters and
 * error word live in a static 16 MiB device array inside the library.  A GPU
 * holds that array from the moment the library's device code is loaded there
 * (with lazy module loading, the first use of it on that GPU) until the
 * process exits.  Plans that need more than that (their workspace_bytes without
 * the lists that only other calls read) are rejected with
 * ATTN_ERR_WORKSPACE_TOO_SMALL.  It allocates nothing (no cudaMalloc /
 * cudaFree): each call uploads the work list with cudaMemcpyAsync from the
 * plan's host memory (pageable, so the call returns once the copy has been
 * staged, which may wait for earlier work on `stream`) and zeroes the counters
 * and the error word with cudaMemsetAsync on `stream`, then launches the
 * decode kernel.  The results are bit-identical to attn_decode's on the same
 * plan and inputs.
 *
 * The first call on a device resolves the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture.  All calls share the one array and it keeps the
 * last call's contents, so calls that overlap on the GPU (other streams, other
 * host threads) race: serialise them.  Bad page ids are skipped rather than
 * read and, like bounded-wait timeouts, set bits of the array's error word:
 * read it with attn_decode_noalloc_device_error.
 */
ATTN_API attn_status attn_decode_noalloc(attn_plan_t plan, const void* q, const void* kv_cache,
                                         const float* sinks, void* out, float* lse, void* stream);

/*
 * attn_decode_noalloc_device_error -- wait for `stream`, then read and clear
 * the device error word (ATTN_DEVICE_ERR_* bits) that attn_decode_noalloc
 * calls with this plan's layout left in the current device's static array,
 * into *code.  Returns ATTN_ERR_DEVICE if any bit was set, ATTN_ERR_INVALID_ARG
 * for a NULL argument or a graph plan.  The array is shared by every call, so
 * read it before another call on the device may overwrite it.
 */
ATTN_API attn_status attn_decode_noalloc_device_error(attn_plan_t plan, int32_t* code, void* stream);

/*
 * attn_graph_plan / attn_decode_graph -- decode that can be captured in a CUDA
 * graph and replayed for new batches.  The split-KV plan depends on the
 * requests' lengths, so host planning would freeze it at capture; here the
 * work list is built on the device from device-resident metadata, with the
 * same rule as attn_plan (for plans of up to 128 requests by every CTA of the
 * persistent decode grid itself, else by a planner kernel launched first),
 * and a fixed grid of persistent decode CTAs takes the units from a device
 * queue ("Fast embeddings on GPUs"
 * (Perplexity), section "Managing CUDA graphs": kernels that configure their
 * launches from dynamic host inputs prevent full CUDA graphs; the page's fix
 * is to change those kernels so they can be captured).
 *
 * attn_graph_plan sizes a plan once, for at most `max_batch` decode requests
 * whose KV lengths sum to at most `max_kv_tokens` (0: num_pages_in_pool *
 * page_size); bind a workspace with attn_plan_bind_workspace as usual.  The
 * page table pointer is fixed; its contents may change between replays.
 *
 * attn_decode_graph reads, on the device and at run time:
 *   batch          int32 scalar: B <= max_batch decode requests (query row b =
 *                  request b; q / out are [max_batch][Hq][head_dim], lse
 *                  [max_batch][Hq]; rows >= B are not touched)
 *   kv_indptr      int32 [B + 1] page CSR into page_table, kv_indptr[0] = 0
 *   last_page_len  int32 [B], in [1, page_size]
 * No host synchronisation, copy or allocation happens inside the call, so it
 * can be captured (after one uncaptured call has built the TMA descriptor for
 * this kv_cache pointer).  A request with a malformed entry, or a batch beyond
 * the plan's capacity, sets ATTN_DEVICE_ERR_PLAN; such requests (or, past
 * the capacity, the whole step) produce no output.  attn_decode, attn_prefill
 * and attn_append_kv reject graph plans.
 */
ATTN_API attn_status attn_graph_plan(int32_t max_batch, int32_t num_qo_heads, int32_t num_kv_heads,
                                     int32_t head_dim, int32_t page_size, float sm_scale, int32_t num_pages_in_pool,
                                     int64_t max_kv_tokens, const int32_t* page_table, int32_t num_sms,
                                     attn_plan_t* plan_out, size_t* workspace_bytes_out);
ATTN_API attn_status attn_decode_graph(attn_plan_t plan, const int32_t* kv_indptr, const int32_t* last_page_len,
                                       const int32_t* batch, const void* q, const void* kv_cache, const float* sinks,
                                       void* out, float* lse, void* stream);
/*
 * Copy the work list that the last attn_decode_graph built on the device into
 * host memory (12 int32 per unit, as attn_plan_get_decode_units), after
 * synchronising `stream`; *n_units receives the unit count.  For tests and
 * inspection.
 */
ATTN_API attn_status attn_graph_plan_read_units(attn_plan_t plan, int32_t* units, int64_t capacity,
                                                int64_t* n_units, void* stream);

/*
 * attn_append_kv -- write the step's new K and V rows into the paged cache,
 * the step that runs before attention ("Disaggregated prefill and decode"
 * (Perplexity), section "KV Messenger": the model appends a layer's new tokens
 * to its KV cache, and the entries are valid after that append and before
 * attention).  Every query row of the plan is one new token: row i of request
 * b is cache position t = kv_len - qo_len + i (kv_len as given to attn_plan,
 * i.e. counting the new tokens), stored at page page_table[kv_indptr[b] + t/P],
 * row t % P, so the pages must already be allocated in the plan's page table.
 *
 *   k_new, v_new  bf16 [total_qo_rows][Hkv][head_dim], device, 16-byte aligned
 *   kv_cache      bf16 [num_pages][2][Hkv][page_size][head_dim] HND pool,
 *                 device, 16-byte aligned; only the new tokens' rows change
 * Bit-exact copy.  Needs a bound workspace.  Page ids outside [0, num_pages)
 * set ATTN_DEVICE_ERR_PAGE_ID and that row is skipped.  Async on `stream`.
 */
ATTN_API attn_status attn_append_kv(attn_plan_t plan, const void* k_new, const void* v_new, void* kv_cache,
                                    void* stream);

/*
 * attn_pack_kv_heads / attn_unpack_kv_heads -- move a head slice of HND pages
 * to or from one contiguous buffer, the local half of a head-sharded KV
 * transfer ("Disaggregated prefill and decode", section "Sharded KV transfer":
 * pages are split or rebuilt from head slices when sender and receiver shard
 * the cache over attention heads differently, and the HND layout keeps a
 * page's head slice contiguous).  The network part is not in this library.
 *
 *   kv_cache      bf16 [num_pages][2][num_kv_heads][page_size][head_dim], device
 *   page_ids      int32 [n_pages], device: pages to move, in buffer order
 *   buf           bf16 [n_pages][2][n_heads][page_size][head_dim], device
 *   heads         [head_begin, head_begin + n_heads) of num_kv_heads
 *   device_error  optional device int32; ATTN_DEVICE_ERR_PAGE_ID is OR-ed in
 *                 when a page id lies outside [0, num_pages) (that page is
 *                 skipped).  NULL: such pages are skipped silently.
 * Pack reads the pool and writes buf; unpack reads buf and writes only the
 * slice's bytes of the listed pages.  head_dim a multiple of 8; kv_cache and
 * buf 16-byte aligned.  Bit-exact copies.  Async on `stream`.
 */
ATTN_API attn_status attn_pack_kv_heads(const void* kv_cache, int64_t num_pages, int32_t num_kv_heads,
                                        int32_t page_size, int32_t head_dim, const int32_t* page_ids,
                                        int64_t n_pages, int32_t head_begin, int32_t n_heads, void* buf,
                                        int32_t* device_error, void* stream);
ATTN_API attn_status attn_unpack_kv_heads(const void* buf, int64_t num_pages, int32_t num_kv_heads,
                                          int32_t page_size, int32_t head_dim, const int32_t* page_ids,
                                          int64_t n_pages, int32_t head_begin, int32_t n_heads, void* kv_cache,
                                          int32_t* device_error, void* stream);

/*
 * Rotary positions -- the turn by position that q and k take before attention,
 * with one axis (text) or several (time, height and width of images and video).
 * No source describes it: attn_rope and attn_append_kv_rope are interface
 * additions.  Pair p of a row's first rot_dim dims turns by
 *
 *   theta = positions[axis[p]][row] * inv_freq[p]
 *   (x, y) -> scale * (x cos theta - y sin theta,  x sin theta + y cos theta)
 *
 * and the other dims are copied.  The angle is taken modulo a turn in 64-bit
 * integers, within 2^-31 of a turn at every int32 position, and then rounded to fp32
 * half turns, by up to 2^-26 of a turn; its cosine and sine and the products are
 * fp32, rounded to bf16 once.
 *
 *   rot_dim      a multiple of 16, 16 .. head_dim (else ATTN_ERR_UNSUPPORTED)
 *   interleaved  0: pair p is dims (p, p + rot_dim / 2);  1: dims (2p, 2p + 1)
 *   n_axes       1 .. 8
 *   inv_freq     host fp32 [rot_dim / 2], finite, |inv_freq| < 2^20 (radians per
 *                position)
 *   axis         host int32 [rot_dim / 2] in [0, n_axes), or NULL (all 0)
 *   scale        finite
 */
typedef struct {
    int32_t rot_dim;
    int32_t interleaved;
    int32_t n_axes;
    float scale;
    const float* inv_freq;
    const int32_t* axis;
} attn_rope_spec;

/*
 * attn_rope -- turns the rows of q and of k (either may be absent: NULL with 0
 * heads), for attention without a cache, before attn_append_kv4, or, with
 * inverse = 1 (theta negated: the transposed turn), for their gradients.
 *
 *   positions   device int32 [n_axes][rows]
 *   q, k        bf16 rows of heads, device: element (row, h, d) at
 *               row * stride + h * head_dim + d; strides in elements, multiples of
 *               8, at least heads * head_dim; 16-byte aligned.  So slices of a
 *               fused projection are taken as they are.
 *   q_out, k_out  likewise; may be the input itself with the input's stride (in
 *               place), else must not overlap it
 *   head_dim 64 or 128, rows below 2^31, at most 65,536 heads in all (else
 *   ATTN_ERR_UNSUPPORTED)
 * Async on `stream`.
 *
 * attn_append_kv_rope -- attn_rope of a step's q and k and attn_append_kv of the
 * turned k and of v in one pass: q_out gets the turned q, and the plan's cache
 * positions the turned k (bit-identical to attn_rope followed by attn_append_kv).
 * Row i is the plan's query row i; its positions are the caller's, not the cache's.
 *
 *   q, k_new, v_new  as q and k above, with the plan's heads and head_dim
 *   q_out            bf16 [total_qo_rows][Hq][head_dim]; may be q where that is
 *                    contiguous
 *   kv_cache         as in attn_append_kv, as are bad page ids and plans
 */
ATTN_API attn_status attn_rope(const attn_rope_spec* rope, const int32_t* positions, int64_t rows, int32_t head_dim,
                               const void* q, int64_t q_stride, int32_t num_q_heads, void* q_out,
                               int64_t q_out_stride, const void* k, int64_t k_stride, int32_t num_k_heads,
                               void* k_out, int64_t k_out_stride, int32_t inverse, void* stream);
ATTN_API attn_status attn_append_kv_rope(attn_plan_t plan, const attn_rope_spec* rope, const int32_t* positions,
                                         const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                                         const void* v_new, int64_t v_stride, void* q_out, void* kv_cache,
                                         void* stream);

/*
 * Page management -- the cache's pages handed about on the device, in stream
 * order and without the host waiting (no source describes it: attn_pages_* are
 * interface additions).  The state is one count per page:
 *
 *   refs   device int32 [num_pages], 16-byte aligned: how many page-table entries
 *          hold page p; 0: free.  All zero at first.
 *
 * and the pools are whatever is stored by page (each layer's kv_cache or
 * kv4_cache, weights):
 *
 *   pools       host array of n_pools device pointers, 16-byte aligned; page p of
 *               pool k is the page_bytes[k] bytes (a multiple of 16) at
 *               pools[k] + p * page_bytes[k]
 *   device_error  device int32 or NULL (bits are OR-ed in; then dropped silently)
 *
 * Calls that change refs read what earlier ones left, so they are issued on one
 * stream.  Equal calls give equal tables and counts.
 *
 * attn_pages_alloc -- the n lowest free pages, in order, into page_ids (int32 [n],
 * device), held once.  Where fewer are free, the rest of page_ids is -1 and
 * ATTN_DEVICE_ERR_PAGES is set.
 *
 * attn_pages_free -- every listed page is held once less (a page listed twice,
 * twice).  Ids outside the pool (-1 among them) are skipped and set
 * ATTN_DEVICE_ERR_PAGE_ID; a page that nothing held stays at 0 and sets
 * ATTN_DEVICE_ERR_PAGES.
 *
 * attn_pages_copy -- page src[i] of every pool into page dst[i], bit for bit; the
 * dst are distinct and no dst is a src.  Pairs with an id outside the pool are
 * skipped and set ATTN_DEVICE_ERR_PAGE_ID.  refs are not looked at.
 *
 * attn_pages_fork -- children of requests: child c starts as the first kv_lens[p]
 * tokens of request p = parents[c] (several children may have one parent, which
 * goes on as it was).  Full pages are shared: the child's entry is the parent's,
 * held once more.  A last page that is not full, and will be written into, is
 * copied in every pool into a new page (the lowest free ones, in the children's
 * order), held once.  Parent and children may append from there on, but nothing may
 * write into a shared page.  attn_evict_kv does so in place (evict into new pages,
 * page_table_out, and free the old ones), and so does an append to a request that was
 * shortened below its fork.  attn_key_weights writes the weights of every cached key:
 * requests that share pages each need a weights buffer and a plan of their own.
 *   page_table [table_len], kv_indptr [batch + 1], kv_lens [batch], parents [n]   device int32;
 *                 request p's pages are page_table[kv_indptr[p] ..] as in attn_plan
 *   page_table_out, indptr_out   device int32 [out_len], [n + 1], outputs: child c's
 *                 ceil(kv_lens / page_size) entries from indptr_out[c] on.  Entries
 *                 past the last are left as they were.
 *   scratch       device int32 [attn_pages_scratch(n)], for this call alone
 * A child whose parent is not in [0, batch), or whose kv_lens its entries (within
 * table_len) do not hold, gets no pages (ATTN_DEVICE_ERR_PLAN).  Where no free page is left its entry
 * is -1 (ATTN_DEVICE_ERR_PAGES); where the parent's entry is outside the pool it is
 * -1, or for a last page that is not full a new page that nothing is copied into
 * (ATTN_DEVICE_ERR_PAGE_ID).  Children of more than out_len entries in all are
 * refused as a whole: indptr_out is zero, ATTN_DEVICE_ERR_PLAN, nothing else changes.
 *
 * attn_pages_compact -- with U pages held, moves those from U on into the free ones
 * below U, the highest into the lowest, in every pool; refs move with them and
 * then are positive exactly below U.
 *   remap         device int32 [num_pages], output: the new id of every page, -1 for
 *                 pages that were free
 *   page_table    device int32 [n_entries], changed to the new ids (other tables: look
 *                 ids up in remap).  Ids outside the pool stay and set
 *                 ATTN_DEVICE_ERR_PAGE_ID; a free page's becomes -1 and sets
 *                 ATTN_DEVICE_ERR_PAGES.
 *   scratch       device int32 [attn_pages_scratch(num_pages / 2)], for this call alone
 * Plans hold no copy of page ids, so a plan over that page_table stays valid.
 *
 * num_pages > 0; n, n_entries, table_len, out_len >= 0, below 2^31.  What a call writes (refs,
 * outputs, scratch, the page_table of attn_pages_compact) must overlap neither what it
 * reads nor anything else it writes (compared, but for the pools' contents:
 * ATTN_ERR_INVALID_ARG).  All are asynchronous on `stream` and capturable.
 */
ATTN_API int64_t attn_pages_scratch(int64_t n);
ATTN_API attn_status attn_pages_alloc(int32_t* refs, int32_t num_pages, int32_t n, int32_t* page_ids,
                                      int32_t* device_error, void* stream);
ATTN_API attn_status attn_pages_free(int32_t* refs, int32_t num_pages, const int32_t* page_ids, int64_t n,
                                     int32_t* device_error, void* stream);
ATTN_API attn_status attn_pages_copy(void* const* pools, const int64_t* page_bytes, int32_t n_pools, int32_t num_pages,
                                     const int32_t* src, const int32_t* dst, int64_t n, int32_t* device_error,
                                     void* stream);
ATTN_API attn_status attn_pages_fork(int32_t* refs, int32_t num_pages, const int32_t* page_table,
                                     int64_t table_len, const int32_t* kv_indptr, const int32_t* kv_lens, int32_t batch,
                                     int32_t page_size, const int32_t* parents, int32_t n, int32_t* page_table_out,
                                     int32_t* indptr_out, int64_t out_len, void* const* pools,
                                     const int64_t* page_bytes, int32_t n_pools, int32_t* scratch,
                                     int32_t* device_error, void* stream);
ATTN_API attn_status attn_pages_compact(int32_t* refs, int32_t num_pages, int32_t* page_table, int64_t n_entries,
                                        int32_t* remap, void* const* pools, const int64_t* page_bytes,
                                        int32_t n_pools, int32_t* scratch, int32_t* device_error, void* stream);

/*
 * The 4-bit KV cache -- the same pages, heads and tokens as kv_cache in 4 bits
 * a value plus one 8-bit scale per 16 dims (9/32 of the bytes), for batches
 * whose bf16 cache would not fit or whose decode waits for it.  No source
 * describes one: attn_append_kv4 to attn_decode_kv4 are interface additions.
 *
 *   kv4_cache  uint8 [num_pages][2][Hkv][page_size / 16][9 * head_dim], 16-byte
 *              aligned ([.][0] = K, [.][1] = V).  The last two dimensions are
 *              16 tokens: 16 rows of head_dim / 2 code bytes (dim 2i in the low
 *              nibble of byte i, dim 2i + 1 in the high one), then 16 rows of
 *              head_dim / 16 scale bytes.
 *   value      code * scale * g.  Code: e2m1 (sign; 0, .5, 1, 1.5, 2, 3, 4, 6);
 *              scale: e4m3; g: k_scale for K, v_scale for V, one per pool, a
 *              power of two in [2^-40, 2^40] (else ATTN_ERR_INVALID_ARG), so
 *              that the block scales (2^-9 .. 448) cover the data: 1 for values
 *              around 1.  Use one k_scale and v_scale for all calls on a pool.
 * bf16 holds every such value exactly.
 *
 * attn_append_kv4 -- attn_append_kv into a 4-bit cache: each 16 dims x of a new
 * row are stored as scale s = e4m3 round(max|x| / (6 g)) and codes
 * e2m1 round(x / (g s)), both to nearest, ties to even, saturating (largest
 * magnitude 6 * 448 * g).  A NaN makes its 16 values NaN.  Other rows' bytes
 * keep their values.
 *
 * attn_expand_kv4 -- the listed pages' values as bf16 HND pages
 * buf[n_pages][2][Hkv][page_size][head_dim] (whole pages, exact), for
 * attn_prefill over a 4-bit cache: expand a request's pages into a bf16 pool
 * and plan the prefill on that.  head_dim 64 or 128, page_size a multiple of
 * 16, num_kv_heads * page_size * head_dim below 2^33 (else ATTN_ERR_UNSUPPORTED);
 * page_ids, n_pages, device_error as in attn_pack_kv_heads.
 *
 * attn_decode_kv4 -- attn_decode over a 4-bit cache: the same plan, rows, sinks,
 * out and lse (and the same workspace regions: it must not overlap attn_decode
 * on the same plan).
 *
 * All three are asynchronous on `stream` and capturable (the plan's lengths are
 * fixed; there is no form for attn_graph_plan).  Plans: host-planned paged
 * ones (others: ATTN_ERR_INVALID_ARG).
 */
ATTN_API attn_status attn_append_kv4(attn_plan_t plan, const void* k_new, const void* v_new, float k_scale,
                                     float v_scale, void* kv4_cache, void* stream);
ATTN_API attn_status attn_expand_kv4(const void* kv4_cache, int64_t num_pages, int32_t num_kv_heads,
                                     int32_t page_size, int32_t head_dim, const int32_t* page_ids, int64_t n_pages,
                                     float k_scale, float v_scale, void* buf, int32_t* device_error, void* stream);
ATTN_API attn_status attn_decode_kv4(attn_plan_t plan, const void* q, const void* kv4_cache, float k_scale,
                                     float v_scale, const float* sinks, void* out, float* lse, void* stream);

/*
 * attn_key_weights / attn_key_weights_kv4 -- how much attention each cached key
 * receives, the measure that eviction goes by (no source describes it: an
 * interface addition).  For every request of the plan with query rows, every
 * KV head g and every cached token t < kv_len:
 *
 *   weights[t, g] = decay * prev[t, g] + sum_{i, h} exp(sm_scale q[i,h] . k[t,g] - lse[i,h])
 *
 * over the request's last `window` query rows i (0: all of them) that see key
 * t under the plan's mask and the query heads h of KV head g.  Tokens that the
 * plan appends (t >= kv_len - qo_len) have no previous weight; with decay = 0
 * prev is not read.  lse is what attn_decode / attn_prefill wrote for the same
 * q (with a sink, the weights of a row and head sum to less than 1).
 *
 *   weights, prev  fp32 [num_pages][Hkv][page_size], device, paged like the
 *                  cache (prev may be weights; NULL when decay = 0).  Only the
 *                  slots of the plan's tokens are written; requests without
 *                  query rows are left out.  A weight belongs to a page's slot:
 *                  on a page that two requests of the plan share, which of
 *                  the two requests' weights a slot holds is not defined, and
 *                  with prev = weights one may have been added to the other's.
 *                  Requests that share pages need buffers (and plans) of their
 *                  own for weights that can be told apart.
 *   lse            fp32 [total_qo_rows][Hq];   decay finite, >= 0
 *   kv_cache       as in attn_decode;  kv4_cache, k_scale as in attn_decode_kv4
 * Decode and prefill rows alike.  The sum's order is fixed: equal calls give
 * equal bits (but in shared slots, see above).  Pages out of range set
 * ATTN_DEVICE_ERR_PAGE_ID and their tokens are skipped.  Host-planned paged
 * plans only; ATTN_ERR_UNSUPPORTED where the prefill requests have more than
 * 2^31 - 1 tiles of 128 keys times Hkv.  Async on `stream`.
 */
ATTN_API attn_status attn_key_weights(attn_plan_t plan, const void* q, const void* kv_cache, const float* lse,
                                      const float* prev, float decay, int32_t window, float* weights, void* stream);
ATTN_API attn_status attn_key_weights_kv4(attn_plan_t plan, const void* q, const void* kv4_cache, float k_scale,
                                          const float* lse, const float* prev, float decay, int32_t window,
                                          float* weights, void* stream);

/*
 * attn_evict_kv / attn_evict_kv4 -- shrink every request of the plan to at most
 * `budget` cached tokens per KV head, by weight (no source describes it: an
 * interface addition).  Of a request's n = kv_len tokens each KV head keeps
 * m = min(n, budget): the newest min(n, recent), and of the others those with
 * the largest weights (equal ones: the older token; NaN counts as the lowest).
 * Heads choose on their own; kept tokens stay in order and become tokens
 * 0 .. m - 1 of the request, so that decode, key weights and eviction go on
 * over a cache of m tokens (plan it with kv_len = m; keys carry their
 * positional encoding with them).
 *
 *   weights         fp32 [num_pages][Hkv][page_size] as attn_key_weights writes it,
 *                   16-byte aligned
 *   kept            int32 [batch][Hkv][budget], device, output: the kept token
 *                   indices in order, -1 from m on
 *   page_table_out  device int32: pages that receive the kept tokens, request b's
 *                   ceil(m_b / page_size) ids after those of the requests before
 *                   it, in pools of num_pages_out pages kv_out / weights_out
 *                   (kv_cache's and weights' layout; may be the input pools, the
 *                   pages then distinct from every page the plan reads).
 *                   NULL: in place, in each request's own first pages; kv_out,
 *                   weights_out and num_pages_out are then the inputs' own, and
 *                   no page may belong to two requests.
 *   1 <= budget, 0 <= recent <= budget;  batch * Hkv < 2^30 (else ATTN_ERR_UNSUPPORTED)
 * Slots of the receiving pages past the kept tokens are left as they were.
 * Page ids out of range set ATTN_DEVICE_ERR_PAGE_ID: such a source page's
 * tokens count as NaN weights, and what would be read from or written to such a
 * page is skipped.  Host-planned paged plans only.  Async on `stream`.
 */
ATTN_API attn_status attn_evict_kv(attn_plan_t plan, const float* weights, const void* kv_cache, int32_t budget,
                                   int32_t recent, int32_t* kept, const int32_t* page_table_out,
                                   int32_t num_pages_out, void* kv_out, float* weights_out, void* stream);
ATTN_API attn_status attn_evict_kv4(attn_plan_t plan, const float* weights, const void* kv4_cache, int32_t budget,
                                    int32_t recent, int32_t* kept, const int32_t* page_table_out,
                                    int32_t num_pages_out, void* kv4_out, float* weights_out, void* stream);

/* Copy the plan's summary into *info (host only). */
ATTN_API attn_status attn_plan_get_info(attn_plan_t plan, attn_plan_info* info);

/*
 * Host copies of the plan's work lists, for inspection and tests.  Each
 * decode unit is 12 int32: q_row, page_base, kv_head, head0, n_heads,
 * tok_begin, tok_end, chunk, n_chunks, group, partial0, reserved.  Each
 * prefill item is 12 int32: q_row0, n_rows, page_base, kv_len, pos0, kv_head,
 * head0, n_heads, n_kv_tiles, key_end, reserved, reserved (pos0 = absolute
 * position of the tile's first query; key_end = one past the last key any
 * row of the tile may see).  `capacity` counts units/items; at most that many
 * are copied.  In a cross plan a unit's or item's keys are rows page_base +
 * [tok_begin, tok_end) or [0, kv_len) of k and v, and its rows and heads are pairs: pair p
 * from (q_row, kv_head * G) on is row p / G, head p % G of the KV head's G.  A unit has
 * pairs head0 .. head0 + n_heads - 1 of its sequence; an item has n_rows pairs from q_row0
 * on and, where n_heads = 2, as many as the first reserved word says from row
 * q_row0 + 128 / G on; pos0 >= 0 marks a chunk of split keys, the second reserved
 * word being which.
 */
ATTN_API attn_status attn_plan_get_decode_units(attn_plan_t plan, int32_t* units, int64_t capacity);
ATTN_API attn_status attn_plan_get_prefill_items(attn_plan_t plan, int32_t* items, int64_t capacity);

/* The requests' kv_len (attn_plan's paged plans), at most `capacity` of them:
 * what attn_evict_kv's page_table_out is sized by. */
ATTN_API attn_status attn_plan_get_kv_lens(attn_plan_t plan, int32_t* kv_lens, int64_t capacity);

/*
 * attn_plan_device_error -- wait for `stream`, then read and clear the plan's
 * device error word (ATTN_DEVICE_ERR_* bits) into *code.  Returns
 * ATTN_ERR_DEVICE if any bit was set.
 */
ATTN_API attn_status attn_plan_device_error(attn_plan_t plan, int32_t* code, void* stream);

/* Free the plan's host memory.  Does not touch the workspace.  NULL is a no-op. */
ATTN_API void attn_plan_destroy(attn_plan_t plan);

/* Static, human-readable name of a status code. */
ATTN_API const char* attn_status_string(attn_status status);

/*
 * attn_selftest_bounded_wait -- diagnostic of the kernels' failure detection.
 * Launches one warp on `stream` that waits, through the same bounded mbarrier
 * wait every kernel uses, on a barrier nothing arrives on.  The wait gives up
 * after its wall-time limit (2 s), and the kernel writes
 * ATTN_DEVICE_ERR_TIMEOUT to result[0] (0 had the wait completed) and the
 * nanoseconds it waited to result[1], then returns; the context stays usable.
 *   result   DEVICE int64 [2], caller-owned
 * Returns ATTN_ERR_INVALID_ARG for a NULL result, ATTN_ERR_CUDA if the launch
 * fails.
 */
ATTN_API attn_status attn_selftest_bounded_wait(int64_t* result, void* stream);

/*
 * attn_selftest_exp2 -- diagnostic of the prefill softmax's exponentials.
 * The online softmax of "GPT-OSS on day 0" (Perplexity), section "Sink
 * Attention", needs exp(s - m) for every visible score; the prefill kernel
 * evaluates it as 2^(s * sm_scale * log2(e) - m) and takes part of each
 * tile's exponentials as a cubic polynomial on the FMA pipe instead of the
 * MUFU's ex2.approx.  This launches, on `stream`, the kernel's own inline
 * polynomial (with the kernel's argument set-up) next to ex2.approx:
 *   y_poly[k] = polynomial 2^(x[k] * scale_log2 - m)   (argument clamped to [-126, 126])
 *   y_mufu[k] = ex2.approx.ftz(x[k] * scale_log2 - m)
 *   x, y_poly, y_mufu   DEVICE fp32 [n], caller-owned
 * Returns ATTN_ERR_INVALID_ARG for n < 0 or NULL arrays (n > 0), ATTN_ERR_CUDA
 * if the launch fails.  Allocates nothing.
 */
ATTN_API attn_status attn_selftest_exp2(const float* x, float* y_poly, float* y_mufu, int64_t n,
                                        float scale_log2, float m, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H */
