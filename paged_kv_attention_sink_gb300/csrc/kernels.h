// Launchers of the CUDA kernels (one per translation unit).
#pragma once

#include <cuda_runtime.h>

#include <utility>

#include "attn_internal.h"

namespace attn {

// Launches a kernel as the programmatic dependent of the one before it on the
// stream: its CTAs may start while that one's last are running.  Every CTA of
// such a kernel calls ptx::grid_dependency_wait() before it reads or writes
// anything that other kernels do, and before it exits; ptx::grid_dependents_go()
// lets the kernel after it start in the same way.  Such a kernel is resident
// while what it will read is still being written, so it reads through plain
// loads (or asynchronous copies) alone: neither __ldg nor a const __restrict__
// parameter, whose loads may take the read-only path and be moved before the
// wait, for they promise that the data does not change while the kernel runs.
// What a plan's own lists hold is uploaded ahead of every launch and may be read
// before the wait.
//
// The `late` kernels of a cross-attention call (launch_cross) are the exception: they
// read q, k and v and write their rows before they wait.  That is sound only behind a
// kernel of the same call that waits before it calls grid_dependents_go(), or behind
// another late one that follows such a kernel: whatever came before the call is then
// complete when a late one starts.  A late kernel writes nothing that the kernels
// which it overlaps read or write, reads nothing that they write, and itself waits
// before it ends, on every path, so that what follows it follows all of them.  No
// kernel that opens before its wait (append and expand of 4-bit pages, eviction, key
// weights of prompts) may stand in front of a late one.
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// kv_map / q_map point at CUtensorMap objects built by the API layer.
attn_status launch_decode(attn_plan_s* plan, const void* q, const void* kv_map, const float* sinks,
                          void* out, float* lse, cudaStream_t stream);
// v_map: the V tensor map of a ragged plan (NULL for a paged plan); o_map:
// `out` with the same layout and box as q_map (full 128-row tiles are stored
// through it).  late: a cross plan's launch beside the one before it (launch_cross).
attn_status launch_prefill(attn_plan_s* plan, const void* q_map, const void* kv_map, const void* v_map,
                           const void* o_map, const float* sinks, void* out, float* lse, cudaStream_t stream,
                           bool late = false);
// in_f32 / out_f32: value states / merged values are fp32 (else bf16).
attn_status launch_merge_states(const void* va, const float* lsea, const void* vb, const float* lseb, void* vout,
                                float* lseout, int64_t rows, int head_dim, bool in_f32, bool out_f32,
                                cudaStream_t stream);
// CUDA-graph decode: device planner + persistent decode over its work list.
attn_status launch_decode_graph(attn_plan_s* plan, const int32_t* kv_indptr, const int32_t* last_page_len,
                                const int32_t* batch, const void* q, const void* kv_map, const float* sinks,
                                void* out, float* lse, cudaStream_t stream);
// New K/V rows of the plan's query rows into their HND page slots.
attn_status launch_append_kv(attn_plan_s* plan, const void* k_new, const void* v_new, void* kv_cache,
                             cudaStream_t stream);
// Heads [h0, h0 + nh) of pages page_ids[0..n) <-> buf[n][2][nh][P][D].
attn_status launch_head_slice(bool unpack, void* kv_cache, void* buf, const int32_t* page_ids, int64_t n,
                              int64_t num_pages, int32_t Hkv, int32_t P, int32_t D, int32_t h0, int32_t nh,
                              int32_t* err, cudaStream_t stream);

// 4-bit cache (kv4.cuh): quantising append, pages back to bf16, decode.
attn_status launch_append_kv4(attn_plan_s* plan, const void* k_new, const void* v_new, void* kv4_cache, float k_scale,
                              float v_scale, cudaStream_t stream);
attn_status launch_expand_kv4(const void* kv4_cache, void* buf, const int32_t* page_ids, int64_t n, int64_t num_pages,
                              int32_t Hkv, int32_t P, int32_t D, float k_scale, float v_scale, int32_t* err,
                              cudaStream_t stream);
attn_status launch_decode_kv4(attn_plan_s* plan, const void* q, const void* kv4_cache, float k_scale, float v_scale,
                              const float* sinks, void* out, float* lse, cudaStream_t stream);
// four: `pool` is a 4-bit cache (else bf16; prefill requests read it through
// kv_map).
attn_status launch_key_weights(attn_plan_s* plan, bool four, const void* q, const void* pool, float k_scale,
                               const void* q_map, const void* kv_map, const float* lse, const float* prev, float decay, int32_t window, float* weights,
                               cudaStream_t stream);
// page_table_out NULL: in place (pool_out / weights_out are then the inputs).
attn_status launch_evict(attn_plan_s* plan, bool four, const float* weights, const void* pool, int32_t budget,
                         int32_t recent, int32_t* kept, const int32_t* page_table_out, int32_t num_pages_out,
                         void* pool_out, float* weights_out, cudaStream_t stream);

// Rotary positions (rope.cu).  freq: each pair's frequency in turns, a 64-bit
// fixed-point fraction; axes: which row of positions it takes, 4 bits each.
constexpr int kRopeMaxPairs = 64;
struct RopeTable {
    uint64_t freq[kRopeMaxPairs];
    uint64_t axes[kRopeMaxPairs / 16];
    int32_t pairs;   // a multiple of 8
    float scale;
};
// Rows [rows][heads][head_dim] of bf16 whose last two dimensions are contiguous; strides in elements.
struct RopeRows {
    const void* in = nullptr;
    int64_t stride = 0;
    void* out = nullptr;
    int64_t out_stride = 0;
    int32_t heads = 0;
};
attn_status launch_rope(const RopeTable& t, bool inter, bool inverse, const int32_t* positions, int64_t rows,
                        int32_t head_dim, const RopeRows& q, const RopeRows& k, cudaStream_t stream);
// q.out: contiguous rows; k.out: the page pool.
attn_status launch_append_kv_rope(attn_plan_s* plan, const RopeTable& t, bool inter, const int32_t* positions,
                                  const RopeRows& q, const RopeRows& k, const RopeRows& v, cudaStream_t stream);

// Cross attention (cross.cu): few rows from plan->cross_maps, many through launch_prefill
// (q_map, o_map: of these alone).
attn_status launch_cross(attn_plan_s* plan, const void* q, const void* q_map, const void* o_map, const float* sinks,
                         void* out, float* lse, cudaStream_t stream);

// Page management (pages.cu).
constexpr int kPagePoolsPerLaunch = 64;
struct PagePools {
    unsigned char* pool[kPagePoolsPerLaunch];
    int64_t bytes[kPagePoolsPerLaunch];   // of a page, a multiple of 16
    int32_t n;
};
attn_status launch_pages_alloc(int32_t* refs, int32_t num_pages, int32_t n, int32_t* page_ids, int32_t* err,
                               cudaStream_t stream);
attn_status launch_pages_free(int32_t* refs, int32_t num_pages, const int32_t* page_ids, int64_t n, int32_t* err,
                              cudaStream_t stream);
struct PageFork {
    const int32_t *page_table, *kv_indptr, *kv_lens, *parents;
    int64_t table_len;
    int32_t batch, n, page_size;
    int32_t *table_out, *indptr_out;
    int64_t out_len;
};
// Forks and compactions copy in `pools`, the first ones of the call; the copies that
// other pools need are then in scratch (page_move_words(n) int32, on the device).
attn_status launch_pages_fork(int32_t* refs, int32_t num_pages, const PageFork& f, const PagePools& pools,
                              int32_t* scratch, int32_t* err, cudaStream_t stream);
attn_status launch_pages_compact(int32_t* refs, int32_t num_pages, int32_t* page_table, int64_t entries, int32_t* remap,
                                 const PagePools& pools, int32_t* scratch, int32_t* err, cudaStream_t stream);
// Copies pages src[i] -> dst[i], i < *n (device; NULL: n_max) <= n_max, in every pool.
attn_status launch_pages_copy(const PagePools& pools, int32_t num_pages, const int32_t* src, const int32_t* dst,
                              const int32_t* n, int64_t n_max, int32_t* err, cudaStream_t stream);
// Layout of the scratch of `moves` copies: the count, then the pages written, then the pages read.
constexpr int kMoveHead = 4;
inline int64_t page_move_words(int64_t moves) { return kMoveHead + 2 * moves; }

}  // namespace attn

namespace attn {

// Same decode launch as launch_decode, but with the plan's device work list,
// partial states, merge counters and error word taken from `scratch` (laid
// out as the plan's workspace) instead of the bound workspace.
attn_status launch_decode_scratch(attn_plan_s* plan, unsigned char* scratch, const void* q,
                                  const void* kv_map, const float* sinks, void* out, float* lse,
                                  cudaStream_t stream);

// Build the decode kernel's KV tensor map for `kv_cache` into `map` (128 bytes,
// 64-byte aligned).  Returns false if the driver rejects it.
bool encode_decode_kv_map(void* map, const void* kv_cache, const attn_plan_s* plan);

}  // namespace attn
