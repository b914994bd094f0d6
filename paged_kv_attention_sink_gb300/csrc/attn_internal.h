// Internal declarations shared by the planner (host) and the kernels.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <vector>

#include <cuda_runtime.h>

#include "../../include/attn.h"

namespace attn {

constexpr int kBlockTokens = 16;          // decode streams K/V in 16-token blocks
constexpr int kMaxSliceHeads = 16;        // query heads per decode CTA (one m16 MMA tile)
constexpr int kDecodeWarps = 4;           // warps per decode CTA
constexpr int kDecodeMinChunkBlocks = 8;  // never split a sequence finer than 128 tokens
constexpr int kDecodeMaxChunkBlocks = 512;
constexpr int kDecodeMaxChunkPages = kDecodeMaxChunkBlocks * kBlockTokens / 16 + 2;
constexpr int kPrefillRows = 128;         // query rows per prefill tile (TMEM lanes)
constexpr int kPrefillOutRows = 32;       // rows per output TMA store (one softmax warp's stripe)
constexpr int kPrefillKeys = 128;         // keys per prefill KV tile
constexpr int kGraphMaxBatch = 4096;      // attn_graph_plan: requests the device planner can order

// One decode CTA: a chunk [tok_begin, tok_end) of one request's KV sequence for
// one KV head and up to 16 of its query heads.
struct DecodeUnit {
    int32_t q_row;      // row of q / out / lse
    int32_t page_base;  // kv_indptr[b]: first slot of the request in page_table
    int32_t kv_head;
    int32_t head0;      // first query head of the slice
    int32_t n_heads;    // query heads in the slice (1..16)
    int32_t tok_begin;  // a multiple of 16
    int32_t tok_end;    // <= kv_len
    int32_t chunk;      // index of this chunk within its group; chunk 0 carries the sink
    int32_t n_chunks;   // 1 = not split
    int32_t group;      // split-merge counter index, -1 when not split
    int32_t partial0;   // first partial-state slot of the group
    int32_t reserved;
};
static_assert(sizeof(DecodeUnit) == 48, "decode unit is 12 int32");

// One prefill CTA: 128 query rows of one request for up to two query heads of
// one GQA group.
struct PrefillItem {
    int32_t q_row0;      // first row of the tile in q / out / lse
    int32_t n_rows;      // valid rows (1..128)
    int32_t page_base;
    int32_t kv_len;
    int32_t pos0;        // absolute position of row 0 (kv_len - qo_len + tile offset)
    int32_t kv_head;
    int32_t head0;
    int32_t n_heads;     // 1 or 2
    int32_t n_kv_tiles;  // 128-key KV tiles visited
    int32_t key_end;     // one past the last key any row of the tile may see
    int32_t reserved0;
    int32_t reserved1;
};
static_assert(sizeof(PrefillItem) == 48, "prefill item is 12 int32");

// One request of a paged plan, for the kernels that work on whole requests
// (key weights, eviction).
struct RequestInfo {
    int32_t q_row0;     // first row in q / lse
    int32_t qo_len;
    int32_t page_base;  // kv_indptr[b]: first slot of the request in page_table
    int32_t kv_len;
};
static_assert(sizeof(RequestInfo) == 16, "request info is one 16-byte load");

// 128 keys of a prefill request are the work item of its key weights (times KV
// heads).  A run is consecutive such tiles of one request that equally many query
// rows see: all of those under its prefix, or a single one on the diagonal.
// Tiles are numbered through the runs.
constexpr int kWeightTileKeys = 128;
struct WeightRun {
    int32_t tile0;      // number of its first tile
    int32_t key0;       // first key of that
    RequestInfo request;
    int32_t reserved[2];
};
static_assert(sizeof(WeightRun) == 32, "weight run is one sector");
// A tile's run is found from a table that has the run of every 32nd tile: it is
// that one or one of the 31 after it (that one, where kWeightHintAll is set).
constexpr int kWeightHintTiles = 32;
constexpr uint32_t kWeightHintAll = 0x80000000u;

// A step of a tile is 128 (row, head) pairs: 128 / G query rows with their G
// heads of the KV head, or, beyond 128 heads, one row in slices.
constexpr int kWeightTileRows = 128;
inline int64_t weight_steps(int64_t rows, int G) {
    const int heads = G < kWeightTileRows ? G : kWeightTileRows, per = kWeightTileRows / heads;
    return (rows + per - 1) / per * ((G + heads - 1) / heads);
}

// Two forms of the kernel, for tiles of many steps and for many tiles of few.
constexpr int kWeightShortSteps = 64;
constexpr int weight_short_ctas(int head_dim) { return head_dim == 64 ? 4 : 2; }   // short form, per SM

// Tiles of some prefill requests, and their steps (the last `window` rows alone,
// 0: all; causality not counted).
struct WeightLoad {
    int64_t tiles = 0, steps = 0, longest = 0;   // longest: most steps of one tile
    void add(const RequestInfo& r, int G, int32_t window) {
        const int64_t n = ((int64_t)r.kv_len + kWeightTileKeys - 1) / kWeightTileKeys;
        const int64_t s = weight_steps(window > 0 && window < r.qo_len ? window : r.qo_len, G);
        tiles += n;
        steps += n * s;
        longest = longest > s ? longest : s;
    }
    // Whether the short form takes them; what the rule goes by is in keyweights.cu.
    bool takes_short_form(int Hkv, int sms, int head_dim) const {
        const int64_t ctas = tiles * Hkv;
        return ctas > sms && steps <= kWeightShortSteps * tiles &&
               2 * steps * sms <= 3 * weight_short_ctas(head_dim) * ctas * tiles;
    }
    // Whether the short form's longest CTA ends within the time that all of them take.
    bool even(int Hkv, int sms) const { return 8 * longest * sms <= 5 * steps * Hkv; }
};

// The 4-bit cache holds 16 tokens of a (page, K/V, KV head) block together:
// 16 rows of D / 2 code bytes, then 16 rows of D / 16 scale bytes.
constexpr int kKv4Tokens = 16;
constexpr int kKv4Group = 16;             // dims that share an e4m3 scale
constexpr int kv4_sub_bytes(int head_dim) { return kKv4Tokens * (head_dim / 2 + head_dim / kKv4Group); }

struct WorkspaceLayout {
    size_t units = 0, items = 0, item_off = 0, append = 0, counters = 0, err = 0, n_units = 0, part_lse = 0, part_o = 0,
           total = 0;
};

// The lists of whole requests (key weights, eviction) lie in the workspace in
// front of those regions, and are no part of attn_decode_noalloc's static scratch.
struct ListLayout {
    size_t requests = 0, weight_runs = 0, weight_starts = 0, weight_hints = 0, total = 0;   // total: a multiple of 256
};

// CTAs of the decode kernel resident per SM for a head dim (matches its
// shared-memory footprint); defined next to the kernel.
int decode_ctas_per_sm(int head_dim);

// SM count of the current device, queried once per device (thread-safe).
bool current_sm_count(int32_t* out);

// Device ordinals that the per-device caches below cover; a higher ordinal
// is served without a cache.
constexpr int kMaxDevices = 64;

// Runs `setup` (returning cudaError_t) until it first succeeds on the current
// device, then only checks a flag.  Kernel attributes such as the dynamic
// shared-memory limit belong to one device's context, so a process that
// drives several devices sets them on each.  Two threads may both run setup
// the first time; it must be idempotent.
template <class F>
cudaError_t once_per_device(std::atomic<bool> (&done)[kMaxDevices], F&& setup) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (cached && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = setup();
    if (e == cudaSuccess && cached) done[dev].store(true, std::memory_order_release);
    return e;
}

}  // namespace attn

struct attn_plan_s {
    int32_t batch = 0, Hq = 0, Hkv = 0, D = 0, P = 0, causal = 0;
    float sm_scale = 0.f;
    int32_t num_pages = 0;
    int32_t num_sms = 0;
    const int32_t* page_table = nullptr;  // device, borrowed
    bool ragged = false;                  // contiguous K / V (attn_plan_ragged), no page table
    bool graph = false;                   // attn_graph_plan: decode work list built on the device
                                          // (batch = max batch; n_partials / n_groups = capacities)
    int64_t kv_tokens = 0;                // ragged: rows of K and V (kv_indptr[batch])
    int64_t graph_kv_blocks = 0;          // graph: 16-token blocks a batch may hold in total

    std::vector<attn::RequestInfo> requests;   // paged plans: every request, in order
    std::vector<attn::WeightRun> weight_runs;  // prefill requests' 128-key tiles, most query rows first
    std::vector<int32_t> weight_starts;        // the runs' first tiles once more
    std::vector<uint32_t> weight_hints;        // the run of every 32nd tile
    int32_t weight_tiles = 0;
    int32_t weight_long_tiles = 0;             // > 0: requests of many steps come first, this many tiles
    std::vector<attn::DecodeUnit> units;
    std::vector<attn::PrefillItem> items;
    std::vector<int32_t> append_slots;    // per query row: page-table slot, row in page
    std::vector<int32_t> item_off;        // CTA c runs items [item_off[c], item_off[c+1])
    int32_t prefill_ctas = 0;
    int32_t n_groups = 0;
    int32_t n_partials = 0;
    attn_plan_info info{};
    attn::WorkspaceLayout layout;
    attn::ListLayout lists_layout;

    unsigned char* lists = nullptr;  // device, caller-owned: the lists ...
    unsigned char* ws = nullptr;     // ... and after them the regions of `layout`
    size_t ws_bytes = 0;
    bool bound = false;

    // Tensor maps are 128-byte opaque driver objects; cached per KV / Q pointer.
    alignas(64) unsigned char kv_map_decode[128];
    const void* kv_map_decode_ptr = nullptr;
    alignas(64) unsigned char kv_map_prefill[128];
    const void* kv_map_prefill_ptr = nullptr;
    alignas(64) unsigned char q_map_prefill[128];
    const void* q_map_prefill_ptr = nullptr;
    alignas(64) unsigned char q_map_weights[128];
    const void* q_map_weights_ptr = nullptr;
    alignas(64) unsigned char v_map_prefill[128];   // ragged: K in kv_map_prefill, V here
    const void* v_map_prefill_ptr = nullptr;
    alignas(64) unsigned char o_map_prefill[128];   // out, laid out like q, 32-row boxes
    const void* o_map_prefill_ptr = nullptr;
};
