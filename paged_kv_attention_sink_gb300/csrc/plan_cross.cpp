// Planner of cross attention: the query rows of each sequence over all of its
// encoder states, which have a length of their own.
//
// All rows of a sequence see the same keys, so a KV head's work is a dense
// product of its (row, query head) pairs with the keys.  Few pairs are bound by
// reading K and V: units of up to 64 pairs and a chunk of keys, on the kernel of
// cross.cu.  Many pairs are bound by the tensor cores: items of up to 256 pairs and
// all keys, on the prefill kernel.
#include <algorithm>
#include <cmath>
#include <exception>
#include <memory>
#include <new>
#include <vector>

#include "attn_internal.h"

namespace attn {
namespace {

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Pairs of a sequence and KV head from which it goes to the prefill kernel.
constexpr int64_t kCrossManyPairs = 65;

attn_status build(const int32_t* qo_indptr, const int32_t* kv_start, const int32_t* kv_len, int32_t batch,
                  int32_t kv_rows, int32_t Hq, int32_t Hkv, int32_t D, float sm_scale, int32_t num_sms,
                  attn_plan_t* plan_out, size_t* workspace_bytes_out) {
    if (!plan_out || !workspace_bytes_out || batch < 0 || kv_rows < 0 || num_sms < 0) return ATTN_ERR_INVALID_ARG;
    if (batch > 0 && (!qo_indptr || !kv_start || !kv_len || qo_indptr[0] != 0)) return ATTN_ERR_INVALID_ARG;
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D <= 0) return ATTN_ERR_INVALID_ARG;
    if (!std::isfinite(sm_scale) || !(sm_scale > 0.f)) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    for (int32_t b = 0; b < batch; ++b)
        if (qo_indptr[b + 1] < qo_indptr[b] || kv_start[b] < 0 || kv_len[b] < 0 ||
            (int64_t)kv_start[b] + kv_len[b] > kv_rows)
            return ATTN_ERR_INVALID_ARG;
    const int64_t total_rows = batch > 0 ? qo_indptr[batch] : 0;
    // Keys up to here are counted in 32 bits with a tile on top; so are pairs.
    if (total_rows * Hq > (int64_t)INT32_MAX / 2 || kv_rows > INT32_MAX / 2) return ATTN_ERR_UNSUPPORTED;
    if (num_sms == 0 && !current_sm_count(&num_sms)) return ATTN_ERR_CUDA;

    std::unique_ptr<attn_plan_s> plan(new (std::nothrow) attn_plan_s());
    if (!plan) return ATTN_ERR_INVALID_ARG;
    plan->batch = batch;
    plan->Hq = Hq;
    plan->Hkv = Hkv;
    plan->D = D;
    plan->P = kPrefillKeys;
    plan->sm_scale = sm_scale;
    plan->num_sms = num_sms;
    plan->ragged = plan->cross = true;
    plan->kv_tokens = kv_rows;
    const int G = Hq / Hkv;

    // ---- few pairs (and none but the sinks to see): blocks of pairs x chunks of keys.
    auto few = [&](int64_t pairs, int32_t keys) { return keys == 0 || pairs < kCrossManyPairs || G > kPrefillRows; };
    auto stages_of = [](int32_t keys) { return ((int64_t)keys + kCrossKeys - 1) / kCrossKeys; };
    int64_t work = 0, decode_tokens = 0, prefill_pairs = 0;
    for (int32_t b = 0; b < batch; ++b) {
        const int64_t rows = qo_indptr[b + 1] - qo_indptr[b], pairs = rows * G;
        if (rows == 0) continue;
        if (few(pairs, kv_len[b])) {
            work += (pairs + 63) / 64 * stages_of(kv_len[b]) * Hkv;
            decode_tokens += kv_len[b];
        } else {
            prefill_pairs += rows * kv_len[b];
        }
    }
    const int64_t target = 2 * (int64_t)num_sms * cross_ctas_per_sm(D);
    const int64_t chunk = std::max<int64_t>((work + target - 1) / target, kCrossMinChunk);
    struct Piece {
        int32_t size;   // log2 of the block's 16-pair tiles
        DecodeUnit u;
    };
    std::vector<Piece> pieces;
    int64_t partials = 0;
    for (int32_t b = 0; b < batch; ++b) {
        const int64_t rows = qo_indptr[b + 1] - qo_indptr[b], pairs = rows * G;
        if (rows == 0 || !few(pairs, kv_len[b])) continue;
        const int64_t stages = stages_of(kv_len[b]), n_chunks = std::max<int64_t>(1, (stages + chunk / 2) / chunk);
        for (int64_t p0 = 0; p0 < pairs; p0 += 64) {
            const int32_t n_pairs = (int32_t)std::min<int64_t>(64, pairs - p0);
            const int32_t size = n_pairs <= 16 ? 0 : n_pairs <= 32 ? 1 : 2;
            for (int32_t g = 0; g < Hkv; ++g) {
                DecodeUnit u{};
                u.q_row = qo_indptr[b];
                u.page_base = kv_start[b];
                u.kv_head = g;
                u.head0 = (int32_t)p0;
                u.n_heads = n_pairs;
                u.n_chunks = (int32_t)n_chunks;
                u.group = -1;
                u.reserved = pairs > 64;   // other blocks read the same keys
                if (n_chunks > 1) {
                    u.group = plan->n_groups++;
                    u.partial0 = (int32_t)partials;
                    partials += n_chunks << size;
                    if (partials > INT32_MAX / kMaxSliceHeads) return ATTN_ERR_UNSUPPORTED;
                }
                for (int64_t c = 0; c < n_chunks; ++c) {
                    u.chunk = (int32_t)c;
                    u.tok_begin = (int32_t)(c * stages / n_chunks * kCrossKeys);
                    u.tok_end = (int32_t)std::min<int64_t>(kv_len[b], (c + 1) * stages / n_chunks * kCrossKeys);
                    pieces.push_back({size, u});
                }
            }
        }
    }
    if (pieces.size() > (size_t)INT32_MAX / sizeof(DecodeUnit)) return ATTN_ERR_UNSUPPORTED;
    std::stable_sort(pieces.begin(), pieces.end(), [](const Piece& x, const Piece& y) {
        const int32_t a = x.u.tok_end - x.u.tok_begin, b = y.u.tok_end - y.u.tok_begin;
        return x.size != y.size ? x.size < y.size : a > b;   // longest first
    });
    plan->units.reserve(pieces.size());
    for (const Piece& p : pieces) {
        plan->units.push_back(p.u);
        ++plan->cross_units[p.size];
    }
    plan->n_partials = (int32_t)partials;

    // ---- many pairs: items of one or two head slots of slot_rows rows x G heads.
    const int64_t slot_rows = G <= kPrefillRows ? kPrefillRows / G : 1;
    int64_t slots = 0;
    for (int32_t b = 0; b < batch; ++b) {
        const int64_t rows = qo_indptr[b + 1] - qo_indptr[b];
        if (rows > 0 && !few(rows * G, kv_len[b])) slots += (rows + slot_rows - 1) / slot_rows * Hkv;
    }
    const int64_t per_item = slots <= num_sms ? 1 : 2;   // a slot each while the SMs suffice
    if (slots > (int64_t)INT32_MAX / (int64_t)sizeof(PrefillItem)) return ATTN_ERR_UNSUPPORTED;
    for (int32_t b = 0; b < batch; ++b) {
        const int64_t rows = qo_indptr[b + 1] - qo_indptr[b];
        if (rows == 0 || few(rows * G, kv_len[b])) continue;
        for (int64_t r0 = 0; r0 < rows; r0 += per_item * slot_rows) {
            const int64_t left = rows - r0;
            for (int32_t g = 0; g < Hkv; ++g) {
                PrefillItem it{};
                it.q_row0 = (int32_t)(qo_indptr[b] + r0);
                it.n_rows = (int32_t)(std::min(left, slot_rows) * G);
                it.reserved0 = per_item == 2 && left > slot_rows ? (int32_t)(std::min(left - slot_rows, slot_rows) * G) : 0;
                it.n_heads = it.reserved0 > 0 ? 2 : 1;
                it.page_base = kv_start[b];
                it.kv_len = it.key_end = kv_len[b];
                it.kv_head = g;
                it.head0 = g * G;
                it.n_kv_tiles = (kv_len[b] - 1) / kPrefillKeys + 1;
                plan->items.push_back(it);
            }
        }
    }
    deal_prefill_items(plan.get());

    WorkspaceLayout& L = plan->layout;
    size_t off = 0;
    L.units = off;    off = align_up(off + plan->units.size() * sizeof(DecodeUnit), 256);
    L.items = off;    off = align_up(off + plan->items.size() * sizeof(PrefillItem), 256);
    L.append = off;
    L.item_off = off; off = align_up(off + plan->item_off.size() * sizeof(int32_t), 256);
    L.counters = off; off = align_up(off + (size_t)plan->n_groups * sizeof(int32_t), 256);
    L.err = off;      off = align_up(off + sizeof(int32_t), 256);
    L.n_units = off;  off = align_up(off + sizeof(int32_t), 256);
    L.part_lse = off; off = align_up(off + (size_t)partials * kMaxSliceHeads * sizeof(float), 256);
    L.part_o = off;   off = align_up(off + (size_t)partials * kMaxSliceHeads * D * sizeof(float), 256);
    L.total = off;

    attn_plan_info& I = plan->info;
    I.batch = batch;
    I.total_qo_rows = (int32_t)total_rows;
    I.num_decode_units = (int32_t)plan->units.size();
    I.num_decode_groups_split = plan->n_groups;
    I.num_decode_partials = plan->n_partials;
    I.decode_chunk_blocks = (int32_t)std::min<int64_t>(chunk * (kCrossKeys / kBlockTokens), INT32_MAX);
    I.num_prefill_items = (int32_t)plan->items.size();
    I.num_sms = num_sms;
    I.decode_kv_tokens = decode_tokens;
    I.prefill_pairs = prefill_pairs;
    I.workspace_bytes = L.total;
    *workspace_bytes_out = I.workspace_bytes;
    *plan_out = plan.release();
    return ATTN_OK;
}

}  // namespace
}  // namespace attn

extern "C" attn_status attn_plan_cross(const int32_t* qo_indptr, const int32_t* kv_start, const int32_t* kv_len,
                                       int32_t batch, int32_t kv_rows, int32_t num_qo_heads, int32_t num_kv_heads,
                                       int32_t head_dim, float sm_scale, int32_t num_sms, attn_plan_t* plan_out,
                                       size_t* workspace_bytes_out) {
    try {
        return attn::build(qo_indptr, kv_start, kv_len, batch, kv_rows, num_qo_heads, num_kv_heads, head_dim, sm_scale,
                           num_sms, plan_out, workspace_bytes_out);
    } catch (const std::exception&) {
        return ATTN_ERR_INVALID_ARG;   // no host memory
    }
}
