// Planner of cross attention: the query rows of each sequence over all of its
// encoder states, which have a length of their own.
//
// All rows of a sequence see the same keys, so a KV head's work is a dense
// product of its (row, query head) pairs with the keys.  Few pairs are bound by
// reading K and V: units of up to 32 pairs and a chunk of keys, on the kernel of
// cross.cu.  Many pairs go to the prefill kernel's tensor-core products: items of
// up to 256 pairs and all keys or, where that would leave SMs without work, a
// chunk of them, whose states a small kernel joins.
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

// Pairs of a sequence and KV head from which it goes to the prefill kernel.  Both
// sides, us: 32 pairs, kernel for few against prefill kernel: 64 sequences of 1,500
// keys, 8 heads of 64 dims 46 against 52, 4 heads of 128 dims 36 against 47; one of
// 16,000 keys, 16 heads of 64 dims 20 against 21.  48 pairs (with blocks of 64): 68
// against 52, 68 against 45, 45 against 21.  A slot of the prefill kernel holds whole
// rows' heads, so more than 128 heads per KV head stay with the kernel for few.
constexpr int64_t kCrossManyPairs = 33;
constexpr int64_t kCrossUnitCost = 4;    // a unit's start and end, in stages
constexpr double kCrossFewStages = 6;    // stages a CTA slot that sequences of many pairs may have and be treated as few
constexpr int64_t kCrossItemTiles = 4;   // tiles of 128 keys: never split a sequence finer
constexpr double kCrossItemCost = 2;     // an item's start and end, in tiles of two slots
constexpr double kCrossSplitCost = 4;    // the chunks' states and their joining, likewise

void add_merge(attn_plan_s& plan, const CrossMerge& m) {
    const int32_t* words = reinterpret_cast<const int32_t*>(&m);
    plan.append_slots.insert(plan.append_slots.end(), words, words + sizeof m / sizeof(int32_t));
    ++plan.cross_merges;
}

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

    const int64_t slots = (int64_t)num_sms * cross_ctas_per_sm(D);
    // ---- few pairs (and none but the sinks to see): blocks of pairs x chunks of keys.
    auto stages_of = [](int32_t keys) { return ((int64_t)keys + kCrossKeys - 1) / kCrossKeys; };
    // The sequences of many pairs go to the kernel for few all the same where they are
    // little work: up to kCrossFewStages stages a CTA slot, a block's start and end counted.
    // Kernel for few against the one for many: 5 sequences of 61 rows over up to 35 keys, 5
    // heads on 1 of 64 dims 4.5 us against 8.5; 4 of up to 160 rows over 680 keys, 4 heads on
    // 2 of 128 dims 11.9 against 20.0; beyond the limit 6 of up to 976 rows over 17 keys, 10
    // heads on 5 of 64 dims 11.0 against 7.6.  Of the cross cases that perf/more_operators.py
    // draws for seeds 0 to 699 the choice changes 124 by 2 % or more.  Over these a limit
    // of 2, 4, 5, 6, 8 or 16 takes 6.1, 2.1, 1.1, 1.0, 2.1 or 2.9 % longer
    // than the better kernel for each would (geometric mean); one that 6 gets wrong is 1
    // sequence of up to 1,922 rows over 19 keys, 6 heads on 2 of 128 dims: 13.4 us where
    // 10.3 was to be had.
    double short_work = 0;
    for (int32_t b = 0; b < batch; ++b) {
        const int64_t pairs = (int64_t)(qo_indptr[b + 1] - qo_indptr[b]) * G;
        if (pairs >= kCrossManyPairs && kv_len[b] > 0)
            short_work += (double)((pairs + kCrossBlock - 1) / kCrossBlock * Hkv * (stages_of(kv_len[b]) + kCrossUnitCost));
    }
    const bool all_few = G > kPrefillRows || short_work <= kCrossFewStages * (double)slots;
    auto few = [&](int64_t pairs, int32_t keys) { return keys == 0 || pairs < kCrossManyPairs || all_few; };
    int64_t work = 0, decode_tokens = 0, prefill_pairs = 0;
    for (int32_t b = 0; b < batch; ++b) {
        const int64_t rows = qo_indptr[b + 1] - qo_indptr[b], pairs = rows * G;
        if (rows == 0) continue;
        if (few(pairs, kv_len[b])) {
            work += (pairs + kCrossBlock - 1) / kCrossBlock * stages_of(kv_len[b]) * Hkv;
            decode_tokens += kv_len[b];
        } else {
            prefill_pairs += rows * kv_len[b];
        }
    }
    // The chunk length that gives each CTA slot one unit, two, .. up to four: the one
    // whose units end first.  The rounds are full ones and a last one, which goes up to
    // three times as fast, for its CTAs have the memory to themselves; a unit costs
    // kCrossUnitCost stages more than it has.  (One unit a slot against two: 64 x 1,500
    // keys of 8 heads 38 us against 42, 1 x 16,000 of 16 heads 13 against 18, but 8 x
    // 16,000 of 16 heads 99 against 82.)
    auto chunks_of = [](int64_t n, int64_t size) { return std::max<int64_t>(1, (n + size / 2) / size); };
    int64_t chunk = INT32_MAX;
    double least = 0;
    for (int64_t per_slot = 1; work > 0 && per_slot <= 4; ++per_slot) {
        const int64_t s = std::max<int64_t>((work - 1) / (slots * per_slot) + 1, kCrossMinChunk);
        int64_t units = 0, longest = 0;
        for (int32_t b = 0; b < batch; ++b) {
            const int64_t pairs = (int64_t)(qo_indptr[b + 1] - qo_indptr[b]) * G;
            if (pairs == 0 || !few(pairs, kv_len[b])) continue;
            const int64_t n = stages_of(kv_len[b]), c = chunks_of(n, s);
            units += (pairs + kCrossBlock - 1) / kCrossBlock * Hkv * c;
            longest = std::max(longest, (n + c - 1) / c);
        }
        const double last = (double)(units % slots) / (double)slots;
        const double rounds = (double)(units / slots) + (last > 0 ? std::max(last, 1.0 / 3) : 0.0);
        const double cost = std::max(rounds * ((double)work / (double)units + kCrossUnitCost), (double)longest / 3 + kCrossUnitCost);
        if (per_slot == 1 || cost < least) {
            least = cost;
            chunk = s;
        }
    }
    // A block's chunk, for every KV head in turn (its heads' rows lie side by side).
    struct Piece {
        int32_t b, p0, n_pairs, size, chunk, n_chunks, t0, t1, partial0;   // size: log2 of the 16-pair tiles
    };
    std::vector<Piece> pieces;
    int64_t partials = 0;
    for (int32_t b = 0; b < batch; ++b) {
        const int64_t rows = qo_indptr[b + 1] - qo_indptr[b], pairs = rows * G;
        if (rows == 0 || !few(pairs, kv_len[b])) continue;
        const int64_t stages = stages_of(kv_len[b]), n_chunks = chunks_of(stages, chunk);
        for (int64_t p0 = 0; p0 < pairs; p0 += kCrossBlock) {
            Piece p{b, (int32_t)p0, (int32_t)std::min<int64_t>(kCrossBlock, pairs - p0), 0, 0, (int32_t)n_chunks, 0, 0, (int32_t)partials};
            p.size = p.n_pairs > 16;
            if (n_chunks > 1) {
                const int64_t per_head = n_chunks << p.size;
                partials += per_head * Hkv;
                if (partials > INT32_MAX / kMaxSliceHeads) return ATTN_ERR_UNSUPPORTED;
                for (int32_t g = 0; g < Hkv; ++g)
                    add_merge(*plan, {qo_indptr[b], g * G, p.p0, p.n_pairs, (int32_t)(p.partial0 + g * per_head), p.n_chunks,
                                      1 << p.size, 0});
            }
            for (int64_t c = 0; c < n_chunks; ++c) {
                p.chunk = (int32_t)c;
                p.t0 = (int32_t)(c * stages / n_chunks * kCrossKeys);
                p.t1 = (int32_t)std::min<int64_t>(kv_len[b], (c + 1) * stages / n_chunks * kCrossKeys);
                pieces.push_back(p);
            }
        }
    }
    if (pieces.size() > (size_t)INT32_MAX / sizeof(DecodeUnit) / Hkv) return ATTN_ERR_UNSUPPORTED;
    std::stable_sort(pieces.begin(), pieces.end(), [](const Piece& x, const Piece& y) {
        return x.size != y.size ? x.size < y.size : x.t1 - x.t0 > y.t1 - y.t0;   // longest first
    });
    plan->units.reserve(pieces.size() * Hkv);
    for (const Piece& p : pieces) {
        DecodeUnit u{};
        u.q_row = qo_indptr[p.b];
        u.page_base = kv_start[p.b];
        u.head0 = p.p0;
        u.n_heads = p.n_pairs;
        u.tok_begin = p.t0;
        u.tok_end = p.t1;
        u.chunk = p.chunk;
        u.n_chunks = p.n_chunks;
        u.group = -1;   // no merge counter
        u.reserved = (int64_t)(qo_indptr[p.b + 1] - qo_indptr[p.b]) * G > kCrossBlock;   // other blocks read the same keys
        for (u.kv_head = 0; u.kv_head < Hkv; ++u.kv_head) {
            u.partial0 = p.n_chunks > 1 ? p.partial0 + u.kv_head * (p.n_chunks << p.size) : 0;
            plan->units.push_back(u);
        }
        plan->cross_units[p.size] += Hkv;
    }

    // ---- many pairs: items of up to two head slots of slot_rows rows x G heads.
    const int64_t slot_rows = G <= kPrefillRows ? kPrefillRows / G : 1;
    auto tiles_of = [](int32_t keys) { return ((int64_t)keys + kPrefillKeys - 1) / kPrefillKeys; };
    int64_t blocks = 0, tiles = 0;   // of two slots each, and their tiles
    for (int32_t b = 0; b < batch; ++b) {
        const int64_t rows = qo_indptr[b + 1] - qo_indptr[b];
        if (rows == 0 || few(rows * G, kv_len[b])) continue;
        const int64_t n = (rows + 2 * slot_rows - 1) / (2 * slot_rows) * Hkv;
        blocks += n;
        tiles += n * tiles_of(kv_len[b]);
    }
    if (blocks > (int64_t)INT32_MAX / (int64_t)sizeof(PrefillItem)) return ATTN_ERR_UNSUPPORTED;
    // Blocks that would fill the SMs a few times over stay whole, but for those that
    // are longer than an SM's share.  Others are cut so that the SMs' shares come
    // out even: of the chunk lengths that give each SM one item, two, .., the one that
    // ends first, in tiles of two slots: items that are alike take rounds, others
    // are dealt out to about even shares; a tile of one slot costs 3/4, an item
    // kCrossItemCost, the chunks' states and their joining kCrossSplitCost.
    int64_t size = std::max((tiles + num_sms - 1) / num_sms, kCrossItemTiles);
    if (blocks > 0 && blocks < 4 * (int64_t)num_sms) {
        double best = 0;
        for (int64_t per_sm = 0; per_sm <= 6; ++per_sm) {
            const int64_t s = per_sm == 0 ? INT32_MAX : std::max((tiles - 1) / (num_sms * per_sm) + 1, kCrossItemTiles);
            int64_t items = 0;
            double all = 0, longest = 0;
            bool split = false;
            for (int32_t b = 0; b < batch; ++b) {
                const int64_t rows = qo_indptr[b + 1] - qo_indptr[b], n = tiles_of(kv_len[b]);
                if (rows == 0 || few(rows * G, kv_len[b])) continue;
                const int64_t c = chunks_of(n, s), twos = (rows + slot_rows - 1) / (2 * slot_rows);
                const int64_t ones = (rows + slot_rows - 1) / slot_rows % 2;
                const double len = (double)((n - 1) / c + 1);
                items += (twos + ones) * Hkv * c;
                all += (double)(Hkv * c) * ((double)twos * (len + kCrossItemCost) + (double)ones * (0.75 * len + kCrossItemCost));
                longest = std::max(longest, (twos > 0 ? len : 0.75 * len) + kCrossItemCost);
                split = split || c > 1;
            }
            const double mean = all / (double)items;
            const bool alike = longest <= 1.25 * mean;
            const double cost = (alike ? (double)((items - 1) / num_sms + 1) * mean
                                       : std::max(longest, all / num_sms + 0.5 * mean)) + (split ? kCrossSplitCost : 0);
            if (per_sm == 0 || cost < best) {
                best = cost;
                size = s;
            }
        }
    }
    for (int32_t b = 0; b < batch; ++b) {
        const int64_t rows = qo_indptr[b + 1] - qo_indptr[b];
        if (rows == 0 || few(rows * G, kv_len[b])) continue;
        const int64_t n = tiles_of(kv_len[b]), n_chunks = chunks_of(n, size);
        for (int64_t r0 = 0; r0 < rows; r0 += 2 * slot_rows) {
            const int64_t left = rows - r0;
            for (int32_t g = 0; g < Hkv; ++g) {
                PrefillItem it{};
                it.q_row0 = (int32_t)(qo_indptr[b] + r0);
                it.n_rows = (int32_t)(std::min(left, slot_rows) * G);
                it.reserved0 = left > slot_rows ? (int32_t)(std::min(left - slot_rows, slot_rows) * G) : 0;
                it.n_heads = it.reserved0 > 0 ? 2 : 1;
                it.kv_head = g;
                it.head0 = g * G;
                it.pos0 = -1;
                const int64_t partial0 = partials;
                for (int64_t c = 0; c < n_chunks; ++c) {
                    const int64_t t0 = c * n / n_chunks, t1 = (c + 1) * n / n_chunks;
                    it.page_base = (int32_t)(kv_start[b] + t0 * kPrefillKeys);
                    it.kv_len = (int32_t)(std::min<int64_t>(kv_len[b], t1 * kPrefillKeys) - t0 * kPrefillKeys);
                    it.key_end = it.kv_len;
                    it.n_kv_tiles = (int32_t)(t1 - t0);
                    it.reserved1 = (int32_t)c;
                    if (n_chunks > 1) {
                        plan->cross_chunks = true;
                        it.pos0 = (int32_t)partials;
                        partials += it.n_heads * (kPrefillRows / kMaxSliceHeads);
                        if (partials > INT32_MAX / kMaxSliceHeads) return ATTN_ERR_UNSUPPORTED;
                    }
                    plan->items.push_back(it);
                }
                for (int i = 0; n_chunks > 1 && i < it.n_heads; ++i) {
                    const int32_t pairs = i ? it.reserved0 : it.n_rows;
                    for (int32_t p = 0; p < pairs; p += kCrossBlock)
                        add_merge(*plan, {(int32_t)(it.q_row0 + i * slot_rows), it.head0, p, std::min(kCrossBlock, pairs - p),
                                          (int32_t)(partial0 + (i * kPrefillRows + p) / kMaxSliceHeads), (int32_t)n_chunks,
                                          it.n_heads * (kPrefillRows / kMaxSliceHeads), 0});
                }
            }
        }
    }
    plan->n_partials = (int32_t)partials;
    deal_prefill_items(plan.get());

    WorkspaceLayout& L = plan->layout;
    size_t off = 0;
    L.units = off;    off = align_up(off + plan->units.size() * sizeof(DecodeUnit), 256);
    L.items = off;    off = align_up(off + plan->items.size() * sizeof(PrefillItem), 256);
    L.append = off;   off = align_up(off + plan->append_slots.size() * sizeof(int32_t), 256);
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
    I.num_decode_groups_split = plan->cross_merges;
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
