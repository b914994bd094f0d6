// Accumulated attention weight per cached key.
//
//   w[t, g] = decay * prev[t, g] + sum over the plan's query rows i that see
//             key t and over the query heads h of KV head g of exp(s_ith - lse_ih),
//   s_ith = sm_scale * q_ih . k_tg;  tokens appended by this plan (t >= kv_len -
//   qo_len) have no previous weight.
//
// With the rows' lse known there is no running max and nothing to rescale: one
// product, one exponential and one sum per (row, head, key).  Keys are the rows
// of every product (S^T = K Q^T), so that a key's sum stays with one thread (or
// four lanes) and no atomics are needed: the sums' order is fixed.
//
// Two kernels, by the kind of request:
//  * decode requests (one query row): bound by reading K, 2 D (bf16) or 9 D / 16
//    (4 bits) bytes per key and head.  The plan's decode units, four warps each
//    with a ring of stages (32 tokens, 64 of 4 bits), mma.sync with the heads as
//    columns.  64 requests of 1K-8K tokens, 8 heads of 64 dims in bf16 (339 MB):
//    57 us, 5.9 TB/s, 0.88 of a copy's rate.  32 of 2K-32K, 4 heads of 128 dims,
//    16 query heads each, in 4 bits (163 MB): 40 us, 4.0 TB/s; there turning the
//    codes into operands takes over half of the issue slots.
//  * prefill requests: bound by the exponentials (MUFU: 32 a clock and SM) and
//    the product on the tensor cores.  One CTA per 128 keys of a KV head keeps
//    the K tile in shared memory and streams Q tiles past it, 128 columns of some
//    rows' heads (so that few rows with many heads fill them); tcgen05.mma fills
//    a ring of 128-column accumulators in TMEM ahead of the warpgroups that drain
//    them, one key per thread.  Four prompts of 0.5K-4K tokens, 64 query heads of
//    64 dims: 190 us, where the exponentials of whole tiles take 119 us at the
//    MUFU's rate and the products 73 us.  A CTA starts for some 5,000 clocks
//    (TMEM, K, the first lse), 4.2 times per SM; its steps take 770 instead of
//    the MUFU's 512: the barriers and TMEM loads alone measure 600, and overlap
//    with the exponentials in part.  Steps of 128 rows of one head measured 200
//    us where this form then took 193, but lost less with head counts that leave
//    columns of these steps empty (prompts with 12 heads per KV head 302 us
//    instead of 313, with 5 heads 135 instead of 138); so built, two warpgroups
//    223 and four 252 (fewer registers each), steps of two heads (N = 256) with
//    four warpgroups on 64 columns each 228, the next step's first columns loaded
//    ahead 209, and a query row per thread with a sum of 128 keys in registers 297.
//
// More than 16 query heads per KV head on decode rows take Q from memory again
// for every 16 tokens: 64 requests of 4096 tokens, 2 KV heads with 32 query heads
// of 64 dims, 56 us in bf16 (67 MB) and 70 in 4 bits, bound by that, not by K.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "attn_internal.h"
#include "kernels.h"
#include "kv4_stage.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct KeyWeightArgs {
    const DecodeUnit* units;
    const int32_t* page_table;
    const __nv_bfloat16* q;
    const float* lse;
    const uint8_t* pool;
    const float* prev;
    float* weights;
    int32_t* err;
    int32_t Hq, Hkv, P, page_log2, num_pages, causal, window;   // P = 1 << page_log2
    float scale_log2, decay;    // scale_log2 = sm_scale * log2(e) * k_scale
};

// The 128-key tiles of the prefill requests.
struct WeightTiles {
    const WeightRun* runs;
    const int32_t* starts;      // the runs' first tiles
    const uint32_t* hints;      // the run of every 32nd tile
    int32_t n_runs, tile0;      // tile0: the first tile of this launch
};

// ------------------------------------------------------------ decode requests

// kFour: 4-bit pages, else bf16.
template <int D, bool kFour>
struct StepWeightCfg {
    static constexpr int kWarps = kDecodeWarps;
    static constexpr int kTile = kFour ? 64 : 32;                        // tokens per stage
    static constexpr int kStages = kFour ? 2 : D == 64 ? 4 : 3;
    static constexpr int kSubs = kTile / kBlockTokens;
    static constexpr int kSub = kFour ? kv4_sub_bytes(D) : kBlockTokens * D * 2;   // K of 16 tokens
    static constexpr int kPrev = kSubs * kSub;                           // then the tokens' previous weights
    static constexpr int kStageBytes = kPrev + kTile * 4;
    static constexpr int kPipeBytes = kWarps * kStages * kStageBytes;
    static constexpr int kPageBytes = (kDecodeMaxChunkPages * 4 + 15) / 16 * 16;
    static constexpr int kSmem = 128 + kPipeBytes + 2 * kPageBytes;
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32"
        " {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight query heads (head0 ..; those from n on count nothing) as column
// operand, and per column 2 tq + e the factor and the (negated) lse in log2
// units that turn a product into the exponent.
template <int D, bool kFour>
struct QueryTile {
    uint32_t b[D / 16][2];
    float mult[2], nl[2];
    __device__ __forceinline__ void load(const KeyWeightArgs& a, int row, int head0, int n, int gq, int tq) {
        const int64_t at = (int64_t)row * a.Hq + head0;
        float inv = 1.f;
        if constexpr (kFour) {
            kv4_load_q<D>(gq < n ? a.q + (at + gq) * D : nullptr, tq, b, inv);
        } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    b[kk][j] = gq < n ? *reinterpret_cast<const uint32_t*>(a.q + (at + gq) * D + 16 * kk + 8 * j + 2 * tq) : 0u;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = 2 * tq + e;
            mult[e] = kFour ? __shfl_sync(0xffffffffu, inv, h * 4) * a.scale_log2 : a.scale_log2;
            nl[e] = h < n ? -a.lse[at + h] * kLog2e : -INFINITY;
        }
    }
};

// NT: column tiles of 8 heads held in registers; 0: more than 16 heads, taken
// from memory tile by tile.
template <int D, bool kFour, int NT>
__global__ void __launch_bounds__(kDecodeWarps * 32)
key_weights_step_kernel(const KeyWeightArgs a) {
    using C = StepWeightCfg<D, kFour>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-ptx::smem_u32(smem_raw) & 127u);
    uint32_t* first_s = reinterpret_cast<uint32_t*>(smem + C::kPipeBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gq = lane >> 2, tq = lane & 3;
    const DecodeUnit u = a.units[blockIdx.x];   // uploaded before the kernels this one may overlap
    ptx::grid_dependency_wait();
    const int G = a.Hq / a.Hkv, P = a.P;
    if (u.head0 != u.kv_head * G) return;   // the unit of the first head slice takes all heads
    const int first_page = u.tok_begin >> a.page_log2;
    const int n_pages = ((u.tok_end - 1) >> a.page_log2) - first_page + 1;
    load_sixteens(first_s, a.page_table + u.page_base + first_page, n_pages, a.num_pages, a.Hkv, u.kv_head, a.page_log2, a.err);
    uint32_t* block_s = first_s + C::kPageBytes / 4;   // (page, head) block of the weights
    for (int i = tid; i < n_pages; i += blockDim.x) {
        const int page = a.page_table[u.page_base + first_page + i];
        block_s[i] = page < 0 || page >= a.num_pages ? kBadPage : (uint32_t)(page * a.Hkv + u.kv_head);
    }
    __syncthreads();

    const uint8_t* ring = smem + warp * C::kStages * C::kStageBytes;
    const uint32_t ring_u32 = ptx::smem_u32(ring);
    const int n_tiles = (u.tok_end - u.tok_begin + C::kTile - 1) / C::kTile;
    const int n_it = n_tiles > warp ? (n_tiles - warp + C::kWarps - 1) / C::kWarps : 0;
    auto tile_tok = [&](int it) { return u.tok_begin + (warp + it * C::kWarps) * C::kTile; };
    const TileSource src = tile_source<D, kFour, C::kTile>(a.pool, first_s, first_page, a.page_log2, a.Hkv, lane);
    // Each lane takes one of every 32 of a tile's tokens: sixteen tq >> 1, row
    // (tq & 1) * 8 + its own.  slot: where a token's weight lies, or -1.
    const int row = kFour ? kv4_row(gq) : gq;
    const int mine = (tq >> 1) * kBlockTokens + (tq & 1) * 8 + row;
    auto slot = [&](int tok) -> int64_t {
        const uint32_t block = tok < u.tok_end ? block_s[(tok >> a.page_log2) - first_page] : kBadPage;
        return block == kBadPage ? -1 : ((int64_t)block << a.page_log2) + (tok & (P - 1));
    };
    // The one new token of a decode request, its last, has no previous weight.
    const int prev_end = a.decay == 0.f ? 0 : u.tok_end - (u.chunk == u.n_chunks - 1);
    auto issue = [&](int it, int s) {   // one group per stage, empty past the end
        const uint32_t dst = ring_u32 + s * C::kStageBytes;
        if (it < n_it) {
#pragma unroll
            for (int t = 0; t < C::kTile; t += 32) {
                const int64_t at = slot(tile_tok(it) + t + mine);
                const bool old = at >= 0 && tile_tok(it) + t + mine < prev_end;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                             ::"r"(dst + C::kPrev + (t + lane) * 4), "l"(a.prev + (old ? at : 0)), "r"(old ? 4 : 0) : "memory");
            }
            if constexpr (kFour) kv4_stage_load<D, C::kTile, 1>(src, tile_tok(it), u.tok_end, dst, lane);
            else bf16_stage_load<D, C::kTile>(src, tile_tok(it), u.tok_end, dst, lane);
        }
        cp_async_commit();
    };
    for (int it = 0; it < C::kStages; ++it) issue(it, it);

    constexpr int kHeld = NT > 0 ? NT : 1;
    QueryTile<D, kFour> qt[kHeld];
    if constexpr (NT > 0)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) qt[nt].load(a, u.q_row, u.head0 + nt * 8, G - nt * 8, gq, tq);

    // Scores of 16 tokens (two of them this lane's rows) against the held tiles
    // of heads, exponentiated and added to w.
    auto add_sub = [&](const uint8_t* sub, float (&w)[2]) {
        float s[kHeld][4];
#pragma unroll
        for (int nt = 0; nt < kHeld; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        if constexpr (kFour) {
            kv4_for_k<D>(sub, kv4_row(gq), tq, [&](int kk, const uint32_t (&ka)[4]) {
#pragma unroll
                for (int nt = 0; nt < kHeld; ++nt) mma_f16_16816(s[nt], ka, qt[nt].b[kk][0], qt[nt].b[kk][1]);
            });
        } else {
            const uint32_t at = ptx::smem_u32(sub);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const int mi = lane >> 3, row = (mi & 1) * 8 + (lane & 7), ch = 2 * kk + (mi >> 1);
                uint32_t ka[4];
                ptx::ldmatrix_x4(at + (ch >> 3) * (kBlockTokens * 128) + row * 128 + (((ch & 7) ^ (lane & 7)) << 4), ka[0],
                                 ka[1], ka[2], ka[3]);
#pragma unroll
                for (int nt = 0; nt < kHeld; ++nt) ptx::mma_bf16_16816(s[nt], ka, qt[nt].b[kk][0], qt[nt].b[kk][1]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < kHeld; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float nl = qt[nt].nl[e & 1], p = ptx::ex2(fmaf(s[nt][e], qt[nt].mult[e & 1], nl));
                // A column without a head is 0 also where the key holds infinities (4 bits cannot).
                w[e >> 1] += !kFour && nl == -INFINITY ? 0.f : p;
            }
    };

    for (int it = 0, s = 0; it < n_it; ++it) {
        cp_async_wait<C::kStages - 1>();
        __syncwarp();   // every lane's copies of this stage have landed
        const uint8_t* kt = ring + s * C::kStageBytes;
        float w[C::kSubs][2];
#pragma unroll
        for (int sub = 0; sub < C::kSubs; ++sub) {
            w[sub][0] = w[sub][1] = 0.f;
            if constexpr (NT > 0) {
                add_sub(kt + sub * C::kSub, w[sub]);
            } else {
                for (int h = 0; h < G; h += 8) {
                    qt[0].load(a, u.q_row, u.head0 + h, G - h, gq, tq);
                    add_sub(kt + sub * C::kSub, w[sub]);
                }
            }
        }
        float before[C::kTile / 32];
#pragma unroll
        for (int t = 0; t < C::kTile / 32; ++t)
            before[t] = *reinterpret_cast<const float*>(kt + C::kPrev + (t * 32 + lane) * 4);
        __syncwarp();   // every lane has read the stage
        issue(it + C::kStages, s);
        s = s + 1 == C::kStages ? 0 : s + 1;
        // Sums over the four lanes of a key row, each of which ends with one token's.
#pragma unroll
        for (int t = 0; t < C::kTile / 32; ++t) {
            float v[2];
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                const float(&x)[2] = w[2 * t + sub];
                const float keep = tq & 1 ? x[1] : x[0], give = tq & 1 ? x[0] : x[1];
                v[sub] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
            }
            const float keep = tq & 2 ? v[1] : v[0], give = tq & 2 ? v[0] : v[1];
            const float sum = keep + __shfl_xor_sync(0xffffffffu, give, 2);
            const int64_t at = slot(tile_tok(it) + t * 32 + mine);
            if (at >= 0) a.weights[at] = fmaf(a.decay, before[t], sum);
        }
    }
    // Only now: CTAs of the next grid that start while this one is in its loop
    // crowd onto the SMs that are done first.
    ptx::grid_dependents_go();
}

// ----------------------------------------------------------- prefill requests

constexpr int kTileKeys = kWeightTileKeys;   // 128 keys per CTA: the MMA's M, a TMEM lane each
constexpr int kTileRows = kWeightTileRows;   // 128 columns per step: the MMA's N

// A wait with the same result in every lane of the warp.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity));
}

// Two forms.  The long one has an SM for itself and hides a step's latencies by
// steps in flight; a CTA of few steps is mostly start and end, which the short
// one hides by its several CTAs per SM, where there are that many.
template <int D, bool kShort>
struct PromptWeightCfg {
    static constexpr int kAtom = 128 * 128;                 // 128 rows x 64 dims, 128-byte swizzle
    static constexpr int kTile = kAtom * (D / 64);
    // Q stages: a stage's round trip (refill noticed, copied, multiplied) is
    // some 2,000 clocks, so many must be on their way at once.
    static constexpr int kStages = kShort ? 2 : D == 64 ? 10 : 5;
    static constexpr int kBufs = kShort ? 1 : 4;            // S accumulators: 128 of the 512 TMEM columns each
    static constexpr int kWgs = kShort ? 1 : 3;             // epilogue warpgroups
    static constexpr int kCtas = kShort ? weight_short_ctas(D) : 1;   // per SM
    static constexpr int kEpilogueWarps = 4 * kWgs;
    static constexpr int kThreads = (kEpilogueWarps + 3) * 32;   // + MMA issuer, + Q producer, + lse
    static constexpr int kGroup = kShort ? 4 : 8;           // steps whose lse is staged at a time
    static constexpr int kOffQ = kTile;
    static constexpr int kOffNl = kOffQ + kStages * kTile;    // [2][kGroup steps][128 columns] negated lse
    static constexpr int kOffSum = kOffNl + 2 * kGroup * kTileRows * 4;
    static constexpr int kOffBars = kOffSum + kWgs * kTileKeys * 4;
    static constexpr int kSmem = 1024 + kOffBars + (2 * kStages + kBufs + 6) * 8 + 16;
    static_assert(kCtas * (kSmem + 1024) <= 233472 && kSmem <= 232448 && kCtas * kBufs * kTileRows <= 512, "CTAs per SM");
    // The long form holds all of an SM's TMEM, and a second CTA would wait for it.
    static_assert(kShort || 2 * (kSmem + 1024) > 233472, "one CTA per SM");
    // s_full is waited on by stage: step s + kStages must not complete before
    // step s's S has been read.  The one MMA warp takes the steps in order, and
    // step s + kBufs needs the accumulator of step s.
    static_assert(kStages >= kBufs, "s_full phases");
};

// kRagged: a number of heads that leaves some of a step's last 32 columns empty.
template <int D, bool kFour, bool kShort, bool kRagged>
__global__ void __launch_bounds__(PromptWeightCfg<D, kShort>::kThreads, PromptWeightCfg<D, kShort>::kCtas)
key_weights_prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kv_map,
                          const KeyWeightArgs a, const WeightTiles w) {
    using C = PromptWeightCfg<D, kShort>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-ptx::smem_u32(smem_raw) & 1023u);
    const uint32_t sbase = ptx::smem_u32(smem);
    // Step s uses Q stage s % kStages and S accumulator s % kBufs.  s_full (by
    // stage): the product is done, S may be read and the stage refilled; s_free
    // (by accumulator): S has been read.
    const uint32_t q_full = sbase + C::kOffBars, s_full = q_full + 8 * C::kStages, s_free = s_full + 8 * C::kStages;
    const uint32_t l_full = s_free + 8 * C::kBufs, l_free = l_full + 16, k_full = l_free + 16, drain = k_full + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBars + (2 * C::kStages + C::kBufs + 6) * 8);
    float* nl_s = reinterpret_cast<float*>(smem + C::kOffNl);
    float* sum_s = reinterpret_cast<float*>(smem + C::kOffSum);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // The tile's run: the hint's, or the last of the 32 from there on that begins at or before it.
    const int tile = w.tile0 + blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv;
    const uint32_t hint = w.hints[tile / kWeightHintTiles];
    int at_run = (int)(hint & ~kWeightHintAll);
    if (!(hint & kWeightHintAll)) {
        const bool begun = at_run + lane < w.n_runs && w.starts[min(at_run + lane, w.n_runs - 1)] <= tile;
        at_run += __popc(__ballot_sync(0xffffffffu, begun)) - 1;
    }
    const WeightRun run = w.runs[at_run];
    const int t0 = run.key0 + (tile - run.tile0) * kTileKeys;
    const RequestInfo r = run.request;
    const int G = a.Hq / a.Hkv, P = a.P, prefix = r.kv_len - r.qo_len;
    // First query row that counts: inside the window, and seeing the first key.
    int i0 = a.window > 0 ? max(0, r.qo_len - a.window) : 0;
    if (a.causal) i0 = max(i0, t0 - prefix);
    // A step's 128 columns: `rows` query rows, `heads` heads of each side by side
    // (a row's heads lie together in q and in lse); more than 128 heads in slices.
    const int heads = min(G, kTileRows), rows = kTileRows / heads, used = rows * heads;
    const int slices = (G + heads - 1) / heads;
    const int n_steps = (r.qo_len - i0 + rows - 1) / rows * slices;
    const int n_groups = (n_steps + C::kGroup - 1) / C::kGroup;

    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            ptx::mbar_init(q_full + 8 * i, 1);
            ptx::mbar_init(s_full + 8 * i, 1);
        }
        for (int i = 0; i < C::kBufs; ++i) ptx::mbar_init(s_free + 8 * i, 4);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(l_full + 8 * i, 1);
            ptx::mbar_init(l_free + 8 * i, C::kEpilogueWarps);
        }
        ptx::mbar_init(k_full, kFour ? C::kEpilogueWarps : 1);
        ptx::mbar_init(drain, 1);
        ptx::fence_mbar_init();
    }
    if (warp == C::kEpilogueWarps) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::kBufs * kTileRows);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::grid_dependents_go();     // with this grid's TMEM in hand: a dependent that allocates too waits for it
    ptx::grid_dependency_wait();   // up to here only the plan's own lists were read

    if (warp == C::kEpilogueWarps + 1) {
        // ------------------------------------------------------------ producer
        if (!kFour) {
            const int n_load = (min(kTileKeys, r.kv_len - t0) + P - 1) / P;   // page boxes of the K tile
            int page = -1;
            if (lane < n_load) {
                page = a.page_table[r.page_base + t0 / P + lane];
                if (page < 0 || page >= a.num_pages) {
                    atomicOr(a.err, ATTN_DEVICE_ERR_PAGE_ID);
                    page = -1;
                }
            }
            const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, page >= 0)) * (D / 64);
            if (lane == 0) ptx::mbar_arrive_expect_tx(k_full, boxes * P * 128);
            __syncwarp();
            if (page >= 0)
                for (int c = 0; c < D / 64; ++c)
                    ptx::tma_load_3d(sbase + c * C::kAtom + lane * P * 128, &kv_map, k_full, c * 64, 0,
                                     page * 2 * a.Hkv + g);
        }
        if (lane == 0) {
            int s = 0;   // steps whose q is on its way
            for (int h0 = 0, row = r.q_row0 + i0; s < n_steps; ++s) {
                const int st = s % C::kStages;
                if (s >= C::kStages && !ptx::mbar_wait(s_full + 8 * st, (s / C::kStages - 1) & 1)) {
                    atomicOr(a.err, ATTN_DEVICE_ERR_TIMEOUT);
                    break;
                }
                ptx::mbar_arrive_expect_tx(q_full + 8 * st, used * 128 * (D / 64));
                for (int c = 0; c < D / 64; ++c)
                    ptx::tma_load_3d(sbase + C::kOffQ + st * C::kTile + c * C::kAtom, &q_map, q_full + 8 * st, c * 64,
                                     g * G + h0, row);
                h0 += heads;
                if (h0 >= G) {
                    h0 = 0;
                    row += rows;
                }
            }
            ptx::await_copies(q_full, C::kStages, s);
            if (!kFour) ptx::await_copies(k_full, 1, 1);
        }
        __syncwarp();
    } else if (warp == C::kEpilogueWarps + 2) {
        // ----------------------------------------------------------------- lse
        // This warp stages kGroup steps' lse (negated, in log2 units) at a time, ahead of them.
        // Of this lane's columns: row within the step (huge: none), head, index in lse
        // (below 2^31: the plan's rows times heads are).
        int row_of[kTileRows / 32], head_of[kTileRows / 32], at[kTileRows / 32];
#pragma unroll
        for (int q = 0; q < kTileRows / 32; ++q) {
            const int col = q * 32 + lane;
            row_of[q] = col < used ? col / heads : 1 << 30;
            head_of[q] = col % heads;
            at[q] = col < used ? (r.q_row0 + col / heads) * a.Hq + g * G + head_of[q] : 0;
        }
        int row0 = i0, h0 = 0;
        auto fetch = [&](float (&v)[C::kGroup][kTileRows / 32]) {   // the next group's; past the last step nothing is read
#pragma unroll
            for (int k = 0; k < C::kGroup; ++k) {
#pragma unroll
                for (int q = 0; q < kTileRows / 32; ++q)
                    v[k][q] = row_of[q] < r.qo_len - row0 && head_of[q] < G - h0 ? a.lse[at[q] + (row0 * a.Hq + h0)] : INFINITY;
                h0 += heads;
                if (h0 >= G) {
                    h0 = 0;
                    row0 += rows;
                }
            }
        };
        float v[C::kGroup][kTileRows / 32], next[C::kGroup][kTileRows / 32];   // two groups' loads on their way
        fetch(v);
        for (int grp = 0; grp < n_groups; ++grp) {
            float* dst = nl_s + (grp & 1) * C::kGroup * kTileRows + lane;
            if (grp + 1 < n_groups) fetch(next);
            if (grp >= 2 && !wait_all(l_free + 8 * (grp & 1), ((grp >> 1) - 1) & 1)) {
                if (lane == 0) atomicOr(a.err, ATTN_DEVICE_ERR_TIMEOUT);
                break;
            }
#pragma unroll
            for (int k = 0; k < C::kGroup; ++k)
#pragma unroll
                for (int q = 0; q < kTileRows / 32; ++q) {
                    dst[k * kTileRows + q * 32] = -v[k][q] * kLog2e;
                    v[k][q] = next[k][q];
                }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(l_full + 8 * (grp & 1));
        }
    } else if (warp == C::kEpilogueWarps) {
        // ---------------------------------------------------------- MMA issuer
        // One thread, with the descriptors made beforehand: its loop lies between
        // an S that is released and the next one that is ready.
        constexpr uint32_t idesc = ptx::idesc_bf16(kTileKeys, kTileRows, false, false);
        if (lane == 0) {
            const uint64_t a0 = ptx::smem_desc_sw128(sbase, 16, 1024), b0 = ptx::smem_desc_sw128(sbase + C::kOffQ, 16, 1024);
            bool ok = ptx::mbar_wait(k_full, 0);
            int st = 0, buf = 0;
            uint32_t full = 0, free = 1;   // phases: of Q's stages, and of the accumulators (first use: none to wait for)
            for (int s = 0; ok && s < n_steps; ++s) {
                ok = ptx::mbar_wait(q_full + 8 * st, full) && ptx::mbar_wait(s_free + 8 * buf, free);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint64_t b = b0 + (uint32_t)(st * (C::kTile >> 4));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = kk / 4 * (C::kAtom >> 4) + kk % 4 * 2;   // in 16 bytes
                    ptx::tc_mma_ss(tmem + buf * kTileRows, a0 + off, b + off, idesc, kk > 0);
                }
                ptx::tc_commit(s_full + 8 * st);
                if (++st == C::kStages) {
                    st = 0;
                    full ^= 1;
                }
                if (++buf == C::kBufs) {
                    buf = 0;
                    free ^= 1;
                }
            }
            if (!ok) atomicOr(a.err, ATTN_DEVICE_ERR_TIMEOUT);
            ptx::tc_commit(drain);
        }
        __syncwarp();
    } else {
        // ------------------------------------------- epilogue: one key per thread
        const int wg = warp >> 2, key = (warp & 3) * 32 + lane;   // warpgroup wg takes steps wg, wg + kWgs, ...
        if (kFour) {
            // The K tile: codes and scales to bf16 (exact), in the swizzled
            // layout TMA would have given a bf16 page.
            constexpr int kGroups = D / kKv4Group;
            for (int idx = tid; idx < kTileKeys * kGroups; idx += C::kEpilogueWarps * 32) {
                const int k = idx / kGroups, grp = idx % kGroups, t = t0 + k;
                if (t >= r.kv_len) break;
                const int page = a.page_table[r.page_base + t / P];
                if (page < 0 || page >= a.num_pages) {
                    atomicOr(a.err, ATTN_DEVICE_ERR_PAGE_ID);
                    continue;
                }
                const uint8_t* sub = a.pool + kv4::sub_offset(page, 0, a.Hkv, g, P, t % P, kv4_sub_bytes(D));
                const int in = t % kKv4Tokens;
                const uint2 codes = *reinterpret_cast<const uint2*>(sub + in * (D / 2) + grp * 8);
                const float sc = kv4::f16x2_to_f32(kv4::scales_to_f16x2(sub[8 * D + in * kGroups + grp])).x;
                uint32_t h[2][4], o[8];
                kv4::codes_to_f16x2(codes.x, h[0]);
                kv4::codes_to_f16x2(codes.y, h[1]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 v = kv4::f16x2_to_f32(h[j >> 2][j & 3]);
                    o[j] = ptx::pack_bf16x2(v.x * sc, v.y * sc);
                }
                const uint32_t at = sbase + (grp / 4) * C::kAtom + k * 128;
                const int ch = (grp % 4) * 2;
                ptx::st_shared_v4(at + ((ch ^ (k & 7)) << 4), o[0], o[1], o[2], o[3]);
                ptx::st_shared_v4(at + (((ch + 1) ^ (k & 7)) << 4), o[4], o[5], o[6], o[7]);
            }
            ptx::fence_proxy_async_smem();   // the MMA reads it through the async proxy
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(k_full);
        }
        const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
        // Adds 2^(s scale - lse) over 32 columns; masked: over those in [lo, hi) alone.
        auto add_columns = [&](auto masked, const uint32_t (&v)[32], uint32_t nl_at, int lo, int hi) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                float4 l4;
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(l4.x), "=f"(l4.y), "=f"(l4.z), "=f"(l4.w) : "r"(nl_at + k * 4));
                const float2 x0 = ptx::fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), scale2,
                                            make_float2(l4.x, l4.y));
                const float2 x1 = ptx::fma2(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), scale2,
                                            make_float2(l4.z, l4.w));
                float2 p0 = make_float2(ptx::ex2(x0.x), ptx::ex2(x0.y));
                float2 p1 = make_float2(ptx::ex2(x1.x), ptx::ex2(x1.y));
                if constexpr (decltype(masked)::value) {
                    const uint32_t n = (uint32_t)(hi - lo);   // unsigned: one comparison for both ends
                    p0.x = (uint32_t)(k - lo) < n ? p0.x : 0.f;
                    p0.y = (uint32_t)(k + 1 - lo) < n ? p0.y : 0.f;
                    p1.x = (uint32_t)(k + 2 - lo) < n ? p1.x : 0.f;
                    p1.y = (uint32_t)(k + 3 - lo) < n ? p1.y : 0.f;
                }
                acc0 = ptx::add2(acc0, p0);
                acc1 = ptx::add2(acc1, p1);
            }
        };

        float total = 0.f;
        bool ok = true;
        int s = wg;   // this warpgroup's next step
        auto released = [&](int buf) {   // all of S has been read: a later product may overwrite it
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(s_free + 8 * buf);
        };
        // Row seen0 is the first that sees the warp's first key.  Steps [clear, whole)
        // count in full: all columns, of rows that see all of the warp's keys and are
        // the request's.
        const int seen0 = t0 + (key - lane) - prefix;
        const int clear = a.causal ? (max(0, seen0 + 31 - i0) + rows - 1) / rows : 0;
        const int whole = slices == 1 && (kRagged ? used > 96 : used == kTileRows) ? (r.qo_len - i0) / rows : 0;
        for (int grp = 0; grp < n_groups; ++grp) {
            ok = ok && wait_all(l_full + 8 * (grp & 1), (grp >> 1) & 1);
            for (const int end = min(n_steps, (grp + 1) * C::kGroup); s < end; s += C::kWgs) {
                // After a wait that ran out the warp only keeps the barriers' count.
                const int buf = s % C::kBufs;
                ok = ok && wait_all(s_full + 8 * (s % C::kStages), (s / C::kStages) & 1);
                if (!ok) continue;
                ptx::tc_fence_after();
                const uint32_t nl_at = ptx::smem_u32(nl_s) + s % (2 * C::kGroup) * kTileRows * 4;
                const uint32_t t_s = t_lane + buf * kTileRows;
                if (s >= clear && s < whole) {
                    uint32_t v[2][32];   // 32 columns at a time, the next ones on their way
                    ptx::tmem_ld32(t_s, v[0]);
                    ptx::tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < kTileRows / 32; ++c) {
                        if (c + 1 < kTileRows / 32) ptx::tmem_ld32(t_s + (c + 1) * 32, v[(c + 1) & 1]);
                        if (kRagged && c == 3) add_columns(std::true_type{}, v[1], nl_at + 3 * 128, 0, used - 96);
                        else add_columns(std::false_type{}, v[c & 1], nl_at + c * 128, 0, 32);
                        if (c + 1 < kTileRows / 32) ptx::tc_wait_ld();
                        if (c + 2 == kTileRows / 32) released(buf);
                    }
                } else {
                    // Columns [lo, hi) count: rows that see the key, of this request, and
                    // heads of this KV head.  Over the warp's keys lo rises by 31 rows.
                    const int block = s / slices, row0 = i0 + block * rows;
                    const int hi = slices == 1 ? min(rows, r.qo_len - row0) * heads : min(heads, G - (s - block * slices) * heads);
                    const int seen = a.causal ? seen0 - row0 : -32;
                    const int lo = max(0, seen + (a.causal ? lane : 0)) * heads;
                    const int lo0 = max(0, seen) * heads, lo31 = max(0, seen + 31) * heads;
#pragma unroll 1
                    for (int c = 0; c < kTileRows; c += 32) {
                        if (c + 32 < kTileRows && c + 31 < lo0) continue;   // no key of the warp is seen
                        uint32_t v[32];
                        ptx::tmem_ld32(t_s + c, v);
                        ptx::tc_wait_ld();
                        if (c + 32 == kTileRows) released(buf);
                        if (lo31 <= c && hi >= c + 32) add_columns(std::false_type{}, v, nl_at + c * 4, 0, 32);
                        else add_columns(std::true_type{}, v, nl_at + c * 4, max(0, lo - c), max(max(0, lo - c), min(32, hi - c)));
                    }
                }
                total += (acc0.x + acc0.y) + (acc1.x + acc1.y);
                acc0 = acc1 = make_float2(0.f, 0.f);
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(l_free + 8 * (grp & 1));
        }
        if (!ok && lane == 0) atomicOr(a.err, ATTN_DEVICE_ERR_TIMEOUT);
        // The warpgroups' sums, in a fixed order.
        sum_s[wg * kTileKeys + key] = total;
        asm volatile("bar.sync 3, %0;" ::"n"(C::kEpilogueWarps * 32) : "memory");
        const int t = t0 + key;
        if (wg == 0 && t < r.kv_len) {
            const int page = a.page_table[r.page_base + t / P];
            if (page >= 0 && page < a.num_pages) {
                const int64_t at = ((int64_t)page * a.Hkv + g) * P + t % P;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < C::kWgs; ++i) sum += sum_s[i * kTileKeys + key];
                if (a.decay != 0.f && t < prefix) sum = fmaf(a.decay, a.prev[at], sum);
                a.weights[at] = sum;
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == C::kEpilogueWarps) {
        ptx::mbar_wait(drain, 0);
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::kBufs * kTileRows);
    }
}

template <int D, bool kFour, int NT>
cudaError_t launch_step(const KeyWeightArgs& a, int grid, cudaStream_t stream) {
    using C = StepWeightCfg<D, kFour>;
    auto kernel = key_weights_step_kernel<D, kFour, NT>;
    static std::atomic<bool> configured[kMaxDevices];
    cudaError_t e = once_per_device(configured, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(grid), kDecodeWarps * 32, C::kSmem, stream, a);
}

template <int D, bool kFour, bool kShort, bool kRagged>
cudaError_t launch_prompt(const CUtensorMap& q_map, const CUtensorMap& kv_map, const KeyWeightArgs& a,
                          const WeightTiles& w, int grid, cudaStream_t stream) {
    using C = PromptWeightCfg<D, kShort>;
    auto kernel = key_weights_prompt_kernel<D, kFour, kShort, kRagged>;
    static std::atomic<bool> configured[kMaxDevices];
    cudaError_t e = once_per_device(configured, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(grid), C::kThreads, C::kSmem, stream, q_map, kv_map, a, w);
}

// Which form (WeightLoad::takes_short_form).  Short / long time of some last rows
// on one context, 8 KV heads with 8 query heads each, bf16, by CTAs (down) and
// steps per tile:
//             D = 64:   4     16    32    64      D = 128:  4     16    32    64
//     64              1.24  1.78  1.81  1.84              1.22  1.80  1.71  1.64
//    152              1.26  1.72  1.78  1.81              1.25  1.58  1.54  1.55
//    304              0.84  1.10  1.18  1.25              0.84  1.05  1.08  1.09
//    456              0.75  1.05  1.23  1.38              0.94  1.18  1.20  1.20
//    608              0.61  0.84  0.95  1.05              0.79  0.96  1.01  1.05
//   1216              0.53  0.78  0.90  1.00              0.72  0.90  0.98  1.02
//   3000              0.47  0.70  0.83  0.94              0.65  0.84  0.91  0.98
// With no more CTAs than SMs the long form is ahead (its three warpgroups against
// one); with more the short one, for the more steps the more of its CTAs share an
// SM; beyond 64 steps it is behind in any number (128 steps, 1000 CTAs: 1.05 and
// 1.03).  With 4 bits the ratios are up to 0.15 higher.
//
// A batch goes by its mean, in one launch, but where the few tiles of a prompt
// would outlast all the others of the short form (WeightLoad::even; a lone short
// CTA takes 0.72 us a step, an SM full of them 0.46): there each kind is a launch.
// Microseconds in short form, long form, and apart, 2 KV heads with 8 query heads
// of 64 dims: a prompt of 8K beside 40 rows on 17K in 76 requests 445, 807, 479;
// in 30 requests 403, 370, 311; in 10, 395, 191, 235; in 2 (94 steps by the mean),
// 366, 192, 205; a prompt of 2K beside the 76 291, 731, 337.
template <int D, bool kFour>
attn_status launch_all(const attn_plan_s* plan, const CUtensorMap& q_map, const CUtensorMap& kv_map,
                       const KeyWeightArgs& a, cudaStream_t stream) {
    const int G = plan->Hq / plan->Hkv, units = (int)plan->units.size();
    cudaError_t e = cudaSuccess;
    if (units > 0)
        e = G <= 8    ? launch_step<D, kFour, 1>(a, units, stream)
            : G <= 16 ? launch_step<D, kFour, 2>(a, units, stream)
                      : launch_step<D, kFour, 0>(a, units, stream);
    if (e == cudaSuccess && plan->weight_tiles > 0) {
        const int all = plan->weight_tiles, split = plan->weight_long_tiles;
        WeightLoad load[2];   // the tiles before `split`, and from there on
        for (const RequestInfo& r : plan->requests)
            if (r.qo_len > 1) load[split == 0 || weight_steps(r.qo_len, G) <= kWeightShortSteps].add(r, G, a.window);
        bool is_short[2];
        for (int i = 0; i < 2; ++i) is_short[i] = load[i].takes_short_form(plan->Hkv, plan->num_sms, D);
        if (split == 0) is_short[0] = is_short[1];
        const bool ragged = kTileRows % std::min(G, kTileRows) != 0;
        WeightTiles w;
        w.runs = reinterpret_cast<const WeightRun*>(plan->lists + plan->lists_layout.weight_runs);
        w.starts = reinterpret_cast<const int32_t*>(plan->lists + plan->lists_layout.weight_starts);
        w.hints = reinterpret_cast<const uint32_t*>(plan->lists + plan->lists_layout.weight_hints);
        w.n_runs = (int32_t)plan->weight_runs.size();
        w.tile0 = 0;
        for (int end = is_short[0] == is_short[1] ? all : split; e == cudaSuccess && w.tile0 < all; w.tile0 = end, end = all) {
            const int grid = (end - w.tile0) * plan->Hkv;
            e = is_short[w.tile0 >= split] ? launch_prompt<D, kFour, true, false>(q_map, kv_map, a, w, grid, stream)
                : ragged                   ? launch_prompt<D, kFour, false, true>(q_map, kv_map, a, w, grid, stream)
                                           : launch_prompt<D, kFour, false, false>(q_map, kv_map, a, w, grid, stream);
        }
    }
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

attn_status launch_key_weights(attn_plan_s* plan, bool four, const void* q, const void* pool, float k_scale,
                               const void* q_map, const void* kv_map, const float* lse, const float* prev,
                               float decay, int32_t window, float* weights, cudaStream_t stream) {
    KeyWeightArgs a;
    a.units = reinterpret_cast<const DecodeUnit*>(plan->ws + plan->layout.units);
    a.page_table = plan->page_table;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.lse = lse;
    a.pool = static_cast<const uint8_t*>(pool);
    a.prev = prev ? prev : weights;   // a valid address; not read when decay is 0
    a.weights = weights;
    a.err = reinterpret_cast<int32_t*>(plan->ws + plan->layout.err);
    a.Hq = plan->Hq;
    a.Hkv = plan->Hkv;
    a.P = plan->P;
    a.page_log2 = 31 - __builtin_clz(plan->P);
    a.num_pages = plan->num_pages;
    a.causal = plan->causal;
    a.window = window;
    a.scale_log2 = plan->sm_scale * kLog2e * k_scale;
    a.decay = decay;
    const CUtensorMap& qm = *static_cast<const CUtensorMap*>(q_map);
    const CUtensorMap& km = *static_cast<const CUtensorMap*>(kv_map);
    if (plan->D == 64)
        return four ? launch_all<64, true>(plan, qm, km, a, stream) : launch_all<64, false>(plan, qm, km, a, stream);
    return four ? launch_all<128, true>(plan, qm, km, a, stream) : launch_all<128, false>(plan, qm, km, a, stream);
}

}  // namespace attn
