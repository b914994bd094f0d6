// Decode sink attention (qo_len = 1) over the 4-bit paged cache.
//
// The mathematics is attn_decode's (online softmax with one sink logit per
// query head in the denominator, split-KV chunks merged by log-sum-exp), over
// k = code * scale * k_scale and v = code * scale * v_scale.  A cached token
// costs 9 D / 8 bytes per KV head instead of 4 D, so the kernel has a quarter
// of the bytes to wait for and must spend few instructions on each value:
//
//  * S^T = K Q^T and O^T += V^T P^T (mma.sync m16n8k16, f16 -> fp32): tokens
//    (and then dims) are the 16 MMA rows and the GQA group's query heads the 8
//    columns, so that a group of 8 heads wastes no row, no exponential and no
//    accumulator; up to 16 heads take two column tiles;
//  * codes become f16 by cvt.e2m1x2 and are multiplied by their scale, also
//    f16: exact (kv4.cuh).  Q is scaled per head by a power of two into f16's
//    range (exact for values down to 2^-26 of the head's largest);
//  * both operands' inner orders are free as long as Q (and P) follow, so they
//    are chosen for the loads: a lane's K dims are D / 4 consecutive ones (one
//    8- or 16-byte shared load per token, and whole scale groups), its V dims
//    D / 8 consecutive ones of four tokens;
//  * P^T's fragment is S^T's transposed 8x8 blocks: two movmatrix per 16 tokens;
//  * the softmax shift moves only when a score passes it by 2^15 (any shift is
//    valid as long as P stays within f16), so a tile costs one vote instead of
//    a reduction over its lanes.
//
// Measured, inputs beyond the L2: 64 requests of 1K-8K tokens, 8 KV heads of 64
// dims (181 MB) 42.4 us, 4.3 TB/s; 256 of 0.5K-16K (1.29 GB) 220 us, 5.9 TB/s,
// 0.86 of a copy's rate; 32 of 2K-32K, 4 KV heads of 128 dims with 16 query heads
// each (293 MB) 76.8 us, 3.8 TB/s.  A large batch is bound by memory and the issue
// slots alike; a small one by what a unit does before and after its loop (page
// ids, first tile, merge) and the last wave; the 16-head form, with 230 registers
// and so eight warps per SM, by the latency of a warp's chain of products.
//
// One CTA = one decode unit of the plan (request, KV head, <= 16 query heads,
// KV chunk), four warps, each with its own ring of kTile-token stages filled
// by its own cp.async, so that no barrier sits in the streaming loop.
#include "attn_internal.h"
#include "kernels.h"
#include "kv4.cuh"
#include "kv4_stage.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// P is rounded to f16, as the tensor cores take V's exact values there: half a
// step is 2^-11 of a weight, an eighth of what rounding the output to bf16 may
// cost; the row sum takes P unrounded, in fp32.
// The softmax shift m lies kShift below the running max, so that P's largest is
// 2^7 and f16 is normal down to 2^-21 of it (its subnormals then cost 2^-32 of
// it at most); m moves when a score passes it by kSlack (P stays below 2^15).
constexpr float kShift = 7.f, kSlack = 15.f;   // log2 units

template <int D, int NT>
struct Decode4Cfg {
    static constexpr int kWarps = kDecodeWarps;
    // Tokens per stage, all of whose scores are held at once: independent
    // products hide more than further warps do (256 requests of 0.5K-16K tokens,
    // D = 64: 242 us with 32 tokens at a time and 20 warps per SM, 228 with 64,
    // 236 with 128 and 12 warps).
    static constexpr int kTile = 64;
    static constexpr int kStages = 2;
    // CTAs per SM, for the registers: with a bound the compiler spends what is
    // left on loads ahead.  Without one it took 96 where 123 fit (64 dims, up to
    // 8 heads): 44.7 us instead of 42.4 for 64 requests of 1K-8K; 16 heads of 128
    // dims 78.6 instead of 76.8 (204 registers, 230), 8 heads of 128 dims, 256
    // requests of 0.5K-8K, 190.5 instead of 185.8.
    static constexpr int kCtas = D == 64 ? (NT == 1 ? 4 : 3) : (NT == 1 ? 3 : 2);
    static constexpr int kSubs = kTile / kKv4Tokens;
    static constexpr int kSub = kv4_sub_bytes(D);
    static constexpr int kStageBytes = 2 * kSubs * kSub;              // K, then V
    static constexpr int kHeads = NT * 8;
    static constexpr int kRowStride = D + 8;                          // floats, combine buffers
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kPipeBytes = kWarps * kWarpBytes;
    static constexpr int kPageBytes = (kDecodeMaxChunkPages * 4 + 15) / 16 * 16;
    static constexpr int kStateBytes = (kWarps * 32 + kMaxSliceHeads) * 4 + 16;   // per-warp m, l (16 heads each), sinks, flag
    static constexpr int kSmem = kPipeBytes + kPageBytes + kStateBytes;
    static_assert(kHeads * kRowStride * 4 <= kWarpBytes, "a warp's state fits its ring");
};

struct Decode4Args {
    const DecodeUnit* units;
    const int32_t* page_table;
    const __nv_bfloat16* q;
    const uint8_t* pool;
    __nv_bfloat16* out;
    float* lse;
    const float* sinks;
    float* part_o;
    float* part_lse;
    int32_t* counters;
    int32_t* err;
    int32_t Hq, Hkv, page_log2, num_pages;
    float scale_log2;   // sm_scale * log2(e) * k_scale
    float v_scale;
};

// D[16x8] += A[16x16] * B[16x8], f16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32"
        " {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// D = A * B
__device__ __forceinline__ void mma_f16_16816_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32"
        " {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 2^(m - top) of a state at shift m (log2 units): 0 for one without weight (m = -inf).
__device__ __forceinline__ float weight_at(float m, float top) { return m == -INFINITY ? 0.f : ptx::ex2(m - top); }
__device__ __forceinline__ void store_bf16x4(__nv_bfloat16* dst, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(ptx::pack_bf16x2(a, b), ptx::pack_bf16x2(c, d));
}

template <int D, int NT>
__global__ void __launch_bounds__(Decode4Cfg<D, NT>::kWarps * 32, Decode4Cfg<D, NT>::kCtas)
decode4_sink_attn_kernel(const Decode4Args a) {
    using C = Decode4Cfg<D, NT>;
    constexpr int kKSteps = D / 16;
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t* first_s = reinterpret_cast<uint32_t*>(smem + C::kPipeBytes);
    float* ml_s = reinterpret_cast<float*>(smem + C::kPipeBytes + C::kPageBytes);
    float* sink_s = ml_s + C::kWarps * 32;
    int* flag_s = reinterpret_cast<int*>(sink_s + kMaxSliceHeads);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gq = lane >> 2, tq = lane & 3;
    const DecodeUnit u = a.units[blockIdx.x];   // uploaded before the kernels this one may overlap
    ptx::grid_dependency_wait();
    const int first_page = u.tok_begin >> a.page_log2;
    const int n_pages = ((u.tok_end - 1) >> a.page_log2) - first_page + 1;
    // The sinks (log2 units) of a request's first chunk, for the merge; read here,
    // in the shadow of the page ids.
    float sink = -INFINITY;
    if (tid < u.n_heads && u.chunk == 0 && a.sinks != nullptr) sink = a.sinks[u.head0 + tid] * kLog2e;
    load_sixteens(first_s, a.page_table + u.page_base + first_page, n_pages, a.num_pages, a.Hkv, u.kv_head, a.page_log2, a.err);
    if (tid < kMaxSliceHeads) sink_s[tid] = sink;
    __syncthreads();

    uint8_t* ring = smem + warp * C::kWarpBytes;
    const uint32_t ring_u32 = ptx::smem_u32(ring);
    const int n_tiles = (u.tok_end - u.tok_begin + C::kTile - 1) / C::kTile;
    const int n_it = n_tiles > warp ? (n_tiles - warp + C::kWarps - 1) / C::kWarps : 0;
    const TileSource src = tile_source<D, true, C::kTile>(a.pool, first_s, first_page, a.page_log2, a.Hkv, lane);
    auto issue = [&](int it, int s) {   // one group per stage, empty past the end
        const int tok = u.tok_begin + (warp + it * C::kWarps) * C::kTile;
        if (it < n_it) kv4_stage_load<D, C::kTile, 2>(src, tok, u.tok_end, ring_u32 + s * C::kStageBytes, lane);
        cp_async_commit();
    };
    for (int it = 0; it < C::kStages; ++it) issue(it, it);

    // Q (column operand: heads), scaled per head by a power of two; heads past
    // the slice are zero.  mult[nt] turns columns 2 tq and 2 tq + 1's products into
    // log2 units.
    uint32_t qb[NT][kKSteps][2];
    float2 mult[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + gq;
        float inv = 1.f;
        kv4_load_q<D>(h < u.n_heads ? a.q + ((size_t)u.q_row * a.Hq + u.head0 + h) * D : nullptr, tq, qb[nt], inv);
        mult[nt].x = __shfl_sync(0xffffffffu, inv, (2 * tq) * 4) * a.scale_log2;
        mult[nt].y = __shfl_sync(0xffffffffu, inv, (2 * tq + 1) * 4) * a.scale_log2;
    }

    // Online-softmax state of heads nt * 8 + 2 tq + e (log2 domain).  l is this
    // lane's share of the row sum.  The sink joins at the merge: a shift that
    // followed it would leave the keys beside a large sink no bits in f16.
    float o[NT][kKSteps][4];
    float2 nm[NT], l[NT];   // nm: the shift, negated
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        nm[nt] = l[nt] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kKSteps; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }
    float slack = -INFINITY;   // the first step moves every shift (a score of NaN never does)

    const int row = kv4_row(gq);   // tokens row and row + 8 of each sixteen are this lane's S rows
    for (int it = 0, s = 0; it < n_it; ++it) {
        cp_async_wait<C::kStages - 1>();
        __syncwarp();   // every lane's copies of this stage have landed
        const uint8_t* kt = ring + s * C::kStageBytes;
        const int valid = min(C::kTile, u.tok_end - (u.tok_begin + (warp + it * C::kWarps) * C::kTile));
        if (valid < C::kTile) {
            // Scale 0 for the V of tokens past the end (whatever their page
            // holds there may have a NaN scale; codes are always finite).
            kv4_clear_scales<D, C::kTile>(ring + s * C::kStageBytes + C::kSubs * C::kSub, valid, lane);
            __syncwarp();
        }
        const uint8_t* vt = kt + C::kSubs * C::kSub;
        // S^T of the stage's tokens.
        float x[C::kSubs][NT][4];
#pragma unroll
        for (int sub = 0; sub < C::kSubs; ++sub) {
            kv4_for_k<D>(kt + sub * C::kSub, row, tq, [&](int kk, const uint32_t (&ka)[4]) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (kk == 0) mma_f16_16816_new(x[sub][nt], ka, qb[nt][kk][0], qb[nt][kk][1]);
                    else mma_f16_16816(x[sub][nt], ka, qb[nt][kk][0], qb[nt][kk][1]);
                }
            });
        }
        if (valid < C::kTile) {   // tokens past the end have no score
#pragma unroll
            for (int sub = 0; sub < C::kSubs; ++sub)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (sub * kKv4Tokens + row + 8 * (e >> 1) >= valid) x[sub][nt][e] = -INFINITY;
        }

        // Scores above their shift, in log2 units; where one is by too
        // much (and at the start), the shifts move.
        float top = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int sub = 0; sub < C::kSubs; ++sub)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 v = ptx::fma2(make_float2(x[sub][nt][e], x[sub][nt][e + 1]), mult[nt], nm[nt]);
                    x[sub][nt][e] = v.x;
                    x[sub][nt][e + 1] = v.y;
                    top = fmaxf(top, fmaxf(v.x, v.y));
                }
        if (__any_sync(0xffffffffu, top > slack)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int sub = 0; sub < C::kSubs; ++sub)
                        mx = fmaxf(mx, fmaxf(x[sub][nt][e], x[sub][nt][e + 2]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                    // How far the shift moves: up alone, but at the start, where it holds
                    // no score yet (nor now, if all of them are -inf).
                    const bool none = slack < 0.f;
                    const float up = none && mx != -INFINITY ? mx - kShift : fmaxf(0.f, mx - kShift);
                    const float alpha = none ? 0.f : ptx::ex2(-up);
                    (e ? nm[nt].y : nm[nt].x) -= up;
                    (e ? l[nt].y : l[nt].x) *= alpha;
#pragma unroll
                    for (int i = 0; i < kKSteps; ++i) {
                        o[nt][i][e] *= alpha;
                        o[nt][i][e + 2] *= alpha;
                    }
#pragma unroll
                    for (int sub = 0; sub < C::kSubs; ++sub) {
                        x[sub][nt][e] -= up;
                        x[sub][nt][e + 2] -= up;
                    }
                }
            slack = kSlack;
        }

        // P^T as the column operand of the second product; O^T += V^T P^T.
#pragma unroll
        for (int sub = 0; sub < C::kSubs; ++sub) {
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = ptx::ex2(x[sub][nt][e]);
                l[nt] = ptx::add2(l[nt], ptx::add2(make_float2(p[0], p[1]), make_float2(p[2], p[3])));
                pb[nt][0] = transpose8x8(pack_f16x2(p[0], p[1]));
                pb[nt][1] = transpose8x8(pack_f16x2(p[2], p[3]));
            }
            kv4_for_v<D>(vt + sub * C::kSub, gq, tq, [&](int i, const uint32_t (&va)[4]) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[nt][i], va, pb[nt][0], pb[nt][1]);
            });
        }

        __syncwarp();   // every lane has read the stage
        issue(it + C::kStages, s);
        s = s + 1 == C::kStages ? 0 : s + 1;
    }

    // Only now: CTAs of the next grid that start while this one is in its loop
    // crowd onto the SMs that are done first.
    ptx::grid_dependents_go();

    // This warp's state into its own ring: O by head and dim.  Lane (gq, tq)
    // holds dims gq * D / 8 + {0 .. D / 8 - 1} of heads 2 tq and 2 tq + 1.
    __syncwarp();
    float* cs = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float* dst = cs + (nt * 8 + 2 * tq + e) * C::kRowStride + gq * (D / 8);
#pragma unroll
            for (int i = 0; i < kKSteps; ++i)
                *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[nt][i][e], o[nt][i][e + 2]);
            float sum = e ? l[nt].y : l[nt].x;
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (gq == 0) {
                ml_s[warp * 32 + nt * 8 + 2 * tq + e] = sum == 0.f ? -INFINITY : -(e ? nm[nt].y : nm[nt].x);   // no weight: no state
                ml_s[warp * 32 + 16 + nt * 8 + 2 * tq + e] = sum;
            }
        }
    __syncthreads();

    // Merge the warps, and in a request's first chunk the sink, a state of value
    // 0 and weight 1 at its own shift: heads < n_heads, 4 dims per item.
    const int items = u.n_heads * (D / 4);
    for (int idx = tid; idx < items; idx += blockDim.x) {
        const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
        float ms = fmaxf(sink_s[r], -INFINITY);   // -inf also where the sink is NaN
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) ms = fmaxf(ms, ml_s[w * 32 + r]);
        float L = weight_at(sink_s[r], ms);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
            const float mw = ml_s[w * 32 + r];
            const float f = weight_at(mw, ms);
            L += f * ml_s[w * 32 + 16 + r];
            const float4 ow = *reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(smem + w * C::kWarpBytes) + r * C::kRowStride + d);
            if (f > 0.f) { acc.x += f * ow.x; acc.y += f * ow.y; acc.z += f * ow.z; acc.w += f * ow.w; }
        }
        const float inv = L == 0.f ? 0.f : (u.n_chunks == 1 ? a.v_scale : 1.f) / L;   // no weight at all: 0, lse -inf
        const float lse2 = ms + log2f(L);
        if (u.n_chunks == 1) {
            store_bf16x4(a.out + ((size_t)u.q_row * a.Hq + u.head0 + r) * D + d, acc.x * inv, acc.y * inv, acc.z * inv,
                         acc.w * inv);
            if (d == 0 && a.lse) a.lse[(size_t)u.q_row * a.Hq + u.head0 + r] = lse2 * kLn2;
        } else {
            const size_t slot = (size_t)(u.partial0 + u.chunk) * kMaxSliceHeads + r;
            *reinterpret_cast<float4*>(a.part_o + slot * D + d) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (d == 0) a.part_lse[slot] = lse2;
        }
    }
    if (u.n_chunks == 1) return;

    // Split sequence: the last chunk to finish merges all chunks (no waiting),
    // in chunk order, so the result does not depend on which one that is.
    __threadfence();
    __syncthreads();
    if (tid == 0) *flag_s = atomicAdd(&a.counters[u.group], 1) == u.n_chunks - 1;
    __syncthreads();
    if (!*flag_s) return;
    __threadfence();
    constexpr int kMergeBatch = 8;   // chunks read with independent loads
    for (int idx = tid; idx < items; idx += blockDim.x) {
        const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
        float M = -INFINITY, W = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = 0; c0 < u.n_chunks; c0 += kMergeBatch) {
            float lc[kMergeBatch];
            float4 oc[kMergeBatch];
#pragma unroll
            for (int k = 0; k < kMergeBatch; ++k) {
                const int c = c0 + k;
                const size_t slot = (size_t)(u.partial0 + c) * kMaxSliceHeads + r;
                lc[k] = c < u.n_chunks ? __ldcg(a.part_lse + slot) : -INFINITY;
                oc[k] = c < u.n_chunks ? __ldcg(reinterpret_cast<const float4*>(a.part_o + slot * D + d))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float mb = M;
#pragma unroll
            for (int k = 0; k < kMergeBatch; ++k) mb = fmaxf(mb, lc[k]);
            const float sc = weight_at(M, mb);
            W *= sc;
            acc.x *= sc; acc.y *= sc; acc.z *= sc; acc.w *= sc;
#pragma unroll
            for (int k = 0; k < kMergeBatch; ++k) {
                const float w = weight_at(lc[k], mb);
                W += w;
                acc.x += w * oc[k].x; acc.y += w * oc[k].y; acc.z += w * oc[k].z; acc.w += w * oc[k].w;
            }
            M = mb;
        }
        const float inv = W == 0.f ? 0.f : a.v_scale / W;
        store_bf16x4(a.out + ((size_t)u.q_row * a.Hq + u.head0 + r) * D + d, acc.x * inv, acc.y * inv, acc.z * inv,
                     acc.w * inv);
        if (d == 0 && a.lse) a.lse[(size_t)u.q_row * a.Hq + u.head0 + r] = (M + log2f(W)) * kLn2;
    }
    if (tid == 0) a.counters[u.group] = 0;   // ready for the next launch
}

template <int D, int NT>
cudaError_t launch(const Decode4Args& args, int grid, cudaStream_t stream) {
    auto kernel = decode4_sink_attn_kernel<D, NT>;
    static std::atomic<bool> configured[kMaxDevices];
    cudaError_t e = once_per_device(configured, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Decode4Cfg<D, NT>::kSmem);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(grid), Decode4Cfg<D, NT>::kWarps * 32, Decode4Cfg<D, NT>::kSmem, stream, args);
}

}  // namespace

attn_status launch_decode_kv4(attn_plan_s* plan, const void* q, const void* kv4_cache, float k_scale, float v_scale,
                              const float* sinks, void* out, float* lse, cudaStream_t stream) {
    if (plan->units.empty()) return ATTN_OK;
    Decode4Args a;
    a.units = reinterpret_cast<const DecodeUnit*>(plan->ws + plan->layout.units);
    a.page_table = plan->page_table;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.pool = static_cast<const uint8_t*>(kv4_cache);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.sinks = sinks;
    a.part_o = reinterpret_cast<float*>(plan->ws + plan->layout.part_o);
    a.part_lse = reinterpret_cast<float*>(plan->ws + plan->layout.part_lse);
    a.counters = reinterpret_cast<int32_t*>(plan->ws + plan->layout.counters);
    a.err = reinterpret_cast<int32_t*>(plan->ws + plan->layout.err);
    a.Hq = plan->Hq;
    a.Hkv = plan->Hkv;
    a.page_log2 = 31 - __builtin_clz(plan->P);
    a.num_pages = plan->num_pages;
    a.scale_log2 = plan->sm_scale * kLog2e * k_scale;
    a.v_scale = v_scale;
    const bool two = plan->Hq / plan->Hkv > 8;
    const int grid = (int)plan->units.size();
    cudaError_t e;
    if (plan->D == 64) e = two ? launch<64, 2>(a, grid, stream) : launch<64, 1>(a, grid, stream);
    else e = two ? launch<128, 2>(a, grid, stream) : launch<128, 1>(a, grid, stream);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
