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
// One CTA = one decode unit of the plan (request, KV head, <= 16 query heads,
// KV chunk), four warps, each with its own ring of kTile-token stages filled
// by cp.async.bulk (one copy per page run: sixteen tokens' codes and scales
// lie together in the pool).
#include "attn_internal.h"
#include "kernels.h"
#include "kv4.cuh"
#include "kv4_stage.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The softmax shift m lies kShift below the running max, so that P's largest is
// 2^7 and f16 is normal down to 2^-21 of it (its subnormals then cost 2^-32 of
// it at most); m moves when a score passes it by kSlack (P stays below 2^15).
constexpr float kShift = 7.f, kSlack = 15.f;   // log2 units

template <int D, int NT>
struct Decode4Cfg {
    static constexpr int kWarps = kDecodeWarps;
    static constexpr int kStages = 3;
    static constexpr int kTile = 32;                                  // tokens per stage
    static constexpr int kSubs = kTile / kKv4Tokens;
    static constexpr int kSub = kv4_sub_bytes(D);
    static constexpr int kStageBytes = 2 * kSubs * kSub;              // K, then V
    static constexpr int kHeads = NT * 8;
    static constexpr int kRowStride = D + 8;                          // floats, combine buffers
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kPipeBytes = kWarps * kWarpBytes;
    static constexpr int kPageBytes = (kDecodeMaxChunkPages * 4 + 15) / 16 * 16;
    static constexpr int kBarBytes = kWarps * kStages * 8;
    static constexpr int kStateBytes = kWarps * 32 * 4 + 16;          // per-warp m, l (16 heads each) + flag
    static constexpr int kSmem = 128 + kPipeBytes + kPageBytes + kBarBytes + kStateBytes;
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
    int32_t Hq, Hkv, P, num_pages;
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
__device__ __forceinline__ void store_bf16x4(__nv_bfloat16* dst, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(ptx::pack_bf16x2(a, b), ptx::pack_bf16x2(c, d));
}

template <int D, int NT>
__global__ void __launch_bounds__(kDecodeWarps * 32)
decode4_sink_attn_kernel(const Decode4Args a) {
    using C = Decode4Cfg<D, NT>;
    constexpr int kKSteps = D / 16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                               ~static_cast<uintptr_t>(127));
    int32_t* pages_s = reinterpret_cast<int32_t*>(smem + C::kPipeBytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kPipeBytes + C::kPageBytes);
    float* ml_s = reinterpret_cast<float*>(smem + C::kPipeBytes + C::kPageBytes + C::kBarBytes);
    int* flag_s = reinterpret_cast<int*>(ml_s + C::kWarps * 32);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gq = lane >> 2, tq = lane & 3;
    if (lane == 0)
        for (int s = 0; s < C::kStages; ++s) ptx::mbar_init(ptx::smem_u32(&bars[warp * C::kStages + s]), 1);
    ptx::fence_mbar_init();

    const DecodeUnit u = a.units[blockIdx.x];
    const int P = a.P;
    const int first_page = u.tok_begin / P;
    const int n_pages = (u.tok_end - 1) / P - first_page + 1;
    for (int i = tid; i < n_pages; i += blockDim.x) pages_s[i] = a.page_table[u.page_base + first_page + i];
    __syncthreads();

    uint8_t* ring = smem + warp * C::kWarpBytes;
    const uint32_t ring_u32 = ptx::smem_u32(ring);
    const uint32_t bar0 = ptx::smem_u32(&bars[warp * C::kStages]);
    const int n_tiles = (u.tok_end - u.tok_begin + C::kTile - 1) / C::kTile;
    const int n_it = n_tiles > warp ? (n_tiles - warp + C::kWarps - 1) / C::kWarps : 0;
    const Kv4Source src{a.pool, pages_s, first_page, a.num_pages, a.Hkv, u.kv_head, P, a.err};
    auto issue = [&](int it) {
        const int s = it % C::kStages, tok = u.tok_begin + (warp + it * C::kWarps) * C::kTile;
        kv4_stage_load<D, C::kTile, 2>(src, tok, u.tok_end, ring_u32 + s * C::kStageBytes, bar0 + s * 8, lane);
    };
    for (int it = 0; it < C::kStages && it < n_it; ++it) issue(it);

    // Q (column operand: heads), scaled per head by a power of two; heads past
    // the slice are zero.  mult[nt][e] turns column 2 tq + e's products into
    // log2 units.
    uint32_t qb[NT][kKSteps][2];
    float mult[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + gq;
        float inv = 1.f;
        kv4_load_q<D>(h < u.n_heads ? a.q + ((size_t)u.q_row * a.Hq + u.head0 + h) * D : nullptr, tq, qb[nt], inv);
        mult[nt][0] = __shfl_sync(0xffffffffu, inv, (2 * tq) * 4) * a.scale_log2;
        mult[nt][1] = __shfl_sync(0xffffffffu, inv, (2 * tq + 1) * 4) * a.scale_log2;
    }

    // Online-softmax state of heads nt * 8 + 2 tq + e (log2 domain).  l is this
    // lane's share of the row sum; the sink counts once, on lane row 0.
    float m[NT][2], l[NT][2], o[NT][kKSteps][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = nt * 8 + 2 * tq + e;
            m[nt][e] = -INFINITY;
            l[nt][e] = 0.f;
            if (warp == 0 && u.chunk == 0 && a.sinks != nullptr && h < u.n_heads) {
                m[nt][e] = a.sinks[u.head0 + h] * kLog2e - kShift;
                l[nt][e] = gq == 0 ? exp2f(kShift) : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kKSteps; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }

    const int row = kv4_row(gq);   // tokens row and row + 8 of each sixteen are this lane's S rows
    bool timed_out = false;
    int it = 0;
    for (; it < n_it; ++it) {
        const int s = it % C::kStages;
        if (!ptx::mbar_wait(bar0 + s * 8, (it / C::kStages) & 1)) { timed_out = true; break; }
        const uint8_t* kt = ring + s * C::kStageBytes;
        const uint8_t* vt = kt + C::kSubs * C::kSub;
        const int valid = min(C::kTile, u.tok_end - (u.tok_begin + (warp + it * C::kWarps) * C::kTile));

        // S^T of the tile's tokens.
        float sc[C::kSubs][NT][4];
#pragma unroll
        for (int sub = 0; sub < C::kSubs; ++sub) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sc[sub][nt][0] = sc[sub][nt][1] = sc[sub][nt][2] = sc[sub][nt][3] = 0.f;
            kv4_for_k<D>(kt + sub * C::kSub, row, tq, [&](int kk, const uint32_t (&ka)[4]) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16_16816(sc[sub][nt], ka, qb[nt][kk][0], qb[nt][kk][1]);
            });
        }
        if (valid < C::kTile) {
            // Tokens past the end: no score, and scale 0 for their V (whatever
            // lies there may have a NaN scale; codes are always finite).
#pragma unroll
            for (int sub = 0; sub < C::kSubs; ++sub)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (sub * kKv4Tokens + row + 8 * (e >> 1) >= valid) sc[sub][nt][e] = -INFINITY;
            kv4_clear_scales<D, C::kTile>(ring + s * C::kStageBytes + C::kSubs * C::kSub, valid, lane);
            __syncwarp();
        }

        // Does a score pass its shift by too much?
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = -INFINITY;
#pragma unroll
                for (int sub = 0; sub < C::kSubs; ++sub) mx = fmaxf(mx, fmaxf(sc[sub][nt][e], sc[sub][nt][e + 2]));
                over = over || mx * mult[nt][e] > m[nt][e] + kSlack;
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int sub = 0; sub < C::kSubs; ++sub)
                        mx = fmaxf(mx, fmaxf(sc[sub][nt][e], sc[sub][nt][e + 2]));
                    mx *= mult[nt][e];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                    const float mn = fmaxf(m[nt][e], mx - kShift);
                    const float alpha = mn == -INFINITY ? 1.f : ptx::ex2(m[nt][e] - mn);
                    m[nt][e] = mn;
                    l[nt][e] *= alpha;
#pragma unroll
                    for (int i = 0; i < kKSteps; ++i) {
                        o[nt][i][e] *= alpha;
                        o[nt][i][e + 2] *= alpha;
                    }
                }
        }

        // P^T as the column operand of the second product.
        uint32_t pb[C::kSubs][NT][2];
#pragma unroll
        for (int sub = 0; sub < C::kSubs; ++sub)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = ptx::ex2(fmaf(sc[sub][nt][e], mult[nt][e & 1], -m[nt][e & 1]));
                l[nt][0] += p[0] + p[2];
                l[nt][1] += p[1] + p[3];
                pb[sub][nt][0] = transpose8x8(pack_f16x2(p[0], p[1]));
                pb[sub][nt][1] = transpose8x8(pack_f16x2(p[2], p[3]));
            }

        // O^T += V^T P^T.
#pragma unroll
        for (int sub = 0; sub < C::kSubs; ++sub)
            kv4_for_v<D>(vt + sub * C::kSub, gq, tq, [&](int i, const uint32_t (&va)[4]) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[nt][i], va, pb[sub][nt][0], pb[sub][nt][1]);
            });

        __syncwarp();
        if (it + C::kStages < n_it) {
            ptx::fence_proxy_async_smem();   // reads (and cleared scales) before the copy rewrites the stage
            issue(it + C::kStages);
        }
    }
    if (timed_out) {
        if (lane == 0) atomicOr(a.err, ATTN_DEVICE_ERR_TIMEOUT);
        for (int j = it; j < n_it && j < it + C::kStages; ++j)   // drain copies still in flight
            ptx::mbar_wait(bar0 + (j % C::kStages) * 8, (j / C::kStages) & 1);
    }

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
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
            if (gq == 0) {
                ml_s[warp * 32 + nt * 8 + 2 * tq + e] = m[nt][e];
                ml_s[warp * 32 + 16 + nt * 8 + 2 * tq + e] = l[nt][e];
            }
        }
    __syncthreads();

    // Merge the 4 warps: heads < n_heads, 4 dims per item.
    const int items = u.n_heads * (D / 4);
    for (int idx = tid; idx < items; idx += blockDim.x) {
        const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
        float ms = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) ms = fmaxf(ms, ml_s[w * 32 + r]);
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
            const float mw = ml_s[w * 32 + r];
            const float f = mw == -INFINITY ? 0.f : ptx::ex2(mw - ms);
            L += f * ml_s[w * 32 + 16 + r];
            const float4 ow = *reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(smem + w * C::kWarpBytes) + r * C::kRowStride + d);
            if (f > 0.f) { acc.x += f * ow.x; acc.y += f * ow.y; acc.z += f * ow.z; acc.w += f * ow.w; }
        }
        const float inv = (u.n_chunks == 1 ? a.v_scale : 1.f) / L;
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
            const float sc = M == -INFINITY ? 0.f : ptx::ex2(M - mb);
            W *= sc;
            acc.x *= sc; acc.y *= sc; acc.z *= sc; acc.w *= sc;
#pragma unroll
            for (int k = 0; k < kMergeBatch; ++k) {
                const float w = lc[k] == -INFINITY ? 0.f : ptx::ex2(lc[k] - mb);
                W += w;
                acc.x += w * oc[k].x; acc.y += w * oc[k].y; acc.z += w * oc[k].z; acc.w += w * oc[k].w;
            }
            M = mb;
        }
        const float inv = a.v_scale / W;
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
    kernel<<<grid, kDecodeWarps * 32, Decode4Cfg<D, NT>::kSmem, stream>>>(args);
    return cudaGetLastError();
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
    a.P = plan->P;
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
