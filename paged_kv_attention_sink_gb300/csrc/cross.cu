// Cross attention of few rows: up to 32 (row, query head) pairs of a sequence and
// KV head over a chunk of the sequence's keys, which are rows of contiguous
// K and V [rows][Hkv][D] (the prefill kernel takes sequences of many pairs).
//
//   out = sum_j exp(s_j - m) v_j / (sum_j exp(s_j - m) + exp(sink - m)),  s_j = scale q . k_j
//
// All pairs see all keys, so the beams, samples or draft tokens of a sequence share
// every byte of K and V that is read: HBM is the bound while the pairs are few.
//
//  * A CTA is four warps of products and one that loads.  The loading warp keeps a
//    ring of stages of 64 keys of K and V (boxes of 64 keys x 64 dims, 128-byte
//    swizzled; the last stage in boxes of 16, so that no more than 15 keys past the
//    end are read), full and empty barriers between it and the others.
//  * The four warps are kTiles m16 tiles of pairs times 4 / kTiles parts of a
//    stage's keys: with 16 pairs each warp takes 16 of the 64 keys, with 32 pairs
//    32.  A warp's state (max, sums, O) stays in registers over the chunk.
//  * S = Q K^T and O += P V are mma.sync m16n8k16: 16 to 32 flop per byte of K and V,
//    100 to 200 TFLOP/s at full HBM speed.
//  * P is rounded to bf16 and O normalised by the sum of that rounded P, lse taken
//    from the unrounded sum, as in the other attention kernels.
//  * Keys past the end: scores -inf, and V's fragments zeroed in registers, for
//    what lies there may be NaN.
//  * A chunk's state goes to the workspace; a small kernel joins the chunks.  (With
//    the last CTA of a sequence joining them, 50 chunks of 32 pairs took some 15 us,
//    one CTA reading after the other; joined by many CTAs, 4.)
//
// Measured: 48 x 5 beams over 1,500 keys of 16 heads x 64 dims (295 MB) 45 us, 6.6 TB/s;
// 16 rows over 2K-32K keys, 16 query heads on each of 4 KV heads x 128 dims (644 MB) 98,
// 6.6 TB/s (0.97 of the copy rate; issue 21%, tensor pipe 20%).  Small calls are the
// latency of one kernel, 2.5 to 2.9 us in a graph.  With 32 pairs it takes a seventh to
// a quarter longer than with 16 (64 x 1,500 keys of 8 heads of 64 dims 40 and 47 us, 32 x
// 1,500 of 16 heads of 128 dims 61 and 69, 1 x 16,000 of 16 heads of 64 dims 13.1 and
// 16.2): both read the same, and a warp's chain of products and softmax doubles.
#include <cuda.h>

#include "attn_internal.h"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kCrossWarps = 4;                        // of products
constexpr int kCrossThreads = (kCrossWarps + 1) * 32;

template <int D>
struct CrossCfg {
    static constexpr int kStages = D == 64 ? 4 : 3;
    static constexpr int kCtas = D == 64 ? 3 : 2;     // per SM
    static constexpr int kAtom = kCrossKeys * 128;    // 64 keys x 64 dims
    static constexpr int kTile = kAtom * (D / 64);    // K or V of a stage
    static constexpr int kStageBytes = 2 * kTile;
    static constexpr int kPipe = kStages * kStageBytes;
    static constexpr int kRow = D + 8;                // floats, combine buffers
    static constexpr int kOffBar = kPipe;
    static constexpr int kOffState = kOffBar + 2 * kStages * 8;
    static constexpr int kSmem = 1024 + kOffState + 3 * kCrossWarps * 16 * 4 + 16;
    static_assert(kCrossWarps * 16 * kRow * 4 <= kPipe, "combine buffers fit the stages");
};

struct CrossArgs {
    const DecodeUnit* units;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;
    const float* sinks;
    float* part_o;
    float* part_lse;
    int32_t* err;
    int32_t Hq, G;
    float scale_log2;
    int32_t late;   // runs beside the launch before it,
    int32_t open;   // lets the one after it run beside it (launch_cross)
};

__device__ __forceinline__ uint32_t ld_b32(const __nv_bfloat16* p) { return *reinterpret_cast<const uint32_t*>(p); }

__device__ __forceinline__ void store_bf16x4(__nv_bfloat16* dst, float4 v) {
    uint2 w;
    w.x = ptx::pack_bf16x2(v.x, v.y);
    w.y = ptx::pack_bf16x2(v.z, v.w);
    *reinterpret_cast<uint2*>(dst) = w;
}

// The chunks' states of one pair (`state`: the first chunk's, `stride` apart), 4 dims.
// Where a wait ran out a chunk's state may be an older call's: nothing is written,
// as in the rows of whole keys.  (Looked at behind the loads: 16 rows over 16,000 keys of 16
// heads 13.1 us, 13.5 without it, 14.2 looked at before the store.)
template <int D>
__device__ __forceinline__ void join_chunks(const CrossArgs& a, size_t state, size_t stride, int n_chunks, int row, int head,
                                            int d) {
    constexpr int kBatch = 8;   // chunks whose loads are in flight together
    const int32_t err = __ldcg(a.err);
    float M = -INFINITY, W = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < n_chunks; c0 += kBatch) {
        float lc[kBatch];
        float4 oc[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const size_t at = state + (size_t)(c0 + k) * stride;
            const bool in = c0 + k < n_chunks;
            lc[k] = in ? __ldcg(a.part_lse + at) : -INFINITY;
            oc[k] = in ? __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (err & ATTN_DEVICE_ERR_TIMEOUT) return;
        float mb = M;
        bool nan = false;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            mb = fmaxf(mb, lc[k]);
            nan |= lc[k] != lc[k];
        }
        if (mb == -INFINITY && !nan) continue;
        const float sc = M == -INFINITY ? 0.f : ptx::ex2(M - mb);
        W *= sc;
        acc = make_float4(acc.x * sc, acc.y * sc, acc.z * sc, acc.w * sc);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float w = lc[k] == -INFINITY ? 0.f : ptx::ex2(lc[k] - mb);
            W += w;
            acc.x += w * oc[k].x;
            acc.y += w * oc[k].y;
            acc.z += w * oc[k].z;
            acc.w += w * oc[k].w;
        }
        M = mb;
    }
    const float inv = W > 0.f ? 1.f / W : W;
    store_bf16x4(a.out + ((size_t)row * a.Hq + head) * D + d, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (d == 0 && a.lse) a.lse[(size_t)row * a.Hq + head] = (W == 0.f ? -INFINITY : M + log2f(W)) * kLn2;
}

// k_map, v_map: boxes of 64 keys; k_tail, v_tail: of 16.
template <int D, int kTiles>
__global__ void __launch_bounds__(kCrossThreads, CrossCfg<D>::kCtas)
cross_few_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                 const __grid_constant__ CUtensorMap k_tail, const __grid_constant__ CUtensorMap v_tail,
                 const CrossArgs a) {
    using C = CrossCfg<D>;
    constexpr int kParts = kCrossWarps / kTiles;      // of a stage's keys
    constexpr int kKeys = kCrossKeys / kParts;        // a warp's, of a stage
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = ptx::smem_u32(smem), full = sbase + C::kOffBar, empty = full + 8 * C::kStages;
    float* state = reinterpret_cast<float*>(smem + C::kOffState);   // [warp][m | l | e][16]
    volatile int* flags = reinterpret_cast<volatile int*>(state + 3 * kCrossWarps * 16);   // [1]: gave up

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const DecodeUnit u = a.units[blockIdx.x];         // the plan's own list
    const int keys = u.tok_end - u.tok_begin, n_it = (keys + kCrossKeys - 1) / kCrossKeys;
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(full + 8 * s, 1);
            ptx::mbar_init(empty + 8 * s, kCrossWarps);
        }
        flags[0] = flags[1] = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if (!a.late) ptx::grid_dependency_wait();
    if (a.open) ptx::grid_dependents_go();

    const int wm = warp % kTiles, part = warp / kTiles;   // (products)
    const int gq = lane >> 2, tq = lane & 3;
    // Rows gq and gq + 8 of the tile: pairs of the unit, or none.
    const int p0 = wm * 16 + gq, p1 = p0 + 8;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, e0 = 0.f, e1 = 0.f;
    float o[D / 8][4];
    auto row_head = [&](int p, int& row, int& head) {
        const int x = u.head0 + p;
        row = u.q_row + x / a.G;
        head = u.kv_head * a.G + x % a.G;
    };

    if (warp == kCrossWarps) {
        // ------------------------------------------------------------ loads
        const uint64_t policy = u.reserved ? ptx::policy_evict_last() : ptx::policy_evict_first();
        int it = 0;
        bool ok = true;
        for (; it < n_it; ++it) {
            const int s = it % C::kStages;
            if (it >= C::kStages &&
                !__all_sync(0xffffffffu, ptx::mbar_wait(empty + 8 * s, (it / C::kStages - 1) & 1))) { ok = false; break; }
            const int left = keys - it * kCrossKeys, row = u.page_base + u.tok_begin + it * kCrossKeys;
            const uint32_t dst = sbase + s * C::kStageBytes, bar = full + 8 * s;
            if (left >= kCrossKeys) {
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar, C::kStageBytes);
                __syncwarp();
                if (lane < 2 * (D / 64)) {
                    const int which = lane & 1, c = lane >> 1;
                    ptx::tma_load_3d_hint(dst + which * C::kTile + c * C::kAtom, which ? &v_map : &k_map, bar, c * 64,
                                          u.kv_head, row, policy);
                }
            } else {
                const int boxes = (left + 15) / 16;
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar, boxes * 16 * D * 4);
                __syncwarp();
                if (lane < 2 * (D / 64) * boxes) {
                    const int which = lane & 1, c = (lane >> 1) % (D / 64), b = (lane >> 1) / (D / 64);
                    ptx::tma_load_3d_hint(dst + which * C::kTile + c * C::kAtom + b * 2048, which ? &v_tail : &k_tail,
                                          bar, c * 64, u.kv_head, row + 16 * b, policy);
                }
            }
        }
        if (!ok && lane == 0) {
            atomicOr(a.err, ATTN_DEVICE_ERR_TIMEOUT);
            flags[1] = 1;
        }
        ptx::await_copies(full, C::kStages, it);
    } else {
        // --------------------------------------------------------- products
        uint32_t qa[D / 16][4];
        {
            int row, head;
            const __nv_bfloat16 *q0 = a.q, *q1 = a.q;
            const bool v0 = p0 < u.n_heads, v1 = p1 < u.n_heads;
            if (v0) {
                row_head(p0, row, head);
                q0 = a.q + ((size_t)row * a.Hq + head) * D;
                if (a.sinks != nullptr && u.chunk == 0 && part == 0) {
                    m0 = a.sinks[head] * kLog2e;
                    l0 = e0 = tq == 0 ? 1.f : 0.f;
                }
            }
            if (v1) {
                row_head(p1, row, head);
                q1 = a.q + ((size_t)row * a.Hq + head) * D;
                if (a.sinks != nullptr && u.chunk == 0 && part == 0) {
                    m1 = a.sinks[head] * kLog2e;
                    l1 = e1 = tq == 0 ? 1.f : 0.f;
                }
            }
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qa[kk][0] = v0 ? ld_b32(q0 + 16 * kk + 2 * tq) : 0u;
                qa[kk][2] = v0 ? ld_b32(q0 + 16 * kk + 8 + 2 * tq) : 0u;
                qa[kk][1] = v1 ? ld_b32(q1 + 16 * kk + 2 * tq) : 0u;
                qa[kk][3] = v1 ? ld_b32(q1 + 16 * kk + 8 + 2 * tq) : 0u;
            }
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

        const int mi = lane >> 3;
        for (int it = 0; it < n_it; ++it) {
            const int s = it % C::kStages;
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(full + 8 * s, (it / C::kStages) & 1))) {
                if (lane == 0) {
                    atomicOr(a.err, ATTN_DEVICE_ERR_TIMEOUT);
                    flags[1] = 1;
                }
                break;
            }
            const int valid = min(kKeys, keys - it * kCrossKeys - part * kKeys);   // of this warp's keys
            if (valid > 0) {
                const uint32_t kt = sbase + s * C::kStageBytes + part * kKeys * 128, vt = kt + C::kTile;
                float sc[kKeys / 8][4];
#pragma unroll
                for (int b = 0; b < kKeys / 16; ++b) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[2 * b][e] = sc[2 * b + 1][e] = 0.f;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int row = b * 16 + (mi >> 1) * 8 + (lane & 7), ch = 2 * kk + (mi & 1);
                        uint32_t b0, b1, b2, b3;
                        ptx::ldmatrix_x4(kt + (ch >> 3) * C::kAtom + row * 128 + (((ch & 7) ^ (lane & 7)) << 4), b0, b1, b2, b3);
                        ptx::mma_bf16_16816(sc[2 * b], qa[kk], b0, b1);
                        ptx::mma_bf16_16816(sc[2 * b + 1], qa[kk], b2, b3);
                    }
                }
                if (valid < kKeys) {
#pragma unroll
                    for (int nt = 0; nt < kKeys / 8; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (nt * 8 + 2 * tq + (e & 1) >= valid) sc[nt][e] = -INFINITY;
                }
                float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < kKeys / 8; ++nt) {
                    x0 = ptx::max3(x0, sc[nt][0], sc[nt][1]);
                    x1 = ptx::max3(x1, sc[nt][2], sc[nt][3]);
                }
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2)) * a.scale_log2;
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)) * a.scale_log2;
                if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
                    const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
                    const float a0 = n0 == -INFINITY ? 1.f : ptx::ex2(m0 - n0), a1 = n1 == -INFINITY ? 1.f : ptx::ex2(m1 - n1);
                    m0 = n0;
                    m1 = n1;
                    l0 *= a0;
                    e0 *= a0;
                    l1 *= a1;
                    e1 *= a1;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        o[j][0] *= a0;
                        o[j][1] *= a0;
                        o[j][2] *= a1;
                        o[j][3] *= a1;
                    }
                }
                const float s0 = m0 == -INFINITY ? 0.f : -m0, s1 = m1 == -INFINITY ? 0.f : -m1;
#pragma unroll
                for (int b = 0; b < kKeys / 16; ++b) {
                    uint32_t pa[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float* x = sc[2 * b + h];
                        const float y0 = ptx::ex2(fmaf(x[0], a.scale_log2, s0)), y1 = ptx::ex2(fmaf(x[1], a.scale_log2, s0));
                        const float y2 = ptx::ex2(fmaf(x[2], a.scale_log2, s1)), y3 = ptx::ex2(fmaf(x[3], a.scale_log2, s1));
                        e0 += y0 + y1;
                        e1 += y2 + y3;
                        pa[2 * h] = ptx::pack_bf16x2(y0, y1);
                        pa[2 * h + 1] = ptx::pack_bf16x2(y2, y3);
                        const float2 r0 = ptx::unpack_bf16x2(pa[2 * h]), r1 = ptx::unpack_bf16x2(pa[2 * h + 1]);
                        l0 += r0.x + r0.y;
                        l1 += r1.x + r1.y;
                    }
                    uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;   // V's keys 2 tq, 2 tq + 1 (+ 8) of the block
                    if (valid < kKeys) {
                        const int t = b * 16 + 2 * tq;
                        keep0 = (t < valid ? 0xffffu : 0u) | (t + 1 < valid ? 0xffff0000u : 0u);
                        keep1 = (t + 8 < valid ? 0xffffu : 0u) | (t + 9 < valid ? 0xffff0000u : 0u);
                    }
#pragma unroll
                    for (int j2 = 0; j2 < D / 16; ++j2) {
                        const int row = b * 16 + (mi & 1) * 8 + (lane & 7), ch = 2 * j2 + (mi >> 1);
                        uint32_t v0, v1, v2, v3;
                        ptx::ldmatrix_x4_trans(vt + (ch >> 3) * C::kAtom + row * 128 + (((ch & 7) ^ (lane & 7)) << 4), v0, v1, v2, v3);
                        if (valid < kKeys) {
                            v0 &= keep0;
                            v1 &= keep1;
                            v2 &= keep0;
                            v3 &= keep1;
                        }
                        ptx::mma_bf16_16816(o[2 * j2], pa, v0, v1);
                        ptx::mma_bf16_16816(o[2 * j2 + 1], pa, v2, v3);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty + 8 * s);
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, d);
            l1 += __shfl_xor_sync(0xffffffffu, l1, d);
            e0 += __shfl_xor_sync(0xffffffffu, e0, d);
            e1 += __shfl_xor_sync(0xffffffffu, e1, d);
        }
    }
    __syncthreads();                 // the stages are free
    ptx::grid_dependents_go();
    if (a.late) ptx::grid_dependency_wait();   // (ends after the launch before it)
    if (flags[1]) return;            // a wait ran out: nothing is written (join_chunks looks at the error word)

    if (warp < kCrossWarps) {
        float* cs = reinterpret_cast<float*>(smem) + warp * 16 * C::kRow;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
            const int d = 8 * j + 2 * tq;
            *reinterpret_cast<float2*>(&cs[gq * C::kRow + d]) = make_float2(o[j][0], o[j][1]);
            *reinterpret_cast<float2*>(&cs[(gq + 8) * C::kRow + d]) = make_float2(o[j][2], o[j][3]);
        }
        if (tq == 0) {
            float* st = state + warp * 48;
            st[gq] = m0;
            st[16 + gq] = l0;
            st[32 + gq] = e0;
            st[gq + 8] = m1;
            st[16 + gq + 8] = l1;
            st[32 + gq + 8] = e1;
        }
    }
    __syncthreads();

    // The parts' states of a pair, 4 dims per item.
    const int items = u.n_heads * (D / 4);
    for (int idx = tid; idx < items; idx += kCrossThreads) {
        const int p = idx / (D / 4), d = (idx % (D / 4)) * 4, tile = p >> 4, r = p & 15;
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < kParts; ++k) M = fmaxf(M, state[(tile + k * kTiles) * 48 + r]);
        float L = 0.f, E = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            const int w = tile + k * kTiles;
            const float mw = state[w * 48 + r];
            const float f = mw == -INFINITY ? 0.f : ptx::ex2(mw - M);
            L += f * state[w * 48 + 16 + r];
            E += f * state[w * 48 + 32 + r];
            const float4 ow = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) + (w * 16 + r) * C::kRow + d);
            acc.x += f * ow.x;
            acc.y += f * ow.y;
            acc.z += f * ow.z;
            acc.w += f * ow.w;
        }
        const float inv = L > 0.f ? 1.f / L : L;   // (0 keys: 0; NaN stays)
        const float lse2 = E == 0.f ? -INFINITY : M + log2f(E);
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (u.n_chunks == 1) {
            int row, head;
            row_head(p, row, head);
            store_bf16x4(a.out + ((size_t)row * a.Hq + head) * D + d, acc);
            if (d == 0 && a.lse) a.lse[(size_t)row * a.Hq + head] = lse2 * kLn2;
        } else {
            const size_t slot = ((size_t)u.partial0 + (size_t)u.chunk * kTiles) * kMaxSliceHeads + p;
            *reinterpret_cast<float4*>(a.part_o + slot * D + d) = acc;
            if (d == 0) a.part_lse[slot] = lse2;
        }
    }
}

template <int D, int kTiles>
cudaError_t launch(const CUtensorMap* maps, const CrossArgs& args, int units, cudaStream_t stream) {
    auto kernel = cross_few_kernel<D, kTiles>;
    static std::atomic<bool> configured[kMaxDevices];
    cudaError_t e = once_per_device(configured, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CrossCfg<D>::kSmem);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(units), kCrossThreads, CrossCfg<D>::kSmem, stream, maps[0], maps[1], maps[2],
                            maps[3], args);
}

// Joins the chunks' states of split keys, this kernel's and the prefill kernel's.  A
// thread has 4 dims of a pair, a CTA as many pairs of a record as that makes.
constexpr int kMergeThreads = 256;
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
cross_merge_kernel(const CrossMerge* merges, const CrossArgs a) {
    constexpr int kPairs = kMergeThreads / (D / 4), kCtas = kCrossBlock / kPairs;   // CTAs of a record
    const CrossMerge m = merges[blockIdx.x / kCtas];   // the plan's own list
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    const int p = blockIdx.x % kCtas * kPairs + threadIdx.x / (D / 4), x = m.pair0 + p;
    if (p < m.pairs)
        join_chunks<D>(a, (size_t)m.partial0 * kMaxSliceHeads + p, (size_t)m.stride * kMaxSliceHeads, m.n_chunks,
                       m.q_row0 + x / a.G, m.head0 + x % a.G, threadIdx.x % (D / 4) * 4);
}

template <int D>
cudaError_t launch_merge(const attn_plan_s* plan, const CrossArgs& args, cudaStream_t stream) {
    constexpr int kCtas = kCrossBlock / (kMergeThreads / (D / 4));
    return launch_dependent(cross_merge_kernel<D>, dim3(plan->cross_merges * kCtas), kMergeThreads, 0, stream,
                            reinterpret_cast<const CrossMerge*>(plan->ws + plan->layout.append), args);
}

}  // namespace

int cross_ctas_per_sm(int head_dim) { return head_dim == 64 ? CrossCfg<64>::kCtas : CrossCfg<128>::kCtas; }

// The kernels for 16 pairs, for 32 and for many write different rows and read nothing of
// one another, so that each may run beside the one before it: the first waits for
// what is on the stream and then lets the next one start; those (`late`) wait only
// before they end, so that whatever follows them follows all.  In turn, each would
// leave SMs idle while its last CTAs run (23 sequences of up to 38 rows over 0.7K-1.4K
// keys, 8 heads on 4 of 128 dims: 39 us in turn, 27 beside one another).
attn_status launch_cross(attn_plan_s* plan, const void* q, const void* q_map, const void* o_map, const float* sinks,
                         void* out, float* lse, cudaStream_t stream) {
    CrossArgs a;
    a.units = reinterpret_cast<const DecodeUnit*>(plan->ws + plan->layout.units);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.sinks = sinks;
    a.part_o = reinterpret_cast<float*>(plan->ws + plan->layout.part_o);
    a.part_lse = reinterpret_cast<float*>(plan->ws + plan->layout.part_lse);
    a.err = reinterpret_cast<int32_t*>(plan->ws + plan->layout.err);
    a.Hq = plan->Hq;
    a.G = plan->Hq / plan->Hkv;
    a.scale_log2 = plan->sm_scale * kLog2e;
    a.late = a.open = 0;
    const CUtensorMap* maps = reinterpret_cast<const CUtensorMap*>(plan->cross_maps);
    for (int size = 0; size < 2; ++size) {
        const int n = plan->cross_units[size];
        if (n == 0) continue;
        a.open = (size == 0 && plan->cross_units[1] > 0) || !plan->items.empty();
        const cudaError_t e = plan->D == 64 ? (size ? launch<64, 2>(maps, a, n, stream) : launch<64, 1>(maps, a, n, stream))
                                            : (size ? launch<128, 2>(maps, a, n, stream) : launch<128, 1>(maps, a, n, stream));
        if (e != cudaSuccess) return ATTN_ERR_CUDA;
        a.units += n;
        a.late = 1;
    }
    if (!plan->items.empty()) {
        const attn_status st = launch_prefill(plan, q_map, plan->kv_map_prefill, plan->v_map_prefill, o_map, sinks, out,
                                              lse, stream, a.late != 0);
        if (st != ATTN_OK) return st;
    }
    if (plan->cross_merges == 0) return ATTN_OK;
    const cudaError_t e = plan->D == 64 ? launch_merge<64>(plan, a, stream) : launch_merge<128>(plan, a, stream);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
