// Accumulated attention weight per cached key.
//
//   w[t, g] = decay * prev[t, g] + sum over the plan's query rows i that see
//             key t and over the query heads h of KV head g of exp(s_ith - lse_ih),
//   s_ith = sm_scale * q_ih . k_tg;  tokens appended by this plan (t >= kv_len -
//   qo_len) have no previous weight.
//
// One warp owns 16 keys of one KV head: their K rows are the row operand of
// mma.sync m16n8k16 (bf16, exact for either cache), held in registers, and the
// query rows stream past as columns (query row i, head h), eight at a time.  A
// lane then holds the scores of two keys for two columns, exponentiates them
// with the rows' own lse and adds them up: no max, no reduction until the end,
// where the four lanes of a key row are summed (a fixed order).
#include <cuda_bf16.h>

#include "attn_internal.h"
#include "kernels.h"
#include "kv4_stage.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWeightWarps = 4;
constexpr int kWeightKeys = kWeightWarps * 16;   // keys per CTA

struct KeyWeightArgs {
    const RequestInfo* requests;
    const int32_t* page_table;
    const __nv_bfloat16* q;
    const float* lse;
    const void* pool;
    const float* prev;
    float* weights;
    int32_t* err;
    int32_t batch, Hq, Hkv, P, num_pages, causal, window;
    float scale_log2, decay;
};

// K rows of 16 keys as row operand: lane (gq, tq)'s dims of step kk are
// tq * D / 4 + 4 kk + {0..3}; keys gq and gq + 8 (bf16) or kv4_row order.
template <int D, bool kFour>
__device__ __forceinline__ void load_keys(const KeyWeightArgs& a, int64_t page, int g, int row0, int gq, int tq,
                                          uint32_t (&ka)[D / 16][4]) {
    if constexpr (kFour) {
        const uint8_t* sub = static_cast<const uint8_t*>(a.pool) +
                             kv4::sub_offset(page, 0, a.Hkv, g, a.P, row0, kv4_sub_bytes(D));
        kv4_for_k<D>(sub, kv4_row(gq), tq, [&](int kk, const uint32_t (&x)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = kv4::f16x2_to_f32(x[j]);
                ka[kk][j] = ptx::pack_bf16x2(v.x, v.y);   // exact
            }
        });
    } else {
        const __nv_bfloat16* k0 = static_cast<const __nv_bfloat16*>(a.pool) +
                                  ((page * 2 * a.Hkv + g) * a.P + row0 + kv4_row(gq)) * D + tq * (D / 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint2 x = *reinterpret_cast<const uint2*>(k0 + 4 * kk);
            const uint2 y = *reinterpret_cast<const uint2*>(k0 + 8 * D + 4 * kk);
            ka[kk][0] = x.x; ka[kk][1] = y.x; ka[kk][2] = x.y; ka[kk][3] = y.y;
        }
    }
}

template <int D, bool kFour>
__global__ void __launch_bounds__(kWeightWarps * 32)
key_weights_kernel(const KeyWeightArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const int b = blockIdx.z, g = blockIdx.y;
    const RequestInfo r = a.requests[b];
    if (r.qo_len == 0) return;
    const int G = a.Hq / a.Hkv, prefix = r.kv_len - r.qo_len;
    for (int64_t tile = blockIdx.x; tile * kWeightKeys < r.kv_len; tile += gridDim.x) {
        const int t0 = (int)tile * kWeightKeys + warp * 16;
        if (t0 >= r.kv_len) continue;
        const int page = a.page_table[r.page_base + t0 / a.P];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) atomicOr(a.err, ATTN_DEVICE_ERR_PAGE_ID);
            continue;
        }
        uint32_t ka[D / 16][4];
        load_keys<D, kFour>(a, page, g, t0 % a.P, gq, tq, ka);
        // Rows that count and can see any of these keys.
        int i0 = a.window > 0 ? max(0, r.qo_len - a.window) : 0;
        if (a.causal) i0 = max(i0, t0 - prefix);
        const int key0 = t0 + kv4_row(gq);
        float w0 = 0.f, w1 = 0.f;   // keys key0 and key0 + 8
        const int64_t cols = (int64_t)(r.qo_len - i0) * G;
        for (int64_t c0 = 0; c0 < cols; c0 += 8) {
            const int64_t c = c0 + gq;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            const __nv_bfloat16* q = a.q + ((int64_t)(r.q_row0 + i0 + (int)(c / G)) * a.Hq + g * G + (int)(c % G)) * D +
                                     tq * (D / 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint2 x = make_uint2(0u, 0u);
                if (c < cols) x = *reinterpret_cast<const uint2*>(q + 4 * kk);
                ptx::mma_bf16_16816(s, ka[kk], x.x, x.y);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t ce = c0 + 2 * tq + e;
                if (ce >= cols) continue;
                const int i = i0 + (int)(ce / G);
                const float l2 = a.lse[(int64_t)(r.q_row0 + i) * a.Hq + g * G + (int)(ce % G)] * kLog2e;
                const int last = a.causal ? prefix + i : r.kv_len - 1;   // last key row i sees
                if (key0 <= last) w0 += ptx::ex2(fmaf(s[e], a.scale_log2, -l2));
                if (key0 + 8 <= last) w1 += ptx::ex2(fmaf(s[e + 2], a.scale_log2, -l2));
            }
        }
        w0 += __shfl_xor_sync(0xffffffffu, w0, 1);
        w0 += __shfl_xor_sync(0xffffffffu, w0, 2);
        w1 += __shfl_xor_sync(0xffffffffu, w1, 1);
        w1 += __shfl_xor_sync(0xffffffffu, w1, 2);
        if (tq < 2) {
            const int key = key0 + 8 * tq;
            if (key < r.kv_len) {
                const int64_t at = ((int64_t)page * a.Hkv + g) * a.P + key % a.P;
                float w = tq ? w1 : w0;
                if (a.decay != 0.f && key < prefix) w = fmaf(a.decay, a.prev[at], w);
                a.weights[at] = w;
            }
        }
    }
}

}  // namespace

attn_status launch_key_weights(attn_plan_s* plan, bool four, const void* q, const void* pool, float k_scale,
                               const float* lse, const float* prev, float decay, int32_t window, float* weights,
                               cudaStream_t stream) {
    if (plan->info.total_qo_rows == 0) return ATTN_OK;
    KeyWeightArgs a;
    a.requests = reinterpret_cast<const RequestInfo*>(plan->ws + plan->layout.requests);
    a.page_table = plan->page_table;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.lse = lse;
    a.pool = pool;
    a.prev = prev;
    a.weights = weights;
    a.err = reinterpret_cast<int32_t*>(plan->ws + plan->layout.err);
    a.batch = plan->batch;
    a.Hq = plan->Hq;
    a.Hkv = plan->Hkv;
    a.P = plan->P;
    a.num_pages = plan->num_pages;
    a.causal = plan->causal;
    a.window = window;
    a.scale_log2 = plan->sm_scale * kLog2e * k_scale;
    a.decay = decay;
    int32_t longest = 0;
    for (const RequestInfo& r : plan->requests) longest = std::max(longest, r.kv_len);
    const dim3 grid(std::min((longest + kWeightKeys - 1) / kWeightKeys, 4096), plan->Hkv, plan->batch);
    if (plan->D == 64) {
        if (four) key_weights_kernel<64, true><<<grid, kWeightWarps * 32, 0, stream>>>(a);
        else key_weights_kernel<64, false><<<grid, kWeightWarps * 32, 0, stream>>>(a);
    } else {
        if (four) key_weights_kernel<128, true><<<grid, kWeightWarps * 32, 0, stream>>>(a);
        else key_weights_kernel<128, false><<<grid, kWeightWarps * 32, 0, stream>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
