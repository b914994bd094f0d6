// The 4-bit KV cache's own data movement: quantising a step's new K/V rows
// into their pages, and expanding pages back to bf16.
//
// Sixteen dims x of a row share one scale.  With g the pool's scale (a power
// of two) and round() to nearest, ties to even, saturating:
//   s = e4m3 round(max|x| / (6 g)),   code_i = e2m1 round(x_i / (g s)),
//   value_i = code_i * s * g.
// 6 is e2m1's largest magnitude.  A NaN in a group makes the scale NaN, and
// with it the whole group; an infinity saturates (448 * 6 * g).
//
// Both kernels are HBM-bound copies with a few instructions per value; a
// thread owns one group of 16 dims (32 bytes of bf16, 8 code bytes and a
// scale byte).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "kernels.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kKv4Threads = 256;

// Quantise 16 bf16 values (w: pairs): the scale byte, and 8 code bytes.
__device__ __forceinline__ uint32_t quantise16(const uint32_t (&w)[8], float inv_pool_scale, uint2& codes) {
    // max |x| on the bits: bf16 magnitudes order like integers, NaN above infinity.
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        hi = max(hi, w[i] & 0x7FFF0000u);
        lo = max(lo, w[i] & 0x00007FFFu);
    }
    const float amax = __uint_as_float(max(hi, lo << 16)) * inv_pool_scale;
    // amax has 8 significant bits and a border between two e4m3 values 5, so
    // that amax * fl(1/6) falls on the same side of (or onto) each border as
    // amax / 6: fl(1/6)'s relative error 2^-25 is below half an ulp of a tie
    // and far below the distance of anything else.
    const uint32_t sb = kv4::scale_byte(amax * (1.f / 6.f));
    const float s = kv4::f16x2_to_f32(kv4::scales_to_f16x2(sb)).x;
    const float inv = s > 0.f ? 1.f / s : 0.f;
    // x / s correctly rounded (one Newton step on the quotient), so that a
    // quotient on a border between two codes lands on it and goes to the even
    // code.  0 * inf (a scale that underflowed to 0) cannot occur: inv = 0.
    auto div = [&](float x) {
        const float q = x * inv;
        const float q1 = fmaf(fmaf(-q, s, x), inv, q);
        return fabsf(q) < 16.f ? q1 : q;   // saturates either way; keeps an infinite x from turning NaN
    };
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 x = ptx::unpack_bf16x2(w[i]);
        c[i >> 2] |= kv4::code_pair(div(x.x * inv_pool_scale), div(x.y * inv_pool_scale)) << (8 * (i & 3));
    }
    codes = make_uint2(c[0], c[1]);
    return sb;
}

// One thread per (row, K/V, KV head, group of 16 dims).
template <int D>
__global__ void __launch_bounds__(kKv4Threads)
append_kv4_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new, uint8_t* __restrict__ pool,
                  const int2* __restrict__ slots, const int32_t* __restrict__ page_table, int64_t rows, int32_t Hkv,
                  int32_t P, int32_t num_pages, float inv_k, float inv_v, int32_t* err) {
    constexpr int kGroups = D / kKv4Group;
    const int32_t per_half = Hkv * kGroups;   // groups of one row's K (or V)
    const int64_t total = rows * 2 * per_half;
    for (int64_t i = (int64_t)blockIdx.x * kKv4Threads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kKv4Threads) {
        const int64_t r = i / (2 * per_half);
        const int32_t in_row = (int32_t)(i - r * (2 * per_half));
        const int half = in_row >= per_half;
        const int32_t in_half = in_row - half * per_half;
        const int g = in_half / kGroups, grp = in_half % kGroups;
        const int2 slot = slots[r];
        const int32_t page = page_table[slot.x];
        if (page < 0 || page >= num_pages) {
            if (in_row == 0) atomicOr(err, ATTN_DEVICE_ERR_PAGE_ID);
            continue;
        }
        const uint4* src = (half ? v_new : k_new) + (r * per_half + in_half) * 2;
        const uint4 a = __ldg(src), b = __ldg(src + 1);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint2 codes;
        const uint32_t sb = quantise16(w, half ? inv_v : inv_k, codes);
        uint8_t* sub = pool + kv4::sub_offset(page, half, Hkv, g, P, slot.y, kv4_sub_bytes(D));
        const int t = slot.y % kKv4Tokens;
        *reinterpret_cast<uint2*>(sub + t * (D / 2) + grp * 8) = codes;
        sub[8 * D + t * kGroups + grp] = (uint8_t)sb;
    }
}

// One thread per (listed page, K/V, KV head, token, group of 16 dims).
template <int D>
__global__ void __launch_bounds__(kKv4Threads)
expand_kv4_kernel(const uint8_t* __restrict__ pool, uint4* __restrict__ buf, const int32_t* __restrict__ page_ids,
                  int64_t n, int32_t Hkv, int32_t P, int64_t num_pages, float k_scale, float v_scale, int32_t* err) {
    constexpr int kGroups = D / kKv4Group, kSub = kv4_sub_bytes(D);
    const int64_t per_half = (int64_t)Hkv * P * kGroups;
    const int64_t total = n * 2 * per_half;
    for (int64_t i = (int64_t)blockIdx.x * kKv4Threads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kKv4Threads) {
        const int64_t blk = i / per_half;                 // (page in the list, K/V)
        const int64_t in_half = i - blk * per_half;       // ((head, sixteen tokens), token, group)
        const int32_t page = page_ids[blk >> 1];
        if (page < 0 || page >= num_pages) {
            if (in_half == 0 && (blk & 1) == 0 && err) atomicOr(err, ATTN_DEVICE_ERR_PAGE_ID);
            continue;
        }
        const int64_t sub_idx = in_half / (kKv4Tokens * kGroups);
        const int tg = (int)(in_half % (kKv4Tokens * kGroups));   // token * kGroups + group
        const uint8_t* sub = pool + (((int64_t)page * 2 + (blk & 1)) * Hkv * (P / kKv4Tokens) + sub_idx) * kSub;
        const uint2 codes = *reinterpret_cast<const uint2*>(sub + tg * 8);
        const float pool_scale = (blk & 1) ? v_scale : k_scale;
        const float s = kv4::f16x2_to_f32(kv4::scales_to_f16x2(sub[8 * D + tg])).x * pool_scale;
        uint32_t h[2][4], o[8];
        kv4::codes_to_f16x2(codes.x, h[0]);
        kv4::codes_to_f16x2(codes.y, h[1]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 v = kv4::f16x2_to_f32(h[k >> 2][k & 3]);
            o[k] = ptx::pack_bf16x2(v.x * s, v.y * s);    // exact: see kv4.cuh
        }
        buf[i * 2] = make_uint4(o[0], o[1], o[2], o[3]);
        buf[i * 2 + 1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

int kv4_grid(int64_t threads, int per_sm) {
    int32_t sms = 0;
    if (!current_sm_count(&sms)) return 0;
    const int64_t blocks = (threads + kKv4Threads - 1) / kKv4Threads, cap = (int64_t)sms * per_sm;
    return (int)(blocks < cap ? (blocks > 0 ? blocks : 1) : cap);
}

}  // namespace

attn_status launch_append_kv4(attn_plan_s* plan, const void* k_new, const void* v_new, void* kv4_cache, float k_scale,
                              float v_scale, cudaStream_t stream) {
    const int64_t rows = plan->info.total_qo_rows;
    if (rows == 0) return ATTN_OK;
    const int grid = kv4_grid(rows * 2 * plan->Hkv * (plan->D / kKv4Group), 8);
    if (grid == 0) return ATTN_ERR_CUDA;
    auto run = [&](auto kernel) {
        kernel<<<grid, kKv4Threads, 0, stream>>>(
            static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), static_cast<uint8_t*>(kv4_cache),
            reinterpret_cast<const int2*>(plan->ws + plan->layout.append), plan->page_table, rows, plan->Hkv, plan->P,
            plan->num_pages, 1.f / k_scale, 1.f / v_scale, reinterpret_cast<int32_t*>(plan->ws + plan->layout.err));
    };
    if (plan->D == 64) run(append_kv4_kernel<64>);
    else run(append_kv4_kernel<128>);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status launch_expand_kv4(const void* kv4_cache, void* buf, const int32_t* page_ids, int64_t n, int64_t num_pages,
                              int32_t Hkv, int32_t P, int32_t D, float k_scale, float v_scale, int32_t* err,
                              cudaStream_t stream) {
    if (n == 0) return ATTN_OK;
    const int grid = kv4_grid(n * 2 * Hkv * P * (D / kKv4Group), 8);
    if (grid == 0) return ATTN_ERR_CUDA;
    auto run = [&](auto kernel) {
        kernel<<<grid, kKv4Threads, 0, stream>>>(static_cast<const uint8_t*>(kv4_cache), static_cast<uint4*>(buf),
                                                 page_ids, n, Hkv, P, num_pages, k_scale, v_scale, err);
    };
    if (D == 64) run(expand_kv4_kernel<64>);
    else run(expand_kv4_kernel<128>);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
