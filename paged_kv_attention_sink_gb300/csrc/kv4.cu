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
// Both kernels are copies that must spend few instructions on a value: packed
// fp32 arithmetic, and each thread finds its place by a division once and then
// steps.  Append also fetches its next item while it works on one.  57K rows of
// 8 heads x 128 dims (301 MB each way): append 62 us (73 with a division per
// item and nothing fetched ahead), 4.8 TB/s, bound by instruction issue (71% of
// its slots); expand 56 us, 5.4 TB/s, four of five bytes written (58 with one
// item per thread at a time instead of two, 64 with four).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "kernels.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kKv4Threads = 256;

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(ptx::f2_bits(a)), "l"(ptx::f2_bits(b)));
    return ptx::bits_f2(r);
}

// Quantise 16 bf16 values (w: pairs): the scale byte, and 8 code bytes.  g: the
// pool's scale, a power of two.
__device__ __forceinline__ uint32_t quantise16(const uint32_t (&w)[8], float g, float inv_g, uint2& codes) {
    // max |x| on the bits: bf16 magnitudes order like integers, NaN above infinity.
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        hi = max(hi, w[i] & 0x7FFF0000u);
        lo = max(lo, w[i] & 0x00007FFFu);
    }
    const float amax = __uint_as_float(max(hi, lo << 16)) * inv_g;
    // amax has 8 significant bits and a border between two e4m3 values 5, so
    // that amax * fl(1/6) falls on the same side of (or onto) each border as
    // amax / 6: fl(1/6)'s relative error 2^-25 is below half an ulp of a tie
    // and far below the distance of anything else.
    const uint32_t sb = kv4::scale_byte(amax * (1.f / 6.f));
    const float s = kv4::f16x2_to_f32(kv4::scales_to_f16x2(sb)).x;
    const float inv = s > 0.f ? 1.f / s : 0.f;      // a scale that underflowed to 0: all codes 0
    // x / (s g) correctly rounded (a Newton step on the quotient), so that a
    // quotient on a border between two codes lands on it and goes to the even
    // code.  Groups far beyond the largest scale saturate either way; there the
    // step is left out, for it would turn an infinity into NaN.
    const float2 d = make_float2(inv * inv_g, inv * inv_g), m = make_float2(-s * g, -s * g);
    const bool far = amax * inv >= 16.f;
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 x = ptx::unpack_bf16x2(w[i]);
        float2 q = mul2(x, d);
        if (!far) q = ptx::fma2(ptx::fma2(q, m, x), d, q);
        c[i >> 2] |= kv4::code_pair(q.x, q.y) << (8 * (i & 3));
    }
    codes = make_uint2(c[0], c[1]);
    return sb;
}

// One thread per (row, K/V, KV head, group of 16 dims), stepping through the
// items (a row's are per_row = 2 * Hkv * D / 16).
template <int D>
__global__ void __launch_bounds__(kKv4Threads)
append_kv4_kernel(const uint4* k_new, const uint4* v_new, uint8_t* pool, const int2* slots, const int32_t* page_table,
                  int64_t rows, int32_t Hkv, int32_t page_log2, int32_t num_pages, float k_scale, float inv_k,
                  float v_scale, float inv_v, int32_t* err) {
    ptx::grid_dependents_go();
    ptx::grid_dependency_wait();
    constexpr int kGroups = D / kKv4Group, kSub = kv4_sub_bytes(D);
    const int32_t per_half = Hkv * kGroups, per_row = 2 * per_half;
    const int64_t i = (int64_t)blockIdx.x * kKv4Threads + threadIdx.x, step = (int64_t)gridDim.x * kKv4Threads;
    const int64_t step_rows = step / per_row;
    const int32_t step_in = (int32_t)(step - step_rows * per_row);
    int64_t r = i / per_row;
    int32_t in_row = (int32_t)(i - r * per_row);
    // The next item's values and slot are on their way while this one is worked on.
    uint4 next_a, next_b;
    int2 next_slot;
    auto fetch = [&] {
        if (r >= rows) return;
        const int half = in_row >= per_half;
        const uint4* src = (half ? v_new : k_new) + (r * per_half + in_row - half * per_half) * 2;
        next_a = src[0];
        next_b = src[1];
        next_slot = slots[r];
    };
    fetch();
    while (r < rows) {
        const int half = in_row >= per_half;
        const int32_t in_half = in_row - half * per_half, in_row0 = in_row;
        const int g = in_half / kGroups, grp = in_half % kGroups;
        const uint4 a = next_a, b = next_b;
        const int2 slot = next_slot;
        const int32_t page = page_table[slot.x];
        r += step_rows;
        in_row += step_in;
        if (in_row >= per_row) {
            in_row -= per_row;
            ++r;
        }
        fetch();
        if (page >= 0 && page < num_pages) {
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            uint2 codes;
            const uint32_t sb = quantise16(w, half ? v_scale : k_scale, half ? inv_v : inv_k, codes);
            const int64_t block = ((int64_t)page * 2 + half) * Hkv + g;
            uint8_t* sub = pool + ((block << (page_log2 - 4)) + (slot.y >> 4)) * kSub;
            const int t = slot.y & (kKv4Tokens - 1);
            *reinterpret_cast<uint2*>(sub + t * (D / 2) + grp * 8) = codes;
            sub[8 * D + t * kGroups + grp] = (uint8_t)sb;
        } else if (in_row0 == 0) {
            atomicOr(err, ATTN_DEVICE_ERR_PAGE_ID);
        }
    }
}

// One thread per 8 values: (listed page, K/V, KV head, token, 8 dims), so that
// a warp writes 512 consecutive bytes; stepping as above (a (page, K/V) half
// has per_half = Hkv * P * D / 8 of them).
template <int D>
__global__ void __launch_bounds__(kKv4Threads)
expand_kv4_kernel(const uint8_t* pool, uint4* buf, const int32_t* page_ids, int64_t n, int32_t Hkv, int32_t P,
                  int64_t num_pages, float k_scale, float v_scale, int32_t* err) {
    ptx::grid_dependents_go();
    ptx::grid_dependency_wait();
    constexpr int kOctets = D / 8, kSub = kv4_sub_bytes(D), kPerSub = kKv4Tokens * kOctets, kBatch = 2;
    const int32_t per_half = Hkv * P * kOctets, half_subs = Hkv * (P / kKv4Tokens);
    const int64_t step = (int64_t)gridDim.x * kKv4Threads, step_halves = step / per_half;
    const int32_t step_in = (int32_t)(step - step_halves * per_half);
    int64_t i = (int64_t)blockIdx.x * kKv4Threads + threadIdx.x, blk = i / per_half;   // blk: (page in the list, K/V)
    int32_t in_half = (int32_t)(i - blk * per_half);   // ((head, sixteen tokens), token, 8 dims)
    while (blk < 2 * n) {
        // kBatch items: their pages, then their codes and scales, on the way together.
        int32_t page[kBatch], item[kBatch];
        bool v_half[kBatch];
        const int64_t i0 = i;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            page[u] = -1;
            item[u] = in_half;
            v_half[u] = blk & 1;
            if (blk < 2 * n) {
                page[u] = page_ids[blk >> 1];
                if (page[u] < 0 || page[u] >= num_pages) {
                    if (in_half == 0 && (blk & 1) == 0 && err) atomicOr(err, ATTN_DEVICE_ERR_PAGE_ID);
                    page[u] = -1;
                }
            }
            i += step;
            blk += step_halves;
            in_half += step_in;
            if (in_half >= per_half) {
                in_half -= per_half;
                ++blk;
            }
        }
        uint32_t codes[kBatch], sb[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (page[u] < 0) continue;
            const int32_t sub_idx = item[u] / kPerSub, at = item[u] % kPerSub;
            const uint8_t* sub = pool + (((int64_t)page[u] * 2 + v_half[u]) * half_subs + sub_idx) * kSub;
            codes[u] = *reinterpret_cast<const uint32_t*>(sub + at * 4);
            sb[u] = sub[8 * D + at / 2];
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (page[u] < 0) continue;
            const float s = kv4::f16x2_to_f32(kv4::scales_to_f16x2(sb[u])).x * (v_half[u] ? v_scale : k_scale);
            uint32_t h[4], o[4];
            kv4::codes_to_f16x2(codes[u], h);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 v = mul2(kv4::f16x2_to_f32(h[k]), make_float2(s, s));
                o[k] = ptx::pack_bf16x2(v.x, v.y);    // exact: see kv4.cuh
            }
            buf[i0 + u * step] = make_uint4(o[0], o[1], o[2], o[3]);
        }
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
    // As many CTAs as stay resident (48 registers a thread): a grid of 8 per SM
    // left a third of the last wave idle.
    const int grid = kv4_grid(rows * 2 * plan->Hkv * (plan->D / kKv4Group), 5);
    if (grid == 0) return ATTN_ERR_CUDA;
    const cudaError_t e = launch_dependent(
        plan->D == 64 ? append_kv4_kernel<64> : append_kv4_kernel<128>, dim3(grid), kKv4Threads, 0, stream,
        static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), static_cast<uint8_t*>(kv4_cache),
        reinterpret_cast<const int2*>(plan->ws + plan->layout.append), plan->page_table, rows, plan->Hkv,
        31 - __builtin_clz(plan->P), plan->num_pages, k_scale, 1.f / k_scale, v_scale, 1.f / v_scale,
        reinterpret_cast<int32_t*>(plan->ws + plan->layout.err));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status launch_expand_kv4(const void* kv4_cache, void* buf, const int32_t* page_ids, int64_t n, int64_t num_pages,
                              int32_t Hkv, int32_t P, int32_t D, float k_scale, float v_scale, int32_t* err,
                              cudaStream_t stream) {
    if (n == 0) return ATTN_OK;
    const int grid = kv4_grid(n * 2 * Hkv * P * (D / 8), 8);
    if (grid == 0) return ATTN_ERR_CUDA;
    const cudaError_t e = launch_dependent(D == 64 ? expand_kv4_kernel<64> : expand_kv4_kernel<128>, dim3(grid), kKv4Threads,
                                           0, stream, static_cast<const uint8_t*>(kv4_cache), static_cast<uint4*>(buf),
                                           page_ids, n, Hkv, P, num_pages, k_scale, v_scale, err);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
