// Pieces of the kernels that multiply with 4-bit K and V tiles: copying a
// tile's page runs into shared memory, and turning its codes into mma.sync
// operand fragments.
#pragma once

#include "kv4.cuh"
#include "ptx.cuh"

namespace attn {

// Where a unit's tokens lie: page ids (shared memory, from token
// first_page * P on) of one KV head in the pool.
struct Kv4Source {
    const uint8_t* pool;
    const int32_t* pages;
    int first_page, num_pages, Hkv, kv_head, P;
    int32_t* err;
};

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
        ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy) : "memory");
}

// A whole warp: start the copies of tokens [tok, min(tok + kTile, tok_end))
// into a stage (kTile / 16 sub-blocks of K, then, for kHalves = 2, of V); tok
// is a multiple of 16.  One copy per run of sub-blocks within a page; `bar`
// (one arrival) completes when all have landed.  Runs of a page id outside
// the pool are skipped and recorded.
template <int D, int kTile, int kHalves>
__device__ __forceinline__ void kv4_stage_load(const Kv4Source& s, int tok, int tok_end, uint32_t dst, uint32_t bar,
                                               int lane) {
    constexpr int kSubs = kTile / kKv4Tokens, kSub = kv4_sub_bytes(D);
    const int n_subs = min(kSubs, (tok_end - tok + kKv4Tokens - 1) / kKv4Tokens);
    const int half = lane / kSubs, sub = lane % kSubs;
    const int t = tok + sub * kKv4Tokens, off = t % s.P;
    uint32_t bytes = 0;
    const uint8_t* src = nullptr;
    if (half < kHalves && sub < n_subs && (sub == 0 || off == 0)) {
        const int page = s.pages[t / s.P - s.first_page];
        if (page < 0 || page >= s.num_pages) {
            atomicOr(s.err, ATTN_DEVICE_ERR_PAGE_ID);
        } else {
            bytes = min(n_subs - sub, (s.P - off) / kKv4Tokens) * kSub;
            src = s.pool + kv4::sub_offset(page, half, s.Hkv, s.kv_head, s.P, off, kSub);
        }
    }
    const uint32_t total = __reduce_add_sync(0xffffffffu, bytes);
    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, total);
    __syncwarp();
    if (bytes) bulk_load(dst + (half * kSubs + sub) * kSub, src, bytes, bar, ptx::policy_evict_first());
}

// Token of a sixteen that MMA row i (0..7) stands for; row i + 8 is 8 further.
// Any order would do; in this one the eight lanes of a shared-memory phase
// read tokens whose rows fall into different banks, in K's order (consecutive
// i) as well as in V's (every other i).
__device__ __forceinline__ int kv4_row(int i) { return i ^ ((i >> 2) & 1); }

// K as row operand: calls f(kk, a) with the 16x16 fragments of 16 tokens x
// dims of step kk.  Lane (gq, tq)'s dims of step kk are tq * D / 4 + 4 kk +
// {0..3} (kv4_load_q holds Q in the same order); `row` = kv4_row(gq).
template <int D, class F>
__device__ __forceinline__ void kv4_for_k(const uint8_t* sub, int row, int tq, F&& f) {
    constexpr int kWords = D / 32;    // 4-byte words of a lane's dims in one token
    uint32_t w[2][kWords];
    uint32_t sc[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const uint8_t* at = sub + (row + 8 * r) * (D / 2) + tq * (D / 8);
        if constexpr (D == 64) {
            const uint2 v = *reinterpret_cast<const uint2*>(at);
            w[r][0] = v.x; w[r][1] = v.y;
            sc[r] = sub[8 * D + (row + 8 * r) * (D / 16) + tq];
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(at);
            w[r][0] = v.x; w[r][1] = v.y; w[r][2] = v.z; w[r][3] = v.w;
            sc[r] = *reinterpret_cast<const uint16_t*>(sub + 8 * D + (row + 8 * r) * (D / 16) + 2 * tq);
        }
    }
    // Scale pairs (one token's scale twice), per group of 16 dims.
    uint32_t s2[2][D / 64];
    if constexpr (D == 64) {
        const uint32_t both = kv4::scales_to_f16x2(sc[0] | (sc[1] << 8));
        s2[0][0] = __byte_perm(both, both, 0x1010);
        s2[1][0] = __byte_perm(both, both, 0x3232);
    } else {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t both = kv4::scales_to_f16x2(sc[r]);
            s2[r][0] = __byte_perm(both, both, 0x1010);
            s2[r][1] = __byte_perm(both, both, 0x3232);
        }
    }
#pragma unroll
    for (int k2 = 0; k2 < kWords; ++k2) {     // a word is two steps
        uint32_t x[2][4];
        kv4::codes_to_f16x2(w[0][k2], x[0]);
        kv4::codes_to_f16x2(w[1][k2], x[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t a[4];
            a[0] = kv4::mul_f16x2(x[0][2 * k], s2[0][k2 / 2]);
            a[1] = kv4::mul_f16x2(x[1][2 * k], s2[1][k2 / 2]);
            a[2] = kv4::mul_f16x2(x[0][2 * k + 1], s2[0][k2 / 2]);
            a[3] = kv4::mul_f16x2(x[1][2 * k + 1], s2[1][k2 / 2]);
            f(2 * k2 + k, a);
        }
    }
}

// V^T as row operand: calls f(i, a) with the 16x16 fragments of 16 dims x 16
// tokens.  Lane (gq, tq)'s dims are gq * D / 8 + 2 i (rows gq) and + 1 (rows
// gq + 8); its tokens follow kv4_row, as S^T's rows do.
template <int D, class F>
__device__ __forceinline__ void kv4_for_v(const uint8_t* sub, int gq, int tq, F&& f) {
    constexpr int kWords = D / 64;
    uint32_t w[4][kWords], sb[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int token = kv4_row(2 * tq + (t & 1)) + 8 * (t >> 1);
        const uint8_t* at = sub + token * (D / 2) + gq * (D / 16);
        if constexpr (D == 64) {
            w[t][0] = *reinterpret_cast<const uint32_t*>(at);
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(at);
            w[t][0] = v.x; w[t][1] = v.y;
        }
        sb[t] = sub[8 * D + token * (D / 16) + gq * D / 128];
    }
    const uint32_t s01 = kv4::scales_to_f16x2(sb[0] | (sb[1] << 8));
    const uint32_t s23 = kv4::scales_to_f16x2(sb[2] | (sb[3] << 8));
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
        uint32_t x[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) kv4::codes_to_f16x2(w[t][j], x[t]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t a[4];
            a[0] = kv4::mul_f16x2(__byte_perm(x[0][i], x[1][i], 0x5410), s01);
            a[1] = kv4::mul_f16x2(__byte_perm(x[0][i], x[1][i], 0x7632), s01);
            a[2] = kv4::mul_f16x2(__byte_perm(x[2][i], x[3][i], 0x5410), s23);
            a[3] = kv4::mul_f16x2(__byte_perm(x[2][i], x[3][i], 0x7632), s23);
            f(4 * j + i, a);
        }
    }
}

// A whole warp: zero the scales of tokens [valid, kTile) of a staged half.
template <int D, int kTile>
__device__ __forceinline__ void kv4_clear_scales(uint8_t* half, int valid, int lane) {
    constexpr int kRow = D / 16, kSub = kv4_sub_bytes(D);
    for (int t = valid + lane; t < kTile; t += 32) {
        uint32_t* s = reinterpret_cast<uint32_t*>(half + (t / kKv4Tokens) * kSub + 8 * D + (t % kKv4Tokens) * kRow);
#pragma unroll
        for (int k = 0; k < kRow / 4; ++k) s[k] = 0;
    }
}

// One query head as column operand (column gq of the lane's tile), in f16,
// scaled by the power of two that brings its largest magnitude to [2^12,
// 2^13); inv is that power's inverse.  f16 then holds values down to 2^-26 of
// the largest exactly and rounds smaller ones to 2^-37 of it, below what the
// fp32 sum of the products resolves.  A head with an infinity or NaN is not
// scaled and stays what it is.  q may be NULL: a zero head.
template <int D>
__device__ __forceinline__ void kv4_load_q(const __nv_bfloat16* q, int tq, uint32_t (&b)[D / 16][2], float& inv) {
    uint32_t w[D / 16][2];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        uint2 v = make_uint2(0u, 0u);
        if (q) v = *reinterpret_cast<const uint2*>(q + tq * (D / 4) + 4 * k);
        w[k][0] = v.x; w[k][1] = v.y;
        top = max(max(top, v.x & 0x7FFF0000u), max((v.x & 0x7FFFu) << 16, max(v.y & 0x7FFF0000u, (v.y & 0x7FFFu) << 16)));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = (int)(top >> 23);            // biased exponent of the largest
    float f = 1.f;
    inv = 1.f;
    if (e != 255 && top != 0) {
        const int shift = max(-126, min(126, 12 - (e - 127)));
        f = __uint_as_float((uint32_t)(127 + shift) << 23);
        inv = __uint_as_float((uint32_t)(127 - shift) << 23);
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 v = ptx::unpack_bf16x2(w[k][j]);
            __half2 h = __floats2half2_rn(v.x * f, v.y * f);
            b[k][j] = *reinterpret_cast<uint32_t*>(&h);
        }
}

}  // namespace attn
