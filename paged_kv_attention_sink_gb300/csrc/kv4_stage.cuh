// Pieces of the kernels that multiply with 4-bit K and V tiles: copying a
// tile's page runs into shared memory, and turning its codes into mma.sync
// operand fragments.
#pragma once

#include "kv4.cuh"
#include "ptx.cuh"

namespace attn {

// A "sixteen": 16 consecutive tokens of a (page, K/V, KV head) block, which lie
// together in either pool (P is a multiple of 16, and units start on one, so a
// sixteen never crosses a page).  Sixteens are numbered through the pool:
//   ((page * 2 + half) * Hkv + head) * (P / 16) + row / 16,
// below 2^31 for any pool that fits the device.
constexpr uint32_t kBadPage = 0x80000000u;

// All threads of a CTA: K's first sixteen in each of a unit's pages (kBadPage,
// recorded, for an id outside the pool) into shared memory.  A barrier follows.
__device__ __forceinline__ void load_sixteens(uint32_t* first, const int32_t* page_table, int n_pages, int num_pages,
                                              int Hkv, int kv_head, int page_log2, int32_t* err) {
    for (int i = threadIdx.x; i < n_pages; i += blockDim.x) {
        const int page = page_table[i];
        const bool bad = page < 0 || page >= num_pages;
        if (bad) atomicOr(err, ATTN_DEVICE_ERR_PAGE_ID);
        first[i] = bad ? kBadPage : (uint32_t)(page * 2 * Hkv + kv_head) << (page_log2 - 4);
    }
}

// A unit's tokens: its table of sixteens, the first of which holds token tok0
// of the request rounded down to a page, and where each lane copies from.
struct TileSource {
    const uint8_t *pool, *pool_v;   // K's and V's sixteen 0, + this lane's 16 bytes
    const uint8_t* pool_s;          // 4-bit: this lane's piece of its sixteen's scales (K or V)
    const uint32_t* first;          // shared memory
    int tok0, page_log2;
    __device__ __forceinline__ uint32_t at(int t) const {
        return first[(t - tok0) >> page_log2] + ((t & ((1 << page_log2) - 1)) >> 4);
    }
};

template <int D, bool kFour, int kTile>
__device__ __forceinline__ TileSource tile_source(const uint8_t* pool, const uint32_t* first, int first_page,
                                                  int page_log2, int Hkv, int lane) {
    constexpr int kSub = kFour ? kv4_sub_bytes(D) : kBlockTokens * D * 2, kPieces = kTile / kKv4Tokens * (D / 16);
    const int64_t v = ((int64_t)Hkv << (page_log2 - 4)) * kSub;
    return {pool + lane * 16, pool + v + lane * 16, pool + (lane >= kPieces ? v : 0) + 8 * D + lane % (D / 16) * 16, first,
            first_page << page_log2, page_log2};
}

// 16 bytes global -> shared, asynchronously (the thread's current group), from
// `offset` bytes into a sixteen; zeros, and no access, where it is a bad one.
__device__ __forceinline__ void cp_async16(uint32_t dst, const uint8_t* pool, uint32_t sixteen, uint32_t bytes, int offset) {
    const uint8_t* src = pool + (uint64_t)(sixteen & ~kBadPage) * bytes + offset;
    const uint32_t size = 16u & ~(uint32_t)((int32_t)sixteen >> 31);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// A whole warp: start the copies of tokens [tok, tok + kTile) of a 4-bit pool
// into a stage (kTile / 16 sixteens of K, then, for kHalves = 2, of V); tok is
// a multiple of 16.  A sixteen's codes are 16 bytes for every lane (or twice
// that), and one copy takes the scales of eight sixteens (or four).  Sixteens
// from tok_end on, and those of a bad page, are set to zero instead.
template <int D, int kTile, int kHalves>
__device__ __forceinline__ void kv4_stage_load(const TileSource& s, int tok, int tok_end, uint32_t dst, int lane) {
    constexpr int kSubs = kTile / kKv4Tokens, kSub = kv4_sub_bytes(D), kScalePieces = D / 16;
    // Lane l looks up sixteen l % kSubs.
    const int t = tok + lane % kSubs * kKv4Tokens;
    const uint32_t mine = t < tok_end ? s.at(t) : kBadPage;
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub) {
        const uint32_t k = __shfl_sync(0xffffffffu, mine, sub);
#pragma unroll
        for (int half = 0; half < kHalves; ++half)
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                cp_async16(dst + (half * kSubs + sub) * kSub + j * 512 + lane * 16, half ? s.pool_v : s.pool, k, kSub, j * 512);
    }
    // Scales: lane l's piece and sixteen are the same in every stage (pool_s).
    constexpr int kPieces = kSubs * kScalePieces;   // of one half
#pragma unroll
    for (int i = 0; i < (kHalves * kPieces + 31) / 32; ++i) {
        const int idx = i * 32 + lane, block = idx / kScalePieces;
        const uint32_t k = __shfl_sync(0xffffffffu, mine, block % kSubs);
        const uint8_t* src = kPieces % 32 == 0 ? s.pool_s + (i * 32 / kPieces) * (s.pool_v - s.pool) : s.pool_s;
        if (kHalves * kPieces % 32 == 0 || idx < kHalves * kPieces)
            cp_async16(dst + block * kSub + 8 * D + idx % kScalePieces * 16, src, k, kSub, 0);
    }
}

// The same for K of a bf16 pool: rows of 64 dims (128 bytes) apart, 16-byte
// piece c of row r at c ^ (r % 8), as ldmatrix reads them without conflicts.
template <int D, int kTile>
__device__ __forceinline__ void bf16_stage_load(const TileSource& s, int tok, int tok_end, uint32_t dst, int lane) {
    constexpr int kSubs = kTile / kBlockTokens, kSub = kBlockTokens * D * 2, kPieces = D / 8;   // pieces of a row
    const int t = tok + lane % kSubs * kBlockTokens;
    const uint32_t mine = t < tok_end ? s.at(t) : kBadPage;
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub) {
        const uint32_t k = __shfl_sync(0xffffffffu, mine, sub);
#pragma unroll
        for (int j = 0; j < kSub / 512; ++j) {
            const int idx = j * 32 + lane, r = idx / kPieces, c = idx % kPieces;
            cp_async16(dst + sub * kSub + (c >> 3) * (kBlockTokens * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), s.pool, k,
                       kSub, j * 512);
        }
    }
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
