// Eviction from the paged cache by accumulated attention weight.
//
// Of each request's n cached tokens every KV head keeps keep = min(n, budget):
// the newest min(n, recent), and of the others those of the largest weight,
// equal weights the older token first (a NaN weight counts as the lowest).
// Heads choose independently; kept tokens stay in order and become tokens
// 0 .. keep - 1 of the request, in new pages or in place.
//
// Select: one CTA per (request, KV head).  Weights map to unsigned keys of the
// same order; a radix selection, a byte of the key at a time, finds the
// threshold key and how many tokens that equal it are kept, and one ordered
// scan then writes the kept indices (and moves the weights).  Move: copies the
// kept tokens' K and V rows.  Both are bound by memory: 4 bytes per token and
// head are read, and the kept rows once read and once written.
//
// In place, token j comes from index kept[j] >= j.  A CTA owns one (request,
// head, K/V) and moves the rows in ascending order, a chunk at a time, all of
// a chunk read before any of it is written: every row it overwrites has been
// read before.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "kernels.h"
#include "kv4.cuh"

namespace attn {
namespace {

constexpr int kSelectThreads = 512;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;   // 16-byte pieces a thread holds between a chunk's reads and its writes

struct EvictArgs {
    const RequestInfo* requests;
    const int32_t* page_table;
    const float* weights;
    const uint8_t* pool;
    const int32_t* page_table_out;   // NULL: in place
    uint8_t* pool_out;
    float* weights_out;
    int32_t* kept;                   // [batch][Hkv][budget]
    int32_t* err;
    int32_t batch, Hkv, P, D, budget, recent, num_pages, num_pages_out;
};

// Unsigned keys in the weights' order: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0;
    const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// First output page slot of request b (pages of the requests before it); all
// threads of the block take part.
__device__ int64_t out_page_base(const EvictArgs& a, int b, int64_t* sh) {
    int64_t n = 0;
    for (int i = threadIdx.x; i < b; i += blockDim.x)
        n += (min(a.requests[i].kv_len, a.budget) + a.P - 1) / a.P;
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) n += sh[w];
    __syncthreads();
    return n;
}

// Output page id of token j of request r; -1 (recorded) when out of range.
__device__ __forceinline__ int out_page(const EvictArgs& a, const RequestInfo& r, int64_t base, int j) {
    const int page = a.page_table_out ? a.page_table_out[base + j / a.P] : a.page_table[r.page_base + j / a.P];
    if (page >= 0 && page < a.num_pages_out) return page;
    atomicOr(a.err, ATTN_DEVICE_ERR_PAGE_ID);
    return -1;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a) {
    constexpr int kWarps = kSelectThreads / 32;
    __shared__ int hist[256];
    __shared__ int64_t sh_base[kWarps];
    __shared__ uint32_t sh_scan[kWarps];
    __shared__ int sh_bucket, sh_above;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv;
    const RequestInfo r = a.requests[b];
    const int n = r.kv_len, keep = min(n, a.budget);
    int32_t* kept = a.kept + ((int64_t)b * a.Hkv + g) * a.budget;
    for (int j = keep + tid; j < a.budget; j += kSelectThreads) kept[j] = -1;
    if (n == 0) return;
    const int64_t base = a.page_table_out ? out_page_base(a, b, sh_base) : 0;

    const int old = n - min(n, a.recent);        // tokens [0, old) compete
    int want = keep - (n - old);                 // that many of them are kept
    auto weight = [&](int t) {
        const int page = a.page_table[r.page_base + t / a.P];
        if (page < 0 || page >= a.num_pages) {
            atomicOr(a.err, ATTN_DEVICE_ERR_PAGE_ID);
            return __uint_as_float(0x7FC00000u);
        }
        return a.weights[((int64_t)page * a.Hkv + g) * a.P + t % a.P];
    };

    // Threshold: the want-th largest key of the old tokens, byte by byte.
    uint32_t prefix = 0;
    int ties = want;                             // of the tokens that match the prefix, still to be kept
    if (want > 0 && want < old) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
            for (int t = tid; t < old; t += kSelectThreads) {
                const uint32_t k = order_key(weight(t));
                if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
            }
            __syncthreads();
            if (warp == 0) {   // the bucket the ties-th largest falls into; 8 buckets a lane, from the top
                int c[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - (lane * 8 + i)];
                int inc = sum;
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += v;
                }
                int above = inc - sum;
                if (above < ties && inc >= ties) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (above < ties && above + c[i] >= ties) {
                            sh_bucket = 255 - (lane * 8 + i);
                            sh_above = above;
                            break;
                        }
                        above += c[i];
                    }
                }
            }
            __syncthreads();
            prefix |= (uint32_t)sh_bucket << shift;
            ties -= sh_above;
        }
    }
    // keys > prefix are kept, of those equal to it the first `ties`; all old
    // tokens when want == old, none when want == 0.
    const bool all = want == old, none = want == 0;

    // Ordered scan: ranks of the kept tokens, chunk by chunk; low half counts
    // larger keys, high half equal ones.
    int greater = 0, equal = 0;
    for (int t0 = 0; t0 < n; t0 += kSelectThreads) {
        const int t = t0 + tid;
        const float w = t < n ? weight(t) : 0.f;
        uint32_t gt = 0, eq = 0;
        if (t >= old) {
            gt = t < n;
        } else if (all) {
            gt = 1;
        } else if (!none) {
            const uint32_t k = order_key(w);
            gt = k > prefix;
            eq = k == prefix;
        }
        uint32_t inc = gt | (eq << 16);
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) sh_scan[warp] = inc;
        __syncthreads();                          // also: the whole chunk's weights are read
        uint32_t before = inc - (gt | (eq << 16)), total = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) before += sh_scan[i];
            total += sh_scan[i];
        }
        const int gt_before = greater + (int)(before & 0xFFFF), eq_before = equal + (int)(before >> 16);
        if (gt || (eq && eq_before < ties)) {
            const int j = gt_before + min(eq_before, all || none ? 0 : ties);
            kept[j] = t;
            const int page = out_page(a, r, base, j);
            if (page >= 0) a.weights_out[((int64_t)page * a.Hkv + g) * a.P + j % a.P] = w;
        }
        greater += (int)(total & 0xFFFF);
        equal += (int)(total >> 16);
        __syncthreads();
    }
}

// grid (requests x KV heads x K/V, splits); a split takes every gridDim.y-th
// chunk of rows (one split in place).  kRowPieces: 16-byte pieces of a row's
// values; kFour: the rows also have D / 16 scale bytes.
template <int D, bool kFour>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
    constexpr int kPieces = (kFour ? D / 2 : D * 2) / 16;
    constexpr int kChunk = kMoveThreads * kMoveUnroll / kPieces;   // rows
    __shared__ int64_t sh_base[kMoveThreads / 32];
    const int half = blockIdx.x & 1, g = (blockIdx.x >> 1) % a.Hkv, b = (blockIdx.x >> 1) / a.Hkv;
    const RequestInfo r = a.requests[b];
    const int keep = min(r.kv_len, a.budget);
    if (keep == 0) return;
    const int64_t base = a.page_table_out ? out_page_base(a, b, sh_base) : 0;
    const int32_t* kept = a.kept + ((int64_t)b * a.Hkv + g) * a.budget;

    auto row_at = [&](int64_t page, int row) -> int64_t {   // byte offset of a row's values
        if constexpr (kFour)
            return kv4::sub_offset(page, half, a.Hkv, g, a.P, row, kv4_sub_bytes(D)) + (row % kKv4Tokens) * (D / 2);
        else
            return ((((page * 2 + half) * a.Hkv + g) * a.P) + row) * (D * 2);
    };
    for (int j0 = blockIdx.y * kChunk; j0 < keep; j0 += gridDim.y * kChunk) {
        uint4 x[kMoveUnroll];
        uint32_t sc[kMoveUnroll];
        int64_t dst[kMoveUnroll], dst_sc[kMoveUnroll];
#pragma unroll
        for (int k = 0; k < kMoveUnroll; ++k) {
            const int idx = k * kMoveThreads + threadIdx.x;
            const int j = j0 + idx / kPieces, piece = idx % kPieces;
            dst[k] = -1;
            if (j >= keep) continue;
            const int t = kept[j];
            const int page = a.page_table[r.page_base + t / a.P];
            const int to = out_page(a, r, base, j);
            if (page < 0 || page >= a.num_pages || to < 0) {
                atomicOr(a.err, ATTN_DEVICE_ERR_PAGE_ID);
                continue;
            }
            const int64_t src = row_at(page, t % a.P);
            x[k] = *reinterpret_cast<const uint4*>(a.pool + src + piece * 16);
            dst[k] = row_at(to, j % a.P);
            if constexpr (kFour) {
                // 16 code bytes are two groups: their two scales go along.
                const int in = t % kKv4Tokens, out = j % kKv4Tokens;
                sc[k] = *reinterpret_cast<const uint16_t*>(a.pool + src - in * (D / 2) + 8 * D + in * (D / 16) + 2 * piece);
                dst_sc[k] = dst[k] - out * (D / 2) + 8 * D + out * (D / 16) + 2 * piece;
            }
            dst[k] += piece * 16;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kMoveUnroll; ++k) {
            if (dst[k] < 0) continue;
            *reinterpret_cast<uint4*>(a.pool_out + dst[k]) = x[k];
            if constexpr (kFour) *reinterpret_cast<uint16_t*>(a.pool_out + dst_sc[k]) = (uint16_t)sc[k];
        }
        __syncthreads();   // in place: the next chunk may read what this one wrote over only after it is done
    }
}

}  // namespace

attn_status launch_evict(attn_plan_s* plan, bool four, const float* weights, const void* pool, int32_t budget,
                         int32_t recent, int32_t* kept, const int32_t* page_table_out, int32_t num_pages_out,
                         void* pool_out, float* weights_out, cudaStream_t stream) {
    if (plan->batch == 0) return ATTN_OK;
    EvictArgs a;
    a.requests = reinterpret_cast<const RequestInfo*>(plan->ws + plan->layout.requests);
    a.page_table = plan->page_table;
    a.weights = weights;
    a.pool = static_cast<const uint8_t*>(pool);
    a.page_table_out = page_table_out;
    a.pool_out = static_cast<uint8_t*>(pool_out);
    a.weights_out = weights_out;
    a.kept = kept;
    a.err = reinterpret_cast<int32_t*>(plan->ws + plan->layout.err);
    a.batch = plan->batch;
    a.Hkv = plan->Hkv;
    a.P = plan->P;
    a.D = plan->D;
    a.budget = budget;
    a.recent = recent;
    a.num_pages = plan->num_pages;
    a.num_pages_out = num_pages_out;
    evict_select_kernel<<<plan->batch * plan->Hkv, kSelectThreads, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
    const dim3 grid(plan->batch * plan->Hkv * 2, page_table_out ? 8 : 1);
    if (plan->D == 64) {
        if (four) evict_move_kernel<64, true><<<grid, kMoveThreads, 0, stream>>>(a);
        else evict_move_kernel<64, false><<<grid, kMoveThreads, 0, stream>>>(a);
    } else {
        if (four) evict_move_kernel<128, true><<<grid, kMoveThreads, 0, stream>>>(a);
        else evict_move_kernel<128, false><<<grid, kMoveThreads, 0, stream>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
