// Eviction from the paged cache by accumulated attention weight.
//
// Of each request's n cached tokens every KV head keeps keep = min(n, budget):
// the newest min(n, recent), and of the others those of the largest weight,
// equal weights the older token first (a NaN weight counts as the lowest).
// Heads choose independently; kept tokens stay in order and become tokens
// 0 .. keep - 1 of the request, in new pages or in place.
//
// Select: one CTA per (request, KV head).  The weights are read into shared
// memory once (in chunks, again for each pass, where a row does not fit) and map
// to unsigned keys of the same order; a radix selection, 11 bits of the key at
// a time, finds the threshold key and how many tokens that equal it are kept.
// Then every warp counts the kept tokens of its own range of tokens and, from
// the sum of the ranges before it, writes their indices in order; the listed
// tokens' weights are moved after that, a thread each.  Move: a warp looks up 32
// kept tokens at a time, one per lane, and copies their K and V rows with many
// loads on their way at once.
//
// What has to be moved is 4 bytes per token and head, and the kept rows twice;
// but the selection's passes are a chain of barriers and shared-memory work that
// a row's CTA cannot shorten, while the memory idles.  With many rows one kernel
// does both, so that some CTAs copy while others select: 512 rows of
// 1K-8K tokens, 64 dims in bf16, down to 1024 each (283 MB) take 63 us (4.5 TB/s)
// where two kernels took 76.  With fewer rows the copies need all SMs and stay a
// kernel of their own: 128 rows of 2K-32K tokens, 128 dims in 4 bits, down to
// 4000 each, 31 + 32 us, set by the longest row's 32768 tokens (its weights
// arrive after 10,000 clocks; 23,000 for the three digits, 24,000 for counting
// and listing).  A row's CTA copying there too made the case 176 us instead of
// 133; clusters of CTAs that shared a row's histogram over distributed shared
// memory 157 (two or four of 256 threads) and 260 (eight).
//
// In place, token j comes from index kept[j] >= j.  A CTA owns one (request,
// head, K/V) and moves the rows in ascending order, a chunk at a time, all of
// a chunk read before any of it is written: every row it overwrites has been
// read before.  The weights are moved the same way, chunk by chunk.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "attn_internal.h"
#include "kernels.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kMoveThreads = 256, kBothThreads = 512;
constexpr int kBothChunk = 11 * 1024;   // weights of a row at a time: three CTAs per SM
constexpr int kWholeChunk = 48 * 1024;  // a CTA that has an SM for itself
constexpr int kDigitBits = 11, kDigits = 1 << kDigitBits;   // radix passes over 11, 11 and 10 bits

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
    int32_t batch, Hkv, page_log2, budget, recent, num_pages, num_pages_out;
    int32_t chunk;                   // select: tokens held in shared memory at a time
};

// Unsigned keys in the weights' order: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float w) {
    const int32_t u = __float_as_int(w + 0.f);   // -0 + 0 = +0
    return w == w ? (uint32_t)u ^ ((uint32_t)(u >> 31) | 0x80000000u) : 0u;
}

// The weight of a key.
__device__ __forceinline__ float key_weight(uint32_t k) {
    return __uint_as_float(k ^ (~(uint32_t)((int32_t)k >> 31) | 0x80000000u));
}

constexpr uint32_t kZeroKey = 0x80000000u, kLowestKey = 0x007FFFFFu, kInfKey = 0xFF800000u;   // of 0, -inf and +inf

// First output page slot of request b (pages of the requests before it); the
// lanes of a warp share the work.
__device__ int64_t out_page_base(const EvictArgs& a, int b, int lane) {
    if (!a.page_table_out) return 0;
    int64_t n = 0;
    const int P = 1 << a.page_log2;
    for (int i = lane; i < b; i += 32) n += (min(a.requests[i].kv_len, a.budget) + P - 1) >> a.page_log2;
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n;
}

// Output page id of token j of request r; -1 (recorded) when out of range.
__device__ __forceinline__ int out_page(const EvictArgs& a, const RequestInfo& r, int64_t base, int j) {
    const int slot = j >> a.page_log2;
    const int page = a.page_table_out ? a.page_table_out[base + slot] : a.page_table[r.page_base + slot];
    if (page >= 0 && page < a.num_pages_out) return page;
    atomicOr(a.err, ATTN_DEVICE_ERR_PAGE_ID);
    return -1;
}

// One request and KV head, by all threads of a CTA.
template <int kThreads>
__device__ __forceinline__ void select_tokens(const EvictArgs& a, const RequestInfo& r, int b, int g) {
    constexpr int kWarps = kThreads / 32;
    extern __shared__ __align__(16) float w_s[];   // [chunk] weights
    __shared__ __align__(16) int hist[kDigits];
    __shared__ int2 sh_count[kWarps];     // a warp's range: larger keys, equal keys
    __shared__ int sh_total[kWarps];
    __shared__ int sh_bucket, sh_above;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = r.kv_len, keep = min(n, a.budget), P = 1 << a.page_log2;
    int32_t* kept = a.kept + ((int64_t)b * a.Hkv + g) * a.budget;
    for (int j = keep + tid; j < a.budget; j += kThreads) kept[j] = -1;
    if (n == 0) return;
    const int64_t base = out_page_base(a, b, lane);

    const int old = n - min(n, a.recent);        // tokens [0, old) compete
    const int want = keep - (n - old);           // that many of them are kept
    const bool select = want > 0 && want < old;  // else all of them are, or none

    // Tokens [t0, t1) into shared memory, four (of one page) at a time; t0 is a
    // multiple of 4, and so is the chunk.
    auto load = [&](int t0, int t1) {
        constexpr int kBatch = 4;   // lookups, then loads, on their way together
        __syncthreads();            // the last chunk's readers are done
        for (int q0 = t0 + tid * 4; q0 < t1; q0 += kBatch * kThreads * 4) {
            int page[kBatch];
            float4 w[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int t = q0 + k * kThreads * 4;
                page[k] = t < t1 ? a.page_table[r.page_base + (t >> a.page_log2)] : 0;
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int t = q0 + k * kThreads * 4;
                const int from = page[k] >= 0 && page[k] < a.num_pages ? page[k] : 0;   // no branch between the loads
                if (t < t1)
                    w[k] = *reinterpret_cast<const float4*>(a.weights + ((int64_t)from * a.Hkv + g) * P + (t & (P - 1)));
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int t = q0 + k * kThreads * 4;
                if (t >= t1) continue;
                if (page[k] < 0 || page[k] >= a.num_pages) {
                    atomicOr(a.err, ATTN_DEVICE_ERR_PAGE_ID);
                    w[k] = make_float4(nanf(""), nanf(""), nanf(""), nanf(""));
                }
                *reinterpret_cast<float4*>(w_s + t - t0) = w[k];
            }
        }
        __syncthreads();
    };
    for (int i = tid; i < kDigits; i += kThreads) hist[i] = 0;   // a barrier follows in load()
    const bool fits = n <= a.chunk;
    if (fits) load(0, n);

    // Threshold: the want-th largest key of the old tokens, digit by digit.
    uint32_t prefix = 0;
    int ties = want;                             // of the tokens that match the prefix, still to be kept
    if (select) {
        for (int shift = 32 - kDigitBits;; shift = max(0, shift - kDigitBits)) {
            const int bits = shift == 0 ? 32 - 2 * kDigitBits : kDigitBits;
            for (int t0 = 0; t0 < old; t0 += a.chunk) {
                const int t1 = min(old, t0 + a.chunk);
                if (!fits) load(t0, t1);
                const uint32_t mask = (1u << bits) - 1;
                // Of the digits above this one the weight must have the prefix's:
                // it lies in a range of weights.  The range test is by value and
                // lets a zero of either sign into the range next to it; the few
                // weights that pass are tested by their keys.  (Below -inf there
                // are only NaNs, above +inf nothing.)
                const int high = shift + bits;
                const uint32_t above_mask = high == 32 ? 0u : ~0u << high;
                const bool all = high == 32 || prefix < kLowestKey;
                const float least = key_weight(prefix), most = key_weight(min(prefix | ~above_mask, kInfKey));
                int zeros = 0;   // weights of exactly 0 (keys never attended to) are many: one addition for all of a warp's
                for (int t = t0 + tid * 4; t < t1; t += kThreads * 4) {
                    const float4 w = *reinterpret_cast<const float4*>(w_s + t - t0);
                    const float v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (!(all || (v[e] >= least && v[e] <= most))) continue;
                        const uint32_t k = order_key(v[e]);
                        if (((k ^ prefix) & above_mask) || t + e >= t1) continue;
                        if (k == kZeroKey) ++zeros;
                        else atomicAdd(&hist[(k >> shift) & mask], 1);
                    }
                }
                zeros = __reduce_add_sync(0xffffffffu, zeros);
                if (lane == 0 && zeros) atomicAdd(&hist[(kZeroKey >> shift) & mask], zeros);
            }
            __syncthreads();
            // The bucket that the ties-th largest falls into: each thread sums (and
            // clears) a run of buckets, from the top; then the runs before it.
            constexpr int kRun = kDigits / kThreads;
            int c[kRun], sum = 0;
#pragma unroll
            for (int i = 0; i < kRun; i += 2) {
                int2* at = reinterpret_cast<int2*>(hist + kDigits - 2 - (tid * kRun + i));
                c[i] = at->y;
                c[i + 1] = at->x;
                *at = make_int2(0, 0);
                sum += c[i] + c[i + 1];
            }
            int inc = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 31) sh_total[warp] = inc;
            __syncthreads();
            const int above_warp = __reduce_add_sync(0xffffffffu, lane < warp ? sh_total[lane] : 0);
            int above = above_warp + inc - sum;
            if (above < ties && above + sum >= ties) {
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    if (above < ties && above + c[i] >= ties) {
                        sh_bucket = kDigits - 1 - (tid * kRun + i);
                        sh_above = above;
                        break;
                    }
                    above += c[i];
                }
            }
            __syncthreads();
            prefix |= (uint32_t)sh_bucket << shift;
            ties -= sh_above;
            if (shift == 0) break;
        }
    }
    // Kept: keys > prefix, and of those equal to it the first `ties`.
    const int all_ties = select ? ties : 0;
    int greater = 0, equal = 0, moved = 0;
    for (int t0 = 0; t0 < n; t0 += a.chunk) {
        const int t1 = min(n, t0 + a.chunk);
        if (!fits) load(t0, t1);
        // This warp's range of the chunk, in whole steps of 128 tokens, four a lane.
        const int per = ((t1 - t0 + 127) / 128 + kWarps - 1) / kWarps * 128;
        const int r0 = min(t1, t0 + warp * per), r1 = min(t1, r0 + per);
        // Bits 0-3: token t + e is kept by its key; 4-7: its key equals the threshold.
        // (By value, as the keys are ordered; below -inf there are only NaNs.)
        const float threshold = key_weight(prefix);
        const bool of_nans = prefix < kLowestKey;
        auto classify = [&](int t, const float (&v)[4]) {
            uint32_t c = 0;
            if (select && !of_nans) {
#pragma unroll
                for (int e = 0; e < 4; ++e) c |= v[e] > threshold ? 1u << e : v[e] == threshold ? 16u << e : 0u;
            } else if (select) {
#pragma unroll
                for (int e = 0; e < 4; ++e) c |= v[e] == v[e] ? 1u << e : 16u << e;
            } else if (want == old) {
                c = 15u;
            }
            if (t + 4 > old) {   // the newest are kept
                const uint32_t newest = 15u & ~0u << max(0, old - t);
                c = (c & ~(newest * 17u)) | newest;
            }
            return t + 4 > r1 ? c & (17u * ((1u << max(0, r1 - t)) - 1)) : c;
        };
        auto four = [&](int t, float (&v)[4]) {
            const float4 w = t < r1 ? *reinterpret_cast<const float4*>(w_s + t - t0) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
        };
        int n_gt = 0, n_eq = 0;
        for (int t = r0 + lane * 4; t < r1; t += 128) {
            float v[4];
            four(t, v);
            const uint32_t c = classify(t, v);
            n_gt += __popc(c & 15u);
            n_eq += __popc(c >> 4);
        }
        n_gt = __reduce_add_sync(0xffffffffu, n_gt);
        n_eq = __reduce_add_sync(0xffffffffu, n_eq);
        if (lane == 0) sh_count[warp] = make_int2(n_gt, n_eq);
        __syncthreads();
        const int2 count = lane < kWarps ? sh_count[lane] : make_int2(0, 0);
        int before_gt = greater + __reduce_add_sync(0xffffffffu, lane < warp ? count.x : 0);
        int before_eq = equal + __reduce_add_sync(0xffffffffu, lane < warp ? count.y : 0);
        greater += __reduce_add_sync(0xffffffffu, count.x);
        equal += __reduce_add_sync(0xffffffffu, count.y);
        for (int s = r0; s < r1; s += 128) {
            const int t = s + lane * 4;
            float v[4];
            four(t, v);
            const uint32_t c = classify(t, v);
            uint32_t inc = __popc(c & 15u) | __popc(c >> 4) << 16;
            const uint32_t own = inc;
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += u;
            }
            int gt = before_gt + (int)((inc - own) & 0xFFFF), eq = before_eq + (int)((inc - own) >> 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool is_gt = c >> e & 1, is_eq = c >> (4 + e) & 1;
                if (is_gt || (is_eq && eq < all_ties)) kept[gt + min(eq, all_ties)] = t + e;
                gt += is_gt;
                eq += is_eq;
            }
            const uint32_t total = __shfl_sync(0xffffffffu, inc, 31);
            before_gt += (int)(total & 0xFFFF);
            before_eq += (int)(total >> 16);
        }
        // The weights of the tokens just listed, while they are in shared memory.
        __syncthreads();
        const int listed = greater + min(equal, all_ties);
        for (int j = moved + tid; j < listed; j += kThreads) {
            const int page = out_page(a, r, base, j);
            const float v = w_s[kept[j] - t0];
            if (page >= 0) a.weights_out[((int64_t)page * a.Hkv + g) * P + (j & (P - 1))] = v;
        }
        moved = listed;
        __syncthreads();   // sh_count is written again
    }
}

// Kept rows of one request, KV head and K/V half, by `warps` warps of which this
// is number `warp`: 32 at a time per warp, `skip` from one step to the next, the
// copies of kBatch instructions on their way together.  In place all warps of
// the CTA take part and a step's rows are read before any is written.
// kFour: the rows also have D / 16 scale bytes.
template <int D, bool kFour, bool kInPlace, int kBatch = (kFour ? D / 2 : D * 2) / 16>
__device__ __forceinline__ void move_rows(const EvictArgs& a, const RequestInfo& r, int b, int g, int half, int warp,
                                          int first, int skip) {
    constexpr int kPieces = (kFour ? D / 2 : D * 2) / 16;   // 16-byte pieces of a row's values
    constexpr int kRows = 32 / kPieces;                     // rows a warp copies per instruction
    static_assert(kPieces % kBatch == 0 && (!kInPlace || kBatch == kPieces), "whole batches");
    using Scales = std::conditional_t<D == 64, uint32_t, uint2>;
    const int lane = threadIdx.x & 31;
    const int keep = min(r.kv_len, a.budget), P = 1 << a.page_log2;
    if (keep == 0) return;
    const int64_t base = out_page_base(a, b, lane);
    const int32_t* kept = a.kept + ((int64_t)b * a.Hkv + g) * a.budget;

    auto row_at = [&](int64_t page, int row) -> int64_t {   // byte offset of a row's values
        const int64_t block = (page * 2 + half) * a.Hkv + g;
        if constexpr (kFour)
            return ((block << (a.page_log2 - 4)) + row / kKv4Tokens) * kv4_sub_bytes(D) + (row % kKv4Tokens) * (D / 2);
        else
            return ((block << a.page_log2) + row) * (D * 2);
    };
    for (int c0 = first; c0 < keep; c0 += skip) {
        // Lane l looks up row l of the warp's 32.
        const int j = c0 + warp * 32 + lane;
        int64_t src = -1, dst = -1;
        Scales sc = {};
        int64_t dst_sc = -1;
        if (j < keep) {
            const int t = kept[j];
            const int page = a.page_table[r.page_base + (t >> a.page_log2)];
            const int to = out_page(a, r, base, j);
            if (page < 0 || page >= a.num_pages || to < 0) {
                atomicOr(a.err, ATTN_DEVICE_ERR_PAGE_ID);
            } else {
                const int from_row = t & (P - 1), to_row = j & (P - 1);
                src = row_at(page, from_row);
                dst = row_at(to, to_row);
                if constexpr (kFour) {
                    const int in = from_row % kKv4Tokens, out = to_row % kKv4Tokens;
                    sc = *reinterpret_cast<const Scales*>(a.pool + src - in * (D / 2) + 8 * D + in * (D / 16));
                    dst_sc = dst - out * (D / 2) + 8 * D + out * (D / 16);
                }
            }
        }
#pragma unroll
        for (int k0 = 0; k0 < kPieces; k0 += kBatch) {
            uint4 x[kBatch];
            int64_t to[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int row = (k0 + k) * kRows + lane / kPieces;
                const int64_t from = __shfl_sync(0xffffffffu, src, row);
                to[k] = __shfl_sync(0xffffffffu, dst, row);
                if (from >= 0) x[k] = *reinterpret_cast<const uint4*>(a.pool + from + lane % kPieces * 16);
            }
            if (kInPlace) __syncthreads();
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (to[k] >= 0) *reinterpret_cast<uint4*>(a.pool_out + to[k] + lane % kPieces * 16) = x[k];
        }
        if (kFour && dst_sc >= 0) *reinterpret_cast<Scales*>(a.pool_out + dst_sc) = sc;
        if (kInPlace) __syncthreads();   // the next step may read what this one wrote over only after it is done
    }
}

// grid: requests x KV heads
template <int kThreads>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a) {
    ptx::grid_dependents_go();
    const int b = blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv;
    const RequestInfo r = a.requests[b];   // uploaded before the kernels this one may overlap
    ptx::grid_dependency_wait();
    select_tokens<kThreads>(a, r, b, g);
}

// grid (requests x KV heads x K/V, splits; one split in place)
template <int D, bool kFour, bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
    const int half = blockIdx.x & 1, g = (blockIdx.x >> 1) % a.Hkv, b = (blockIdx.x >> 1) / a.Hkv;
    const RequestInfo r = a.requests[b];
    ptx::grid_dependency_wait();           // kept is complete and visible
    move_rows<D, kFour, kInPlace>(a, r, b, g, half, threadIdx.x >> 5, blockIdx.y * kMoveThreads, gridDim.y * kMoveThreads);
    ptx::grid_dependents_go();
}

// Both for the same request and head, out of place; grid: requests x KV heads.
// Half of the warps move K, the others V.  Three CTAs per SM: 64 us where 256
// threads and five took 87 and four CTAs of 512 (of 32 registers) 74; the rows
// in order of length, 70, for then all CTAs select, and all copy, at once.
template <int D, bool kFour>
__global__ void __launch_bounds__(kBothThreads, 3) evict_both_kernel(const EvictArgs a) {
    const int b = blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv, warp = threadIdx.x >> 5;
    const RequestInfo r = a.requests[b];   // uploaded before the kernels this one may overlap
    ptx::grid_dependency_wait();
    select_tokens<kBothThreads>(a, r, b, g);
    __syncthreads();                       // kept is complete
    move_rows<D, kFour, false, (kFour ? D / 2 : D * 2) / 16 < 4 ? 2 : 4>(a, r, b, g, warp & 1, warp >> 1, 0, kBothThreads / 2);
    ptx::grid_dependents_go();
}

template <int kThreads>
attn_status launch_select(const EvictArgs& a, int longest, int most, cudaStream_t stream) {
    EvictArgs x = a;
    x.chunk = std::max(32, std::min((longest + 31) / 32 * 32, most));
    static std::atomic<bool> configured[kMaxDevices];
    if (once_per_device(configured, [&] {
            return cudaFuncSetAttribute(evict_select_kernel<kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, most * 4);
        }) != cudaSuccess)
        return ATTN_ERR_CUDA;
    return launch_dependent(evict_select_kernel<kThreads>, dim3(a.batch * a.Hkv), kThreads, x.chunk * 4, stream, x) == cudaSuccess
               ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D, bool kFour>
attn_status launch_both(const EvictArgs& a, int longest, cudaStream_t stream) {
    EvictArgs x = a;
    x.chunk = std::max(32, std::min((longest + 31) / 32 * 32, kBothChunk));
    static std::atomic<bool> configured[kMaxDevices];
    if (once_per_device(configured, [&] {
            return cudaFuncSetAttribute(evict_both_kernel<D, kFour>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBothChunk * 4);
        }) != cudaSuccess)
        return ATTN_ERR_CUDA;
    return launch_dependent(evict_both_kernel<D, kFour>, dim3(a.batch * a.Hkv), kBothThreads, x.chunk * 4, stream, x) ==
                   cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D, bool kFour, bool kInPlace>
attn_status launch_move(const EvictArgs& a, int splits, cudaStream_t stream) {
    return launch_dependent(evict_move_kernel<D, kFour, kInPlace>, dim3(a.batch * a.Hkv * 2, splits), kMoveThreads, 0, stream,
                            a) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

attn_status launch_evict(attn_plan_s* plan, bool four, const float* weights, const void* pool, int32_t budget,
                         int32_t recent, int32_t* kept, const int32_t* page_table_out, int32_t num_pages_out,
                         void* pool_out, float* weights_out, cudaStream_t stream) {
    if (plan->batch == 0) return ATTN_OK;
    EvictArgs a;
    a.requests = reinterpret_cast<const RequestInfo*>(plan->lists + plan->lists_layout.requests);
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
    a.page_log2 = 31 - __builtin_clz(plan->P);
    a.budget = budget;
    a.recent = recent;
    a.num_pages = plan->num_pages;
    a.num_pages_out = num_pages_out;
    a.chunk = 0;
    int32_t longest = 0;
    for (const RequestInfo& r : plan->requests) longest = std::max(longest, r.kv_len);
    // A CTA takes all of an SM's threads and shared memory where there are few rows,
    // else a part of it.  Up to two rows per SM are few if that is what holds the
    // longest at once: in part of an SM it would be read four times.  Rows of
    // 64 dims in bf16 down to an eighth, part of an SM / all of it, us, out of place
    // and in place: 152 rows of 8K 28 / 21 and 21 / 25, of 32K 136 / 83 and 117 / 97;
    // 160 rows of 8K 30 / 31 and 30 / 30, of 12K 59 / 46 and 52 / 41, of 32K 145 / 112 and
    // 146 / 119, one of 32K among 8K 130 / 95 and 129 / 103, all of 64K 286 / 261 and
    // 291 / 326; 304 rows of 32K 197 / 162 and 192 / 176, of 2K-16K 77 / 83 and 91 / 84;
    // 456 of 32K 240 / 242 and 282 / 261, of 1K-32K 196 / 222 and 263 / 245.  (152 rows
    // of 2K: 14 / 16 and 10 / 11.)
    int32_t sms = 0;
    if (!current_sm_count(&sms)) return ATTN_ERR_CUDA;
    const int64_t all_rows = (int64_t)plan->batch * plan->Hkv;
    const bool few = all_rows <= sms || (all_rows <= 2 * sms && longest > kBothChunk && longest <= kWholeChunk);
    const bool in_place = !page_table_out;
    if (!few && !in_place) {
        if (plan->D == 64) return four ? launch_both<64, true>(a, longest, stream) : launch_both<64, false>(a, longest, stream);
        return four ? launch_both<128, true>(a, longest, stream) : launch_both<128, false>(a, longest, stream);
    }
    const attn_status st = few ? launch_select<1024>(a, longest, kWholeChunk, stream)
                               : launch_select<512>(a, longest, kBothChunk, stream);
    if (st != ATTN_OK) return st;
    // Out of place, enough CTAs for some eight per SM.
    const int64_t rows = std::min<int64_t>(longest, budget), most = (rows + kMoveThreads - 1) / kMoveThreads;
    const int64_t want = std::max<int64_t>(1, (int64_t)sms * 8 / ((int64_t)plan->batch * plan->Hkv * 2));
    const int splits = in_place ? 1 : (int)std::max<int64_t>(1, std::min(most, want));
    if (plan->D == 64) {
        if (four) return in_place ? launch_move<64, true, true>(a, splits, stream) : launch_move<64, true, false>(a, splits, stream);
        return in_place ? launch_move<64, false, true>(a, splits, stream) : launch_move<64, false, false>(a, splits, stream);
    }
    if (four) return in_place ? launch_move<128, true, true>(a, splits, stream) : launch_move<128, true, false>(a, splits, stream);
    return in_place ? launch_move<128, false, true>(a, splits, stream) : launch_move<128, false, false>(a, splits, stream);
}

}  // namespace attn
