// The cache's pages handed about on the device: allocated, freed, copied,
// forked for samples and beams, and compacted to the front of their pools.
//
// refs[p] counts the page-table entries that hold page p; 0 is free.  New pages
// are the lowest free ones, so that equal calls give equal tables.  Finding
// them is a prefix sum over refs: one cluster of 8 CTAs reads it (each warp a
// contiguous part, 128 counts at a time), the CTAs' totals are exchanged
// through distributed shared memory, and each warp then numbers its own free
// pages by ballots.  A pool of 32K pages is 128 KB of counts: one cluster reads
// that in a microsecond or two, and a wider grid would need a second launch to
// join its parts.  The first reading's lines are in L1 or L2 for the second.
//
// Copies are memory-bound: a persistent grid takes (page, pool, 16 KB) pieces,
// 64 bytes per thread in flight.  How many pages move is only known on the
// device, so the grid reads the count there; nothing waits on the host.
//
// All counts and tables are integers changed by atomics or by one owner: equal
// calls give equal results whatever the order.
#include <cstdint>

#include "attn_internal.h"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kScanCtas = 8;            // one cluster
constexpr int kScanThreads = 1024;
constexpr int kScanWarps = kScanCtas * kScanThreads / 32;
constexpr int kPagesPerStep = 128;      // per warp: four counts per lane
constexpr int kMoveThreads = 256;
constexpr int kMoveBytes = 16384;       // a piece: four 16-byte chunks per thread
constexpr int kMoveCtasPerSm = 8;

// ------------------------------------------------------- sums over the cluster

struct ClusterSums {
    int64_t warp[32];
    int64_t total[2];   // of this CTA; two, used in turn
};

// Exclusive prefix of v over all threads of the cluster in order, and the sum.
// Every thread calls it; `turn` alternates between calls.
__device__ __forceinline__ int64_t cluster_prefix(int64_t v, ClusterSums& s, int turn, int64_t& sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    __syncthreads();   // the warps' sums of the call before have been read
    if (lane == 31) s.warp[warp] = inc;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll 8
    for (int w = 0; w < 32; ++w) {
        const int64_t x = s.warp[w];
        before += w < warp ? x : 0;
        all += x;
    }
    if (threadIdx.x == 0) s.total[turn] = all;
    ptx::cluster_sync();
    const uint32_t rank = ptx::cluster_rank(), addr = ptx::smem_u32(&s.total[turn]);
    sum = 0;
#pragma unroll
    for (uint32_t c = 0; c < kScanCtas; ++c) {
        const int64_t x = ptx::ld_cluster_s64(addr, c);
        before += c < rank ? x : 0;
        sum += x;
    }
    return before + inc - v;
}

// ------------------------------------------------------------------ free pages

// This warp's pages: steps of 128, [begin, end).
struct WarpPages {
    int32_t begin, end;
    __device__ WarpPages(int32_t num_pages) {
        const int64_t w = (int64_t)blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5);
        const int64_t steps = ((int64_t)num_pages + kPagesPerStep - 1) / kPagesPerStep;
        begin = (int32_t)(w * steps / kScanWarps);
        end = (int32_t)((w + 1) * steps / kScanWarps);
    }
};

// Counts of the lane's four pages of a step (past the pool: 1, not free).
__device__ __forceinline__ int4 load_counts(const int32_t* refs, int32_t num_pages, int32_t step, int32_t& page) {
    const int64_t p = (int64_t)step * kPagesPerStep + (threadIdx.x & 31) * 4;
    page = (int32_t)min(p, (int64_t)num_pages);
    if (p + 4 <= num_pages) return *reinterpret_cast<const int4*>(refs + p);
    int4 v = make_int4(1, 1, 1, 1);
    if (p < num_pages) v.x = refs[p];
    if (p + 1 < num_pages) v.y = refs[p + 1];
    if (p + 2 < num_pages) v.z = refs[p + 2];
    return v;
}

__device__ __forceinline__ uint32_t free_bits(int4 v) {
    return (v.x == 0 ? 1u : 0u) | (v.y == 0 ? 2u : 0u) | (v.z == 0 ? 4u : 0u) | (v.w == 0 ? 8u : 0u);
}

// Free pages among the lane's share of the warp's part.
__device__ int64_t count_free(const int32_t* refs, int32_t num_pages, const WarpPages& w) {
    int64_t n = 0;
    int32_t page;
#pragma unroll 8
    for (int32_t s = w.begin; s < w.end; ++s) n += __popc(free_bits(load_counts(refs, num_pages, s, page)));
    return n;
}

// Free pages of lower lanes in this step, and of the whole step.
__device__ __forceinline__ int lanes_before(uint32_t bits, int& all) {
    const uint32_t below = (1u << (threadIdx.x & 31)) - 1;
    int before = 0;
    all = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t b = __ballot_sync(0xffffffffu, bits >> k & 1);
        before += __popc(b & below);
        all += __popc(b);
    }
    return before;
}

// Numbers the free pages: found(rank, page) for every one of the first `want`.
// `base`: free pages before this warp's part.
template <class F>
__device__ void take_free(const int32_t* refs, int32_t num_pages, const WarpPages& w, int64_t base, int64_t want, F&& found) {
    for (int32_t s = w.begin; s < w.end && base < want; ++s) {
        int32_t page;
        const uint32_t bits = free_bits(load_counts(refs, num_pages, s, page));
        int all;
        int64_t rank = base + lanes_before(bits, all);
        base += all;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (bits >> k & 1) {
                if (rank < want) found(rank, page + k);
                ++rank;
            }
    }
}

// The prefix of the warp's first lane is that of its part.
__device__ __forceinline__ int64_t warp_base(int64_t prefix) { return __shfl_sync(0xffffffffu, prefix, 0); }

__device__ __forceinline__ void flag(int32_t* err, int bit) {
    if (err) atomicOr(err, bit);
}

__global__ void __cluster_dims__(kScanCtas) __launch_bounds__(kScanThreads)
alloc_kernel(int32_t* refs, int32_t num_pages, int32_t n, int32_t* page_ids, int32_t* err) {
    __shared__ ClusterSums sums;
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    const WarpPages part(num_pages);
    int64_t free_pages;
    const int64_t before = cluster_prefix(count_free(refs, num_pages, part), sums, 0, free_pages);
    take_free(refs, num_pages, part, warp_base(before), n, [&](int64_t rank, int32_t page) {
        page_ids[rank] = page;
        refs[page] = 1;
    });
    const int32_t thread = blockIdx.x * kScanThreads + threadIdx.x;
    for (int64_t i = free_pages + thread; i < n; i += kScanCtas * kScanThreads) page_ids[i] = -1;
    if (thread == 0 && free_pages < n) flag(err, ATTN_DEVICE_ERR_PAGES);
    ptx::cluster_sync();   // no CTA ends while another reads its sums
}

__global__ void __launch_bounds__(kMoveThreads)
free_kernel(int32_t* refs, int32_t num_pages, const int32_t* page_ids, int64_t n, int32_t* err) {
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    for (int64_t i = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kMoveThreads) {
        const int32_t page = page_ids[i];
        if (page < 0 || page >= num_pages) {
            flag(err, ATTN_DEVICE_ERR_PAGE_ID);
        } else if (atomicSub(&refs[page], 1) <= 0) {   // nobody holds it: taken back
            atomicAdd(&refs[page], 1);
            flag(err, ATTN_DEVICE_ERR_PAGES);
        }
    }
}

// ------------------------------------------------------------------------ fork

// Pages of child c (0 where its parent is not sound), whether its last one is a
// copy, and the parent's first table slot.
struct Child {
    int32_t pages, part, base;
    bool bad;
    __device__ Child(const PageFork& f, int32_t c) : pages(0), part(0), base(0), bad(true) {
        const int32_t p = f.parents[c];
        if (p < 0 || p >= f.batch) return;
        const int32_t len = f.kv_lens[p];
        base = f.kv_indptr[p];
        const int64_t held = (int64_t)f.kv_indptr[p + 1] - base;
        if (len < 0 || base < 0 || base + held > f.table_len || held < ((int64_t)len + f.page_size - 1) / f.page_size) return;
        bad = false;
        pages = len / f.page_size + (len % f.page_size != 0);
        part = len % f.page_size != 0;
    }
};

__global__ void __cluster_dims__(kScanCtas) __launch_bounds__(kScanThreads)
fork_kernel(int32_t* refs, int32_t num_pages, const PageFork f, int32_t* scratch, int32_t* err) {
    __shared__ ClusterSums sums;
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    const WarpPages part(num_pages);
    const int32_t thread = blockIdx.x * kScanThreads + threadIdx.x, threads = kScanCtas * kScanThreads;
    const int32_t c0 = (int32_t)((int64_t)thread * f.n / threads), c1 = (int32_t)((int64_t)(thread + 1) * f.n / threads);
    int64_t entries = 0, fresh = 0;
    bool bad = false;
    for (int32_t c = c0; c < c1; ++c) {
        const Child child(f, c);
        entries += child.pages;
        fresh += child.part;
        bad |= child.bad;
    }
    int64_t all_entries, all_fresh, free_pages;
    int64_t at = cluster_prefix(entries, sums, 0, all_entries);
    int64_t rank = cluster_prefix(fresh, sums, 1, all_fresh);
    const bool refused = all_entries > f.out_len;
    const int64_t before = cluster_prefix(refused ? 0 : count_free(refs, num_pages, part), sums, 0, free_pages);
    int32_t *dst = scratch + kMoveHead, *src = dst + f.n;
    if (!refused)
        take_free(refs, num_pages, part, warp_base(before), all_fresh, [&](int64_t r, int32_t page) {
            dst[r] = page;
            refs[page] = 1;
        });
    if (bad) flag(err, ATTN_DEVICE_ERR_PLAN);
    ptx::cluster_sync();   // dst is complete, and every CTA has read the sums
    if (thread == 0) {
        if (refused) flag(err, ATTN_DEVICE_ERR_PLAN);
        if (!refused && free_pages < all_fresh) flag(err, ATTN_DEVICE_ERR_PAGES);
        scratch[0] = refused ? 0 : (int32_t)min(all_fresh, free_pages);
        f.indptr_out[f.n] = refused ? 0 : (int32_t)all_entries;
    }
    for (int32_t c = c0; c < c1; ++c) {
        f.indptr_out[c] = refused ? 0 : (int32_t)at;
        if (refused) continue;
        const Child child(f, c);
        at += child.pages;
        if (!child.part) continue;
        f.table_out[at - 1] = rank < free_pages ? dst[rank] : -1;
        src[rank++] = f.page_table[child.base + child.pages - 1];
    }
}

// The first n entries of a child are its parent's own pages, held once more.
__device__ void share_pages(int32_t* refs, int32_t num_pages, const PageFork& f, int32_t* err, int32_t block, int32_t blocks) {
    const int64_t total = f.indptr_out[f.n];
    for (int64_t e = (int64_t)block * kMoveThreads + threadIdx.x; e < total; e += (int64_t)blocks * kMoveThreads) {
        int32_t lo = 0, hi = f.n - 1;   // the last child that begins at or before e
        while (lo < hi) {
            const int32_t mid = lo + (hi - lo + 1) / 2;
            if (f.indptr_out[mid] <= e) lo = mid;
            else hi = mid - 1;
        }
        const Child child(f, lo);
        const int32_t j = (int32_t)(e - f.indptr_out[lo]);
        if (j >= child.pages - child.part) continue;   // the copied page: fork_kernel's
        const int32_t page = f.page_table[child.base + j];
        const bool in = page >= 0 && page < num_pages;
        if (in) atomicAdd(&refs[page], 1);
        else flag(err, ATTN_DEVICE_ERR_PAGE_ID);
        f.table_out[e] = in ? page : -1;
    }
}

// --------------------------------------------------------------------- compact

// U pages are in use.  The free ones below U are filled, lowest first, with the
// used ones from U on, highest first.
__global__ void __cluster_dims__(kScanCtas) __launch_bounds__(kScanThreads)
compact_kernel(int32_t* refs, int32_t num_pages, int32_t* remap, int32_t* scratch) {
    __shared__ ClusterSums sums;
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    const WarpPages part(num_pages);
    int32_t *dst = scratch + kMoveHead, *src = dst + num_pages / 2;
    int64_t free_pages, holes = 0, all_holes;
    int64_t base = warp_base(cluster_prefix(count_free(refs, num_pages, part), sums, 0, free_pages));
    const int64_t used = num_pages - free_pages;
    for (int32_t s = part.begin; s < part.end; ++s) {
        int32_t page;
        const uint32_t bits = free_bits(load_counts(refs, num_pages, s, page));
        int all;
        int64_t rank = base + lanes_before(bits, all);   // free pages before `page`
        base += all;
#pragma unroll
        for (int k = 0; k < 4; ++k, ++page) {
            if (page >= num_pages) break;
            if (bits >> k & 1) {
                if (page < used) {
                    dst[rank] = page;
                    ++holes;
                }
                ++rank;
                remap[page] = -1;
            } else if (page < used) {
                remap[page] = page;
            } else {
                src[used - 1 - (page - rank)] = page;   // used pages before it: page - rank
            }
        }
    }
    cluster_prefix(holes, sums, 1, all_holes);   // also: dst and src are complete
    const int32_t thread = blockIdx.x * kScanThreads + threadIdx.x;
    if (thread == 0) scratch[0] = (int32_t)all_holes;
    for (int64_t i = thread; i < all_holes; i += kScanCtas * kScanThreads) {
        const int32_t to = dst[i], from = src[i];
        remap[from] = to;
        refs[to] = refs[from];
        refs[from] = 0;
    }
    ptx::cluster_sync();
}

__device__ void remap_table(int32_t num_pages, int32_t* table, int64_t entries, const int32_t* remap, int32_t* err,
                            int32_t block, int32_t blocks) {
    for (int64_t e = (int64_t)block * kMoveThreads + threadIdx.x; e < entries; e += (int64_t)blocks * kMoveThreads) {
        const int32_t page = table[e];
        if (page < 0 || page >= num_pages) {
            flag(err, ATTN_DEVICE_ERR_PAGE_ID);
            continue;
        }
        const int32_t to = remap[page];
        if (to < 0) flag(err, ATTN_DEVICE_ERR_PAGES);   // nobody held it
        table[e] = to;
    }
}

// ------------------------------------------------------------------------ copy

__global__ void __launch_bounds__(kMoveThreads)
copy_kernel(const __grid_constant__ PagePools pools, int32_t num_pages, const int32_t* src, const int32_t* dst,
            const int32_t* n_dev, int64_t n, int32_t pieces, int32_t* err) {
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    if (n_dev) n = min(n, (int64_t)*n_dev);
    const int64_t per_page = (int64_t)pools.n * pieces, units = n * per_page;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t i = u / per_page;
        const int32_t x = (int32_t)(u - i * per_page), k = x / pieces, piece = x - k * pieces;
        const int64_t bytes = pools.bytes[k], off = (int64_t)piece * kMoveBytes;
        if (off >= bytes) continue;
        const int32_t from = src[i], to = dst[i];
        if (from < 0 || from >= num_pages || to < 0 || to >= num_pages) {
            if (threadIdx.x == 0 && x == 0) flag(err, ATTN_DEVICE_ERR_PAGE_ID);
            continue;
        }
        const int chunks = (int)min((int64_t)kMoveBytes, bytes - off) / 16;
        const uint4* a = reinterpret_cast<const uint4*>(pools.pool[k] + from * bytes + off);
        uint4* b = reinterpret_cast<uint4*>(pools.pool[k] + to * bytes + off);
        constexpr int kChunks = kMoveBytes / 16 / kMoveThreads;
        uint4 v[kChunks];
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
            if ((int)threadIdx.x + j * kMoveThreads < chunks) v[j] = a[threadIdx.x + j * kMoveThreads];
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
            if ((int)threadIdx.x + j * kMoveThreads < chunks) b[threadIdx.x + j * kMoveThreads] = v[j];
    }
}

__global__ void __launch_bounds__(kMoveThreads)
share_kernel(int32_t* refs, int32_t num_pages, const PageFork f, int32_t* err) {
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    share_pages(refs, num_pages, f, err, blockIdx.x, gridDim.x);
}

__global__ void __launch_bounds__(kMoveThreads)
remap_kernel(int32_t num_pages, int32_t* table, int64_t entries, const int32_t* remap, int32_t* err) {
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    remap_table(num_pages, table, entries, remap, err, blockIdx.x, gridDim.x);
}

// CTAs for `work` items of a CTA each, at most `per_sm` per SM; 0: no device.
int grid_for(int64_t work, int per_sm) {
    int32_t sms = 0;
    if (!current_sm_count(&sms)) return 0;
    const int64_t cap = (int64_t)sms * per_sm;
    return (int)(work < cap ? work : cap);
}

attn_status done(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

}  // namespace

attn_status launch_pages_alloc(int32_t* refs, int32_t num_pages, int32_t n, int32_t* page_ids, int32_t* err,
                               cudaStream_t stream) {
    return done(launch_dependent(alloc_kernel, dim3(kScanCtas), kScanThreads, 0, stream, refs, num_pages, n, page_ids, err));
}

attn_status launch_pages_free(int32_t* refs, int32_t num_pages, const int32_t* page_ids, int64_t n, int32_t* err,
                              cudaStream_t stream) {
    const int grid = grid_for((n + kMoveThreads - 1) / kMoveThreads, kMoveCtasPerSm);
    if (grid == 0) return ATTN_ERR_CUDA;
    return done(launch_dependent(free_kernel, dim3(grid), kMoveThreads, 0, stream, refs, num_pages, page_ids, n, err));
}

attn_status launch_pages_fork(int32_t* refs, int32_t num_pages, const PageFork& f, int32_t* scratch, int32_t* err,
                              cudaStream_t stream) {
    if (cudaError_t e = launch_dependent(fork_kernel, dim3(kScanCtas), kScanThreads, 0, stream, refs, num_pages, f, scratch, err);
        e != cudaSuccess)
        return ATTN_ERR_CUDA;
    if (f.out_len == 0) return ATTN_OK;
    const int grid = grid_for((f.out_len + kMoveThreads - 1) / kMoveThreads, kMoveCtasPerSm);
    if (grid == 0) return ATTN_ERR_CUDA;
    return done(launch_dependent(share_kernel, dim3(grid), kMoveThreads, 0, stream, refs, num_pages, f, err));
}

attn_status launch_pages_compact(int32_t* refs, int32_t num_pages, int32_t* page_table, int64_t entries, int32_t* remap,
                                 int32_t* scratch, int32_t* err, cudaStream_t stream) {
    if (cudaError_t e = launch_dependent(compact_kernel, dim3(kScanCtas), kScanThreads, 0, stream, refs, num_pages,
                                         remap, scratch);
        e != cudaSuccess)
        return ATTN_ERR_CUDA;
    if (entries == 0) return ATTN_OK;
    const int grid = grid_for((entries + kMoveThreads - 1) / kMoveThreads, kMoveCtasPerSm);
    if (grid == 0) return ATTN_ERR_CUDA;
    return done(launch_dependent(remap_kernel, dim3(grid), kMoveThreads, 0, stream, num_pages, page_table, entries,
                                 static_cast<const int32_t*>(remap), err));
}

attn_status launch_pages_copy(const PagePools& pools, int32_t num_pages, const int32_t* src, const int32_t* dst,
                              const int32_t* n, int64_t n_max, int32_t* err, cudaStream_t stream) {
    int64_t largest = 0;
    for (int32_t k = 0; k < pools.n; ++k) largest = pools.bytes[k] > largest ? pools.bytes[k] : largest;
    const int64_t pieces = (largest + kMoveBytes - 1) / kMoveBytes;
    const int grid = grid_for(n_max * pools.n * pieces, kMoveCtasPerSm);
    if (grid == 0) return ATTN_ERR_CUDA;
    return done(launch_dependent(copy_kernel, dim3(grid), kMoveThreads, 0, stream, pools, num_pages, src, dst, n, n_max,
                                 (int32_t)pieces, err));
}

}  // namespace attn
