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
// Copies are memory-bound: CTAs take (page, pool, 16 KB) pieces, 64 bytes per
// thread in flight.  How many pages move is only known on the device, so the
// grid reads the count there; nothing waits on the host.
//
// Measured (in a graph): a fork of 32 children of 8 heads x 64 dims in two layers 11
// us with its free, 1,024 children (382 MB copied, 37K entries shared) 96; the scan of
// 36K pages and its moves 12 (latency: two exchanges of the cluster and three
// dependent loads), the copy after it 160 (1.12 GB, 7.0 TB/s).
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
// CTAs per SM of a copy's grid, eight times what is resident: the hardware hands them
// out as SMs come free (half a pool of 36K 32 KB pages in two layers: 195 us with 8,
// 185 with 16, 179 with 64; a grid without a cap would be mostly empty where few of
// the pages that could move do).
constexpr int kMoveCtasPerSm = 64;

// ------------------------------------------------------- sums over the cluster

template <int N>
struct ClusterSums {
    int64_t warp[N][32];
    int64_t total[N];   // of this CTA
};

// Exclusive prefixes of v over all threads of the cluster in order, and the sums,
// of N values at once (a barrier of the cluster costs about a microsecond).  Every
// thread calls it, once per `s`; what threads wrote before is visible after it.
template <int N>
__device__ __forceinline__ void cluster_prefix(int64_t (&v)[N], int64_t (&sum)[N], ClusterSums<N>& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        inc[k] = v[k];
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, inc[k], o);
            if (lane >= o) inc[k] += x;
        }
        if (lane == 31) s.warp[k][warp] = inc[k];
    }
    __syncthreads();
    if (warp < N) {   // warp k: the warps' sums of value k, up to each
        int64_t x = s.warp[warp][lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        s.warp[warp][lane] = x;
        if (lane == 31) s.total[warp] = x;
    }
    ptx::cluster_sync();
    const uint32_t rank = ptx::cluster_rank();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        int64_t before = warp > 0 ? s.warp[k][warp - 1] : 0;
        sum[k] = 0;
#pragma unroll
        for (uint32_t c = 0; c < kScanCtas; ++c) {
            const int64_t x = ptx::ld_cluster_s64(ptx::smem_u32(&s.total[k]), c);
            before += c < rank ? x : 0;
            sum[k] += x;
        }
        v[k] = before + inc[k] - v[k];
    }
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
    __shared__ ClusterSums<1> sums;
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    const WarpPages part(num_pages);
    int64_t before[1] = {count_free(refs, num_pages, part)}, all[1];
    cluster_prefix(before, all, sums);
    const int64_t free_pages = all[0];
    take_free(refs, num_pages, part, warp_base(before[0]), n, [&](int64_t rank, int32_t page) {
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
    __shared__ ClusterSums<3> sums;
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    const WarpPages part(num_pages);
    const int32_t thread = blockIdx.x * kScanThreads + threadIdx.x, threads = kScanCtas * kScanThreads;
    const int32_t c0 = (int32_t)((int64_t)thread * f.n / threads), c1 = (int32_t)((int64_t)(thread + 1) * f.n / threads);
    int64_t v[3] = {0, 0, 0}, all[3];   // table entries, pages to copy, free pages
    bool bad = false;
    for (int32_t c = c0; c < c1; ++c) {
        const Child child(f, c);
        v[0] += child.pages;
        v[1] += child.part;
        bad |= child.bad;
    }
    v[2] = count_free(refs, num_pages, part);
    cluster_prefix(v, all, sums);
    const bool refused = all[0] > f.out_len;
    const int64_t all_entries = all[0], all_fresh = all[1], free_pages = all[2];
    int64_t at = v[0], rank = v[1];
    int32_t *dst = scratch + kMoveHead, *src = dst + f.n;
    if (!refused)
        take_free(refs, num_pages, part, warp_base(v[2]), all_fresh, [&](int64_t r, int32_t page) {
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

// Entries of a child but for a copied last page are its parent's own pages, held
// once more.  The search for an entry's child begins in shared memory, in up to
// kShareOffsets of the children's offsets.
constexpr int kShareOffsets = 1024;
__device__ void share_pages(int32_t* refs, int32_t num_pages, const PageFork& f, int32_t* err, int32_t block, int32_t blocks) {
    __shared__ int32_t offsets[kShareOffsets];
    const int32_t step = (f.n - 1) / kShareOffsets + 1, known = (f.n - 1) / step + 1;   // (n >= 1)
    for (int32_t k = threadIdx.x; k < known; k += kMoveThreads) offsets[k] = f.indptr_out[k * step];
    const int64_t total = f.indptr_out[f.n];
    __syncthreads();
    for (int64_t e = (int64_t)block * kMoveThreads + threadIdx.x; e < total; e += (int64_t)blocks * kMoveThreads) {
        int32_t lo = 0, hi = known - 1;   // the last child that begins at or before e
        while (lo < hi) {
            const int32_t mid = lo + (hi - lo + 1) / 2;
            if (offsets[mid] <= e) lo = mid;
            else hi = mid - 1;
        }
        int32_t first = offsets[lo];
        lo *= step;
        hi = (int32_t)min((int64_t)lo + step, (int64_t)f.n) - 1;
        while (lo < hi) {
            const int32_t mid = lo + (hi - lo + 1) / 2, x = f.indptr_out[mid];
            if (x <= e) {
                lo = mid;
                first = x;
            } else {
                hi = mid - 1;
            }
        }
        const Child child(f, lo);
        const int32_t j = (int32_t)(e - first);
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
    __shared__ ClusterSums<1> sums, hole_sums;
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    const WarpPages part(num_pages);
    int32_t *dst = scratch + kMoveHead, *src = dst + num_pages / 2;
    int64_t before[1] = {count_free(refs, num_pages, part)}, all_free[1], holes[1] = {0}, all_holes[1];
    cluster_prefix(before, all_free, sums);
    int64_t base = warp_base(before[0]);
    const int64_t used = num_pages - all_free[0];
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
                    ++holes[0];
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
    cluster_prefix(holes, all_holes, hole_sums);   // also: dst and src are complete
    const int32_t thread = blockIdx.x * kScanThreads + threadIdx.x;
    if (thread == 0) scratch[0] = (int32_t)all_holes[0];
    for (int64_t i = thread; i < all_holes[0]; i += kScanCtas * kScanThreads) {
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

// What the first CTAs of a copy do: the table that goes with it (kNone: nothing).
enum class Table { kNone, kShare, kRemap };
struct TableWork {
    int32_t blocks;      // CTAs
    int32_t* refs;       // kShare
    PageFork fork;
    int32_t* table;      // kRemap
    int64_t entries;
    const int32_t* remap;
};

template <Table kTable>
__global__ void __launch_bounds__(kMoveThreads)
copy_kernel(const __grid_constant__ PagePools pools, int32_t num_pages, const int32_t* src, const int32_t* dst,
            const int32_t* n_dev, int64_t n, int32_t pieces, int32_t* err, const __grid_constant__ TableWork t) {
    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    if constexpr (kTable != Table::kNone) {
        if ((int32_t)blockIdx.x < t.blocks) {
            if constexpr (kTable == Table::kShare)
                share_pages(t.refs, num_pages, t.fork, err, blockIdx.x, t.blocks);
            else
                remap_table(num_pages, t.table, t.entries, t.remap, err, blockIdx.x, t.blocks);
            return;
        }
    }
    const int32_t block = kTable == Table::kNone ? blockIdx.x : blockIdx.x - t.blocks;
    const int32_t blocks = kTable == Table::kNone ? gridDim.x : gridDim.x - t.blocks;
    if (n_dev) n = min(n, (int64_t)*n_dev);
    const int64_t per_page = (int64_t)pools.n * pieces, units = n * per_page;
    for (int64_t u = block; u < units; u += blocks) {
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

// CTAs for `work` items of a CTA each; 0: no device.
int grid_for(int64_t work) {
    int32_t sms = 0;
    if (!current_sm_count(&sms)) return 0;
    const int64_t cap = (int64_t)sms * kMoveCtasPerSm;
    return (int)(work < cap ? work : cap);
}

attn_status done(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

template <Table kTable>
attn_status copy(const PagePools& pools, int32_t num_pages, const int32_t* src, const int32_t* dst, const int32_t* n,
                 int64_t n_max, int32_t* err, TableWork t, int64_t entries, cudaStream_t stream) {
    int64_t largest = 0;
    for (int32_t k = 0; k < pools.n; ++k) largest = pools.bytes[k] > largest ? pools.bytes[k] : largest;
    const int64_t pieces = (largest + kMoveBytes - 1) / kMoveBytes, work = n_max * pools.n * pieces;
    const int64_t table_work = kTable == Table::kNone ? 0 : (entries + kMoveThreads - 1) / kMoveThreads;
    if (work + table_work == 0) return ATTN_OK;
    const int grid = grid_for(work);
    t.blocks = grid_for(table_work);
    if (grid + t.blocks == 0) return ATTN_ERR_CUDA;
    return done(launch_dependent(copy_kernel<kTable>, dim3(grid + t.blocks), kMoveThreads, 0, stream, pools, num_pages, src,
                                 dst, n, n_max, (int32_t)pieces, err, t));
}

}  // namespace

attn_status launch_pages_alloc(int32_t* refs, int32_t num_pages, int32_t n, int32_t* page_ids, int32_t* err,
                               cudaStream_t stream) {
    return done(launch_dependent(alloc_kernel, dim3(kScanCtas), kScanThreads, 0, stream, refs, num_pages, n, page_ids, err));
}

attn_status launch_pages_free(int32_t* refs, int32_t num_pages, const int32_t* page_ids, int64_t n, int32_t* err,
                              cudaStream_t stream) {
    const int grid = grid_for((n + kMoveThreads - 1) / kMoveThreads);
    if (grid == 0) return ATTN_ERR_CUDA;
    return done(launch_dependent(free_kernel, dim3(grid), kMoveThreads, 0, stream, refs, num_pages, page_ids, n, err));
}

attn_status launch_pages_copy(const PagePools& pools, int32_t num_pages, const int32_t* src, const int32_t* dst,
                              const int32_t* n, int64_t n_max, int32_t* err, cudaStream_t stream) {
    return copy<Table::kNone>(pools, num_pages, src, dst, n, n_max, err, {}, 0, stream);
}

attn_status launch_pages_fork(int32_t* refs, int32_t num_pages, const PageFork& f, const PagePools& pools,
                              int32_t* scratch, int32_t* err, cudaStream_t stream) {
    if (launch_dependent(fork_kernel, dim3(kScanCtas), kScanThreads, 0, stream, refs, num_pages, f, scratch, err) != cudaSuccess)
        return ATTN_ERR_CUDA;
    if (f.n == 0) return ATTN_OK;
    TableWork t = {};
    t.refs = refs;
    t.fork = f;
    const int32_t* dst = scratch + kMoveHead;
    return copy<Table::kShare>(pools, num_pages, dst + f.n, dst, scratch, f.n, err, t, f.out_len, stream);
}

attn_status launch_pages_compact(int32_t* refs, int32_t num_pages, int32_t* page_table, int64_t entries, int32_t* remap,
                                 const PagePools& pools, int32_t* scratch, int32_t* err, cudaStream_t stream) {
    if (launch_dependent(compact_kernel, dim3(kScanCtas), kScanThreads, 0, stream, refs, num_pages, remap, scratch) != cudaSuccess)
        return ATTN_ERR_CUDA;
    TableWork t = {};
    t.table = page_table;
    t.entries = entries;
    t.remap = remap;
    const int32_t* dst = scratch + kMoveHead;
    return copy<Table::kRemap>(pools, num_pages, dst + num_pages / 2, dst, scratch, num_pages / 2, err, t, entries, stream);
}

}  // namespace attn
