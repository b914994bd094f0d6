// Rotary positions with one or more axes: q and k rows turned by pairs of
// dims, alone or with the turned k and the v written into their HND pages.
//
// Pair p of a row turns by theta = positions[axis[p]][row] * inv_freq[p]:
// (x, y) -> scale (x cos - y sin, x sin + y cos).  Only theta modulo a full
// turn counts, and a far position times a frequency has more bits than fp32 (or
// fp32 pairs) keep, so the frequency is held in turns as a 64-bit fixed-point
// fraction F = round(inv_freq / 2 pi * 2^64): position * F modulo 2^64 is then
// the angle's fraction of a turn, exact but for the rounding of F (2^31 * 2^-65
// of a turn at the farthest position), by one integer product.  Its upper 32
// bits, as a signed number of half turns, go to sincospif: in fp32, which rounds them
// by up to 2^-25 of a half turn, less than 2^-23 radians (bf16 then rounds the row by
// 2^-8 of its values).
//
// Memory-bound: each row is read and written once, in 16-byte chunks.  A thread
// turns 8 pairs at a time, an item: two chunks, which hold the pairs' halves (chunk
// i and the one half the turned width on) or, with neighbouring dims paired, 4
// pairs each.  All rows' items, head by head, are one long list, of which a CTA has
// 1,024, four per thread, loaded at once: every thread of every CTA has the same
// work, wherever the rows begin.  (CTAs of whole rows left the last of their items
// to a quarter of their loads.)  A row's angles are the same for all heads: a CTA
// computes its rows' cosines and sines (up to 63 rows', where they have few heads)
// into shared memory while its loads are on their way.
//
// Measured: 18K rows of 72 heads of 128 dims with their pages (733 MB) 107 us, 6.9
// TB/s, the copy rate (issue 68% of the slots); 123 with CTAs of whole rows; 118 with
// the pages looked up after the angles and a pair's frequency and axis read from
// the parameters by each lane (its own: 32 reads one after the other), 123 and 135
// with 2 and 6 items per thread then.  64 rows: 2.7 us in a graph, a launch and three
// dependent loads.  Rows of few heads are bound by the angles' chain: a CTA of rows of
// two heads has 62 of them, so that a thread has up to eight angles one after the
// other, each after the first behind its position's load, and half of its items are
// none.  400K rows of two heads of 64 dims, where the bytes take 30 us: 61 us; 50 with
// positions computed instead of loaded, 54 without sines and cosines, 41 without both.
#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kRopeThreads = 256;
static_assert(kRopeThreads / 32 * 8 >= kRopeMaxPairs, "the warps load the table");
constexpr int kRopeUnroll = 4;    // items of a thread whose loads are in flight together
constexpr int kRopeMaxRows = 64;  // rows that a CTA's items may lie in

struct RopeArgs {
    RopeTable t;
    const int32_t* positions;   // [n_axes][rows]
    int64_t rows;
    int32_t heads, Hq, Hkv, inverse;   // heads: of a CTA
    const uint4 *q, *k, *v;
    uint4 *q_out, *k_out;       // k_out: the page pool where kCache
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;   // 16-byte chunks
    // kCache
    const int2* slots;          // per row: page-table slot, row in the page
    const int32_t* page_table;
    int32_t P, num_pages;
    int32_t* err;
};

// Turns 8 pairs; t: their (cos, sin), two pairs per float4, `stride` float4 apart.
template <bool kInter>
__device__ __forceinline__ void turn(uint4& lo, uint4& hi, const float4* t, int stride) {
    uint32_t* a = reinterpret_cast<uint32_t*>(&lo);
    uint32_t* b = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 cs = t[j * stride];   // pairs 2j and 2j + 1
        if constexpr (kInter) {
            uint32_t* w = j < 2 ? a : b;
            const int e = (j & 1) * 2;
            const float2 u = ptx::unpack_bf16x2(w[e]), v = ptx::unpack_bf16x2(w[e + 1]);
            w[e] = ptx::pack_bf16x2(fmaf(u.x, cs.x, -u.y * cs.y), fmaf(u.x, cs.y, u.y * cs.x));
            w[e + 1] = ptx::pack_bf16x2(fmaf(v.x, cs.z, -v.y * cs.w), fmaf(v.x, cs.w, v.y * cs.z));
        } else {
            const float2 x = ptx::unpack_bf16x2(a[j]), y = ptx::unpack_bf16x2(b[j]);
            a[j] = ptx::pack_bf16x2(fmaf(x.x, cs.x, -y.x * cs.y), fmaf(x.y, cs.z, -y.y * cs.w));
            b[j] = ptx::pack_bf16x2(fmaf(x.x, cs.y, y.x * cs.x), fmaf(x.y, cs.w, y.y * cs.z));
        }
    }
}

template <int D, bool kInter, bool kCache>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int kItems = D / 16;                       // items of a head: 16 dims each
    __shared__ float4 cs_s[kRopeMaxRows * D / 4];        // [row][pair pair][item]: (cos, sin) of two pairs
    __shared__ uint64_t freq_s[kRopeMaxPairs];
    __shared__ int64_t page_s[kRopeMaxRows];             // kCache: first chunk of the row in its page's K, or -1
    // A thread's items lie at the same place in their heads, kStep heads apart.
    constexpr int kStep = kRopeThreads / kItems;
    const int tid = threadIdx.x, i = tid % kItems;
    const int turned = a.t.pairs / 8;                    // items of a head that turn
    const int heads = a.Hq + a.Hkv * (kCache ? 2 : 1);
    const uint64_t first = (uint64_t)blockIdx.x * a.heads;   // the CTA's heads, counted through the rows
    const int64_t row0 = first >> 32 ? (int64_t)(first / (uint32_t)heads) : (int64_t)((uint32_t)first / (uint32_t)heads);
    const int skip = (int)(first - (uint64_t)row0 * heads);  // heads of row 0 before them
    const int n = (int)min((int64_t)a.heads, a.rows * heads - (int64_t)first), rows = (skip + n - 1) / heads + 1;
    const int step_rows = kStep / heads, step_heads = kStep - step_rows * heads;
    const int y = skip + tid / kItems, r0 = y / heads, h0 = y - r0 * heads;
    const bool turns = i < turned;
    const int c0 = !kInter && turns ? i : 2 * i, c1 = !kInter && turns ? i + turned : 2 * i + 1;   // chunks of the item

    ptx::grid_dependency_wait();
    ptx::grid_dependents_go();
    int2 slot = make_int2(0, 0);   // the longest chain of loads begins first
    if (kCache && tid < rows) slot = a.slots[row0 + tid];
    uint4 lo[kRopeUnroll], hi[kRopeUnroll];
    {
        int r = r0, h = h0;
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            if (tid / kItems + u * kStep < n) {
                const int64_t row = row0 + r;
                if (kCache && h >= a.Hq + a.Hkv) {
                    const uint4* src = a.v + row * a.v_stride + (h - a.Hq - a.Hkv) * (D / 8);
                    lo[u] = src[2 * i];
                    hi[u] = src[2 * i + 1];
                } else {
                    const uint4* src = h < a.Hq ? a.q + row * a.q_stride + h * (D / 8)
                                                : a.k + row * a.k_stride + (h - a.Hq) * (D / 8);
                    lo[u] = src[c0];
                    hi[u] = src[c1];
                }
            }
            r += step_rows;
            h += step_heads;
            if (h >= heads) {
                h -= heads;
                ++r;
            }
        }
    }

    // A thread has one pair, of every few rows.
    const int pair_rows = kRopeThreads / a.t.pairs, first_row = tid / a.t.pairs, p = tid - first_row * a.t.pairs;
    const uint64_t axes = p < 32 ? (p < 16 ? a.t.axes[0] : a.t.axes[1]) : (p < 48 ? a.t.axes[2] : a.t.axes[3]);
    const int32_t* positions = a.positions + (int64_t)(axes >> (p & 15) * 4 & 15) * a.rows + row0;
    const bool mine = first_row < pair_rows && first_row < rows;
    const int32_t first_pos = mine ? positions[first_row] : 0;
    // The frequencies, from the parameters one at a time, a warp 8 of them: lanes that
    // read different parameters wait for one another (so the axes are packed).
    for (int k = 0; k < 8; ++k) {
        const int x = (tid >> 5) * 8 + k;
        if ((tid & 31) == 0 && x < a.t.pairs) freq_s[x] = a.t.freq[x];
    }
    if (kCache && tid < rows) {
        const int32_t page = a.page_table[slot.x];
        const bool in = page >= 0 && page < a.num_pages;
        if (!in) atomicOr(a.err, ATTN_DEVICE_ERR_PAGE_ID);
        page_s[tid] = in ? ((int64_t)page * 2 * a.Hkv * a.P + slot.y) * (D / 8) : -1;
    }
    __syncthreads();
    for (int r = first_row; mine && r < rows; r += pair_rows) {
        int64_t pos = r == first_row ? first_pos : positions[r];
        if (a.inverse) pos = -pos;
        const uint64_t angle = (uint64_t)pos * freq_s[p];
        float s, c;
        sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &s, &c);
        const int item = p >> 3, j = p & 7;
        reinterpret_cast<float2*>(cs_s)[(r * (D / 4) + (j >> 1) * turned + item) * 2 + (j & 1)] =
            make_float2(c * a.t.scale, s * a.t.scale);
    }
    __syncthreads();

    int r = r0, h = h0;
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
        if (tid / kItems + u * kStep < n) {
            const bool is_v = kCache && h >= a.Hq + a.Hkv;
            if (turns && !is_v) turn<kInter>(lo[u], hi[u], cs_s + r * (D / 4) + i, turned);
            uint4* dst;
            if (h < a.Hq)
                dst = a.q_out + (row0 + r) * a.q_out_stride + h * (D / 8);
            else if constexpr (kCache)
                dst = page_s[r] < 0 ? nullptr : a.k_out + page_s[r] + (int64_t)(h - a.Hq) * a.P * (D / 8);   // V's heads follow K's
            else
                dst = a.k_out + (row0 + r) * a.k_out_stride + (h - a.Hq) * (D / 8);
            if (!kCache || dst != nullptr) {
                dst[is_v ? 2 * i : c0] = lo[u];
                dst[is_v ? 2 * i + 1 : c1] = hi[u];
            }
        }
        r += step_rows;
        h += step_heads;
        if (h >= heads) {
            h -= heads;
            ++r;
        }
    }
}

template <int D, bool kInter, bool kCache>
attn_status launch(RopeArgs& a, cudaStream_t stream) {
    int32_t sms = 0;
    if (!current_sm_count(&sms)) return ATTN_ERR_CUDA;
    // One item per thread where that leaves no SM with more than two CTAs.  Rows of 80
    // heads of 64 dims, one item against four, us in a graph: 16 rows 2.05 against 2.74, 64
    // 2.10 against 2.82, 256 3.17 against 2.88, 512 4.18 against 3.45.
    const int64_t heads = (int64_t)a.Hq + a.Hkv * (kCache ? 2 : 1), total = a.rows * heads;
    const int64_t step = kRopeThreads / (D / 16), most = total <= 2 * sms * step ? step : kRopeUnroll * step;
    a.heads = (int32_t)std::min<int64_t>(most, (kRopeMaxRows - 2) * heads);
    const int64_t ctas = (total + a.heads - 1) / a.heads;
    if (ctas > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
    return launch_dependent(rope_kernel<D, kInter, kCache>, dim3((unsigned)ctas), kRopeThreads, 0, stream, a) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}

template <bool kCache>
attn_status launch(RopeArgs& a, int32_t head_dim, bool inter, cudaStream_t stream) {
    if (head_dim == 64) return inter ? launch<64, true, kCache>(a, stream) : launch<64, false, kCache>(a, stream);
    return inter ? launch<128, true, kCache>(a, stream) : launch<128, false, kCache>(a, stream);
}

}  // namespace

attn_status launch_rope(const RopeTable& t, bool inter, bool inverse, const int32_t* positions, int64_t rows,
                        int32_t head_dim, const RopeRows& q, const RopeRows& k, cudaStream_t stream) {
    RopeArgs a = {};
    a.t = t;
    a.positions = positions;
    a.rows = rows;
    a.Hq = q.heads;
    a.Hkv = k.heads;
    a.inverse = inverse;
    a.q = static_cast<const uint4*>(q.in);
    a.k = static_cast<const uint4*>(k.in);
    a.q_out = static_cast<uint4*>(q.out);
    a.k_out = static_cast<uint4*>(k.out);
    a.q_stride = q.stride / 8;
    a.k_stride = k.stride / 8;
    a.q_out_stride = q.out_stride / 8;
    a.k_out_stride = k.out_stride / 8;
    return launch<false>(a, head_dim, inter, stream);
}

attn_status launch_append_kv_rope(attn_plan_s* plan, const RopeTable& t, bool inter, const int32_t* positions,
                                  const RopeRows& q, const RopeRows& k, const RopeRows& v, cudaStream_t stream) {
    RopeArgs a = {};
    a.t = t;
    a.positions = positions;
    a.rows = plan->info.total_qo_rows;
    a.Hq = plan->Hq;
    a.Hkv = plan->Hkv;
    a.q = static_cast<const uint4*>(q.in);
    a.k = static_cast<const uint4*>(k.in);
    a.v = static_cast<const uint4*>(v.in);
    a.q_out = static_cast<uint4*>(q.out);
    a.k_out = static_cast<uint4*>(k.out);
    a.q_stride = q.stride / 8;
    a.k_stride = k.stride / 8;
    a.v_stride = v.stride / 8;
    a.q_out_stride = (int64_t)plan->Hq * plan->D / 8;
    a.slots = reinterpret_cast<const int2*>(plan->ws + plan->layout.append);
    a.page_table = plan->page_table;
    a.P = plan->P;
    a.num_pages = plan->num_pages;
    a.err = reinterpret_cast<int32_t*>(plan->ws + plan->layout.err);
    return launch<true>(a, plan->D, inter, stream);
}

}  // namespace attn
