// The pages of a paged cache: taking, freeing, forking and moving them together (the table and
// the reference counts), copying them (the data), and moving the rows of accepted drafts.
//
// refs[p] counts the table entries that name page p; a page of count <= 0 is free. Which page a
// new entry gets is defined, so that results do not depend on timing: the entries that want one,
// in the order of the table, get the free pages, lowest first. So does a move: the k-th page in
// use at or above the number U of pages in use goes to the k-th free page below U.
//
// Taking, forking and compacting need ranks over the whole pool. They run in one cluster of 8
// CTAs: each counts its eighth of the pool with ballots, the counts are exchanged through
// distributed shared memory, and what passes from CTA to CTA otherwise (the list of free pages,
// the moves) goes through the handle's workspace between two cluster barriers. No CTA waits for
// one of another launch, and a call is one launch. On rows of up to some hundred entries it is bound
// by its latency: five dependent trips to memory and two cluster barriers (compact: three). Beyond,
// take and fork are bound by the walk along a row, which one warp does, 32 entries at a time and none
// ahead (a CTA has 32 rows at least, so few rows leave most CTAs idle). One sequence, pages of 16
// rows, between events that add about 5 us: 256 entries fork 15 and take 13 us, 1024 entries 29 and 23,
// 8192 entries (131072 tokens) 177 and 124, where free, dealt over the GPU, takes 7 and compact, whose
// entries all 8 CTAs share, 15. 16 sequences and 64 children of 8192 entries: 203, 169, 7 and 40.
//
// Copies are bound by HBM: a CTA moves 16 KB, four 16-byte vectors in flight per thread, six CTAs
// on an SM (40 registers a thread), and the GPU deals the CTAs. CTAs that run together have the same part of many pages:
// children of one parent, wherever they stand in the list, then find its rows in L2. 508 copies of
// the last pages of 64 parents, 512 KB each (267 MB written, 34 MB of sources): 55 us; page by page
// 75, and on a grid of 8 CTAs per SM, whose last round is not full, 82. 206 MB of pages moved
// together: 36.6 us (page by page 38.5). 2 and 8 vectors a thread: 61 and 61 us, 44 and 50.
#include <cooperative_groups.h>

#include "ub_attn.h"
#include "ub_device.cuh"
#include "ub_internal.h"

namespace cg = cooperative_groups;

namespace ubk {
namespace {

constexpr int POOL_CTAS = 8;
constexpr int POOL_THREADS = 1024;
constexpr int POOL_WARPS = POOL_THREADS / 32;
constexpr int STEPS = 8;                   // loads in flight of a warp that counts
constexpr int COPY_THREADS = 256, COPY_VECS = 4, COPY_GRID = 1 << 20;
constexpr int ACCEPT_THREADS = 128, ACCEPT_ROWS = 8;

__device__ __forceinline__ void report(int32_t *status, int code) { atomicCAS(status, 0, code); }

// The share [lo, hi) of CTA `rank` of n things, a multiple of 32 each but the last.
struct Span {
    int64_t lo, hi;
};
__device__ __forceinline__ Span share(int64_t n, int rank)
{
    const int64_t per = (n + 32 * POOL_CTAS - 1) / (32 * POOL_CTAS) * 32;
    const int64_t lo = per * rank < n ? per * rank : n;
    return Span{lo, lo + per < n ? lo + per : n};
}

__device__ __forceinline__ int block_sum(int v, int *scratch)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if (lane == 0) scratch[warp] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, scratch[lane]);
}

// Sum over the warps before this one of a value of each warp, and over all of them.
__device__ __forceinline__ int warps_before(int v, int *scratch, int *total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) scratch[warp] = v;
    __syncthreads();
    const int x = scratch[lane];
    *total = __reduce_add_sync(0xffffffffu, x);
    return __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
}

// What the CTAs tell one another, and its sums over the CTAs before this one and over all.
constexpr int TOLD = 3;
struct Sums {
    int before, all;
};
__device__ Sums over_ctas(cg::cluster_group &cluster, int *told, int which)
{
    Sums s{0, 0};
    const int rank = static_cast<int>(cluster.block_rank());
    for (int c = 0; c < POOL_CTAS; ++c) {
        const int v = cluster.map_shared_rank(told, c)[which];
        s.all += v;
        if (c < rank) s.before += v;
    }
    return s;
}

// Pages of a span for which `is(refs[p], p)` holds.
template <typename F>
__device__ int count_pages(const int32_t *refs, Span s, int *scratch, F is)
{
    int n = 0;
    for (int64_t p = s.lo + threadIdx.x; p < s.hi; p += POOL_THREADS) n += is(refs[p], p) ? 1 : 0;
    return block_sum(n, scratch);
}

// Calls f(p, refs[p], k) for every page of the span, k being the number of pages before p in
// the span for which `is` holds; stops behind the `most`-th of those.
template <typename I, typename F>
__device__ void ranked_pages(const int32_t *refs, Span s, int64_t most, int *scratch, I is, F f)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t base = 0;
    for (int64_t p0 = s.lo; p0 < s.hi && base < most; p0 += STEPS * POOL_THREADS) {
        const int64_t mine = p0 + warp * (32 * STEPS) + lane;
        int r[STEPS];
        uint32_t hit[STEPS];
        int n = 0;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) r[i] = mine + i * 32 < s.hi ? refs[mine + i * 32] : 0;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            hit[i] = __ballot_sync(0xffffffffu, mine + i * 32 < s.hi && is(r[i], mine + i * 32));
            n += __popc(hit[i]);
        }
        int total;
        int64_t k = base + warps_before(n, scratch, &total);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            if (mine + i * 32 < s.hi) f(mine + i * 32, r[i], k + __popc(hit[i] & ((1u << lane) - 1u)));
            k += __popc(hit[i]);
        }
        base += total;
    }
}

struct IsFree {
    __device__ bool operator()(int r, int64_t) const { return r <= 0; }
};

// ---------------------------------------------------------------- take and fork

// Table entries [first, last) of row s that a call may fill.
struct Entries {
    int64_t first, last;
};
__device__ __forceinline__ Entries take_range(const PoolParams &p, int s)
{
    const int64_t b = p.begin[s], e = p.end[s], cap = static_cast<int64_t>(p.width) << p.page_shift;
    if (e <= b) return Entries{0, 0};  // no rows, wherever they would be
    if (b < 0 || e > cap) report(p.status, UB_ERR_ARG);
    if (e <= 0 || b >= cap) return Entries{0, 0};
    return Entries{(b < 0 ? 0 : b) >> p.page_shift, ((e > cap ? cap : e) + (int64_t(1) << p.page_shift) - 1) >> p.page_shift};
}

// The parent of child i, the pages it shares, and whether it needs a copy of a part of a page.
struct Child {
    int source;
    int whole;
    int part;
};
__device__ __forceinline__ Child child_of(const PoolParams &p, int i)
{
    Child c{p.source[i], 0, 0};
    if (c.source < 0 || c.source >= p.rows) {
        report(p.status, UB_ERR_ARG);
        c.source = -1;
        return c;
    }
    const int64_t cap = static_cast<int64_t>(p.width) << p.page_shift;
    const int64_t len = p.begin[c.source];
    if (len < 0 || len > cap) report(p.status, UB_ERR_ARG);
    const int64_t n = len < 0 ? 0 : (len > cap ? cap : len);
    c.whole = static_cast<int>(n >> p.page_shift);
    // no copy of what is not there: a page outside the pool, or none
    if ((n & ((int64_t(1) << p.page_shift) - 1)) != 0) {
        const int32_t page = p.table[c.source * p.table_row + c.whole];
        c.part = page >= 0 && page < p.pages ? 1 : 0;
        if (page >= p.pages) report(p.status, UB_ERR_ARG);
    }
    return c;
}

// FORK: a child row for each of `n` parents; else a page for every missing entry of `n` rows.
template <bool FORK>
__global__ void __launch_bounds__(POOL_THREADS) ub_pool_take_kernel(const __grid_constant__ PoolParams p)
{
    __shared__ int scratch[POOL_WARPS], told[TOLD];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const Span rows = share(p.n, rank), pool = share(p.pages, rank);

    // How many pages this CTA's rows want: a warp per row, or a thread per child.
    int wants = 0;
    if (FORK) {
        for (int64_t i = rows.lo + threadIdx.x; i < rows.hi; i += POOL_THREADS) wants += child_of(p, static_cast<int>(i)).part;
    } else {
        for (int64_t s = rows.lo + warp; s < rows.hi; s += POOL_WARPS) {
            const Entries e = take_range(p, static_cast<int>(s));
            for (int64_t j = e.first + lane; j < e.last; j += 32) wants += p.table[s * p.table_row + j] < 0 ? 1 : 0;
        }
    }
    wants = block_sum(wants, scratch);
    const int frees = count_pages(p.refs, pool, scratch, IsFree());
    if (threadIdx.x == 0) {
        told[0] = wants;
        told[1] = frees;
    }
    cluster.sync();
    const Sums want = over_ctas(cluster, told, 0), have = over_ctas(cluster, told, 1);
    // The free pages that will be needed, listed in order.
    const int64_t most = static_cast<int64_t>(want.all) - have.before;
    ranked_pages(p.refs, pool, most, scratch, IsFree(), [&](int64_t page, int r, int64_t k) {
        if (r <= 0 && k < most) p.list[have.before + k] = static_cast<int32_t>(page);
    });
    cluster.sync();

    int64_t next = want.before;              // rank of this CTA's next wish
    auto page_of = [&](int64_t k) {
        if (k < have.all) {
            const int32_t page = __ldcg(p.list + k);
            p.refs[page] = 1;
            return page;
        }
        report(p.status, UB_ERR_CAPACITY);
        return -1;
    };
    if constexpr (FORK) {
        for (int64_t i0 = rows.lo; i0 < rows.hi; i0 += POOL_WARPS) {
            const int64_t i = i0 + warp;
            const Child c = i < rows.hi ? child_of(p, static_cast<int>(i)) : Child{-1, 0, 0};
            int total;
            const int64_t k = next + warps_before(c.part, scratch, &total);
            next += total;
            if (i >= rows.hi) continue;
            const int32_t *from = p.table + (c.source < 0 ? 0 : c.source) * p.table_row;
            int32_t *to = p.new_table + i * p.new_row;
            int32_t copy = -1;
            if (c.part != 0) {
                if (lane == 0) copy = page_of(k);
                copy = __shfl_sync(0xffffffffu, copy, 0);
            }
            if (lane == 0) {
                p.pairs[2 * i] = copy >= 0 ? from[c.whole] : -1;
                p.pairs[2 * i + 1] = copy;
            }
            for (int64_t j = lane; j < p.width; j += 32) {
                int32_t page = c.source >= 0 && j < c.whole ? from[j] : -1;
                if (page >= p.pages) {
                    report(p.status, UB_ERR_ARG);
                    page = -1;
                }
                if (page >= 0 && atomicAdd(p.refs + page, 1) <= 0) report(p.status, UB_ERR_ARG);
                to[j] = c.part != 0 && j == c.whole ? copy : (page < 0 ? -1 : page);
            }
        }
    } else {
        for (int64_t s0 = rows.lo; s0 < rows.hi; s0 += POOL_WARPS) {
            const int64_t s = s0 + warp;
            const Entries e = s < rows.hi ? take_range(p, static_cast<int>(s)) : Entries{0, 0};
            int32_t *row = p.table + s * p.table_row;
            int mine = 0;
            for (int64_t j = e.first + lane; j < e.last; j += 32) mine += row[j] < 0 ? 1 : 0;
            mine = __reduce_add_sync(0xffffffffu, mine);
            int total;
            int64_t k = next + warps_before(mine, scratch, &total);
            next += total;
            for (int64_t j0 = e.first; j0 < e.last; j0 += 32) {
                const bool miss = j0 + lane < e.last && row[j0 + lane] < 0;
                const uint32_t hit = __ballot_sync(0xffffffffu, miss);
                if (miss) row[j0 + lane] = page_of(k + __popc(hit & ((1u << lane) - 1u)));
                k += __popc(hit);
            }
        }
    }
}

// ---------------------------------------------------------------- free

__global__ void __launch_bounds__(256) ub_pool_free_kernel(const __grid_constant__ PoolParams p)
{
    pdl_wait();
    pdl_trigger();
    // A CTA takes 256 entries of a row at a time.
    const int64_t per_row = (p.width + 255) / 256, units = p.n * per_row;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t s = u / per_row, j = (u - s * per_row) * 256 + threadIdx.x;
        const int64_t b = p.begin[s] < 0 ? 0 : p.begin[s], e = p.end[s];
        const int64_t at = j << p.page_shift;
        if (j >= p.width || at < b || at + (int64_t(1) << p.page_shift) > e) continue;
        const int32_t page = p.table[s * p.table_row + j];
        if (page < 0) continue;
        p.table[s * p.table_row + j] = -1;
        if (page >= p.pages) {
            report(p.status, UB_ERR_ARG);
        } else if (atomicSub(p.refs + page, 1) <= 0) {
            atomicAdd(p.refs + page, 1);    // nobody's page any more: its count stays
            report(p.status, UB_ERR_ARG);
        }
    }
}

// ---------------------------------------------------------------- compact

__global__ void __launch_bounds__(POOL_THREADS) ub_pool_compact_kernel(const __grid_constant__ PoolParams p)
{
    __shared__ int scratch[POOL_WARPS], told[TOLD];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    pdl_wait();
    pdl_trigger();
    const Span pool = share(p.pages, rank);
    const auto is_used = [](int r, int64_t) { return r > 0; };
    // The table's entries, the first AHEAD of each thread read now (rows * width stays within 32 bits).
    constexpr int AHEAD = 4;
    const uint32_t tid = rank * POOL_THREADS + threadIdx.x, stride = POOL_CTAS * POOL_THREADS;
    const uint32_t entries = static_cast<uint32_t>(p.rows) * static_cast<uint32_t>(p.width);
    auto at = [&](uint32_t e, int64_t pitch) {
        const uint32_t s = e / static_cast<uint32_t>(p.width);
        return s * pitch + (e - s * static_cast<uint32_t>(p.width));
    };
    int32_t ahead[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) ahead[i] = tid + i * stride < entries ? p.table[at(tid + i * stride, p.table_row)] : -1;
    const int used = count_pages(p.refs, pool, scratch, is_used);
    if (threadIdx.x == 0) told[0] = used;
    cluster.sync();
    const Sums in_use = over_ctas(cluster, told, 0);
    const int64_t U = in_use.all;
    // Pages in use below U stay where they are: those of the shares before the one that U lies in,
    // and those before U in that one, which every CTA counts for itself.
    const int64_t per = share(p.pages, 0).hi;
    const int edge = U < p.pages ? static_cast<int>(U / per) : POOL_CTAS;
    int64_t stay = count_pages(p.refs, Span{edge * per, U}, scratch, is_used);
    for (int c = 0; c < edge; ++c) stay += cluster.map_shared_rank(told, c)[0];
    const int64_t moves = U - stay;
    int32_t *holes = p.list, *movers = p.list + p.pages / 2, *place = p.list + p.pages;
    ranked_pages(p.refs, pool, INT64_MAX, scratch, is_used, [&](int64_t page, int r, int64_t k) {
        const int64_t used_before = in_use.before + k;
        if (r <= 0 && page < U) {
            holes[page - used_before] = static_cast<int32_t>(page);
        } else if (r > 0 && page >= U) {
            movers[used_before - stay] = static_cast<int32_t>(page);
        } else if (p.refs_out != p.refs) {
            p.refs_out[page] = r;
        }
        if (page >= U) place[page] = static_cast<int32_t>(page);
    });
    cluster.sync();
    for (int64_t k = tid; k < p.n; k += stride) {
        int32_t from = -1, to = -1;
        if (k < moves) {
            from = __ldcg(movers + k);
            to = __ldcg(holes + k);
            place[from] = to;
            p.refs_out[to] = p.refs[from];
            p.refs_out[from] = 0;
        }
        p.pairs[2 * k] = from;
        p.pairs[2 * k + 1] = to;
    }
    if (tid == 0) *p.used = static_cast<int32_t>(U);
    cluster.sync();
    auto renamed = [&](uint32_t e, int32_t page) {
        if (page >= p.pages) report(p.status, UB_ERR_ARG);
        if (page >= U && page < p.pages) page = __ldcg(place + page);
        p.new_table[at(e, p.new_row)] = page;
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (tid + i * stride < entries) renamed(tid + i * stride, ahead[i]);
    for (int64_t e = static_cast<int64_t>(tid) + AHEAD * stride; e < entries; e += stride)
        renamed(static_cast<uint32_t>(e), p.table[at(static_cast<uint32_t>(e), p.table_row)]);
}

// ---------------------------------------------------------------- data

template <int D>
__global__ void __launch_bounds__(COPY_THREADS) ub_kv_copy_kernel(const __grid_constant__ PageCopyParams p)
{
    pdl_wait();
    pdl_trigger();
    // The keys and values of a page as one run of 16-byte vectors: [k, v][head][row][D / 8].
    constexpr int VSHIFT = D == 128 ? 4 : 3;
    constexpr int CHUNK = COPY_THREADS * COPY_VECS;
    const int row_mask = (1 << p.page_shift) - 1;
    const int half = p.kv_heads << (p.page_shift + VSHIFT);
    const int chunks = (2 * half + CHUNK - 1) / CHUNK;
    for (int64_t u = blockIdx.x; u < p.n * chunks; u += gridDim.x) {
        const int64_t part = u / p.n, pair = u - part * p.n;
        const int v0 = static_cast<int>(part) * CHUNK + threadIdx.x;
        const int32_t from = p.pairs[2 * pair], to = p.pairs[2 * pair + 1];
        if (from < 0 && to < 0) continue;
        if (from < 0 || to < 0 || from >= p.pages || to >= p.pages) {
            if (threadIdx.x == 0) report(p.status, UB_ERR_ARG);
            continue;
        }
        uint4 x[COPY_VECS];
        int64_t at[COPY_VECS];
#pragma unroll
        for (int i = 0; i < COPY_VECS; ++i) {
            const int v = v0 + i * COPY_THREADS;
            if (v >= 2 * half) continue;
            const bool is_v = v >= half;
            const int w = is_v ? v - half : v;
            const int64_t row = (w >> VSHIFT) & row_mask, head = w >> (VSHIFT + p.page_shift);
            const int64_t in = row * (is_v ? p.vc_row : p.kc_row) + head * (is_v ? p.vc_head : p.kc_head) + (w & (D / 8 - 1)) * 8;
            const int64_t page = is_v ? p.vc_page : p.kc_page;
            const __nv_bfloat16 *base = static_cast<const __nv_bfloat16 *>(is_v ? p.v_cache : p.k_cache);
            x[i] = __ldcg(reinterpret_cast<const uint4 *>(base + from * page + in));
            at[i] = to * page + in;
        }
#pragma unroll
        for (int i = 0; i < COPY_VECS; ++i) {
            const int v = v0 + i * COPY_THREADS;
            if (v >= 2 * half) continue;
            __nv_bfloat16 *base = static_cast<__nv_bfloat16 *>(v >= half ? p.v_cache : p.k_cache);
            *reinterpret_cast<uint4 *>(base + at[i]) = x[i];
        }
    }
}

// Bound by latency: 64 registers leave room for 8 CTAs on an SM, so that 256 sequences of 8 heads of 128
// (2048 CTAs) come in two rounds; a thread looks up two page ids for every row before it loads it,
// and the loads of some rows follow the stores of the last ones (14.5 us for 52 MB; the path, which one
// lane walks in shared memory, has at most 34 drafts there).
//
// A CTA moves 128 of a sequence's 16-byte columns ([k, v][head][D / 8]), the rows of the path in
// rising order. Draft a_d of the path goes to place d <= a_d: a thread loads some rows of its
// column and then stores them, and never overwrites a row that it has yet to load, because the
// places still to be loaded are all above those stored.
template <int D>
__global__ void __launch_bounds__(ACCEPT_THREADS) ub_kv_accept_kernel(const __grid_constant__ AcceptParams p)
{
    __shared__ int16_t parent[UB_ACCEPT_MOST], path[UB_ACCEPT_MOST];
    __shared__ uint8_t on[UB_ACCEPT_MOST];
    __shared__ int sm_len;
    pdl_wait();
    pdl_trigger();
    const int s = static_cast<int>(blockIdx.x / p.parts), part = static_cast<int>(blockIdx.x - s * p.parts);
    const int tid = threadIdx.x;
    const int a = p.b.seq_starts[s], z = p.b.seq_starts[s + 1], leaf = p.leaves[s];
    const bool ordered = a >= 0 && z >= a && z <= p.tokens;
    const int n = ordered ? z - a : 0;
    const int64_t most = static_cast<int64_t>(p.b.table_width) << p.b.page_shift;
    const int64_t len = p.b.kv_lens[s], text = len - n;
    const bool bad = !ordered || leaf < -1 || leaf >= n || n > UB_ACCEPT_MOST || text < 0 || len > most;
    if (bad && tid == 0) report(p.b.status, UB_ERR_ARG);
    if (tid == 0) sm_len = 0;
    const bool some = !bad && leaf >= 0;
    for (int i = tid; some && i <= leaf; i += ACCEPT_THREADS) {
        const int q = p.parents[a + i];
        const bool wrong = q < -1 || q >= i;
        if (wrong) report(p.b.status, UB_ERR_ARG);
        parent[i] = static_cast<int16_t>(wrong ? -1 : q);
        on[i] = 0;
    }
    __syncthreads();
    if (some && tid == 0)
        for (int i = leaf; i >= 0; i = parent[i]) on[i] = 1;
    __syncthreads();
    if (some && tid < 32) {
        int m = 0;
        for (int i0 = 0; i0 <= leaf; i0 += 32) {
            const bool mine = i0 + tid <= leaf && on[i0 + tid] != 0;
            const uint32_t hit = __ballot_sync(0xffffffffu, mine);
            if (mine) path[m + __popc(hit & ((1u << tid) - 1u))] = static_cast<int16_t>(i0 + tid);
            m += __popc(hit);
        }
        if (tid == 0) sm_len = m;
    }
    __syncthreads();
    const int m = sm_len;
    if (part == 0 && tid == 0) p.new_lens[s] = static_cast<int32_t>(text < 0 ? 0 : (text > most ? most : text) + m);
    if (m == 0) return;

    const int col = part * ACCEPT_THREADS + tid;
    if (col >= p.caches * p.kv_heads * (D / 8)) return;
    const bool is_v = col >= p.kv_heads * (D / 8);
    const int c = is_v ? col - p.kv_heads * (D / 8) : col;
    const int64_t page_stride = is_v ? p.vc_page : p.kc_page, row_stride = is_v ? p.vc_row : p.kc_row;
    __nv_bfloat16 *base = static_cast<__nv_bfloat16 *>(is_v ? p.v_cache : p.k_cache) + (c / (D / 8)) * (is_v ? p.vc_head : p.kc_head) +
                          (c & (D / 8 - 1)) * 8;
    const int32_t *table = p.b.page_table + s * p.b.table_row;
    auto at = [&](int64_t slot) -> int64_t {
        const int32_t page = table[slot >> p.b.page_shift];
        if (page < 0 || page >= p.b.num_pages) {
            report(p.b.status, UB_ERR_ARG);
            return -1;
        }
        return page * page_stride + (slot & ((int64_t(1) << p.b.page_shift) - 1)) * row_stride;
    };
    for (int d0 = 0; d0 < m; d0 += ACCEPT_ROWS) {
        uint4 x[ACCEPT_ROWS];
        int64_t to[ACCEPT_ROWS];
#pragma unroll
        for (int i = 0; i < ACCEPT_ROWS; ++i) {
            to[i] = -1;
            if (d0 + i >= m || path[d0 + i] == d0 + i) continue;
            const int64_t from = at(text + path[d0 + i]);
            to[i] = at(text + d0 + i);
            if (from < 0) to[i] = -1;
            if (to[i] >= 0) x[i] = *reinterpret_cast<const uint4 *>(base + from);
        }
#pragma unroll
        for (int i = 0; i < ACCEPT_ROWS; ++i)
            if (to[i] >= 0) *reinterpret_cast<uint4 *>(base + to[i]) = x[i];
    }
}

}  // namespace

cudaError_t launch_pool(PoolOp op, const PoolParams &p, int sms, cudaStream_t s)
{
    const bool pdl = p.pdl != 0;
    switch (op) {
    case PoolOp::take: return launch_ex(ub_pool_take_kernel<false>, p, POOL_CTAS, POOL_THREADS, 0, POOL_CTAS, pdl, s);
    case PoolOp::fork: return launch_ex(ub_pool_take_kernel<true>, p, POOL_CTAS, POOL_THREADS, 0, POOL_CTAS, pdl, s);
    case PoolOp::compact: return launch_ex(ub_pool_compact_kernel, p, POOL_CTAS, POOL_THREADS, 0, POOL_CTAS, pdl, s);
    default: break;
    }
    const int64_t units = p.n * ((p.width + 255) / 256);
    const int64_t grid = units < 8 * sms ? units : 8 * sms;
    return launch_ex(ub_pool_free_kernel, p, static_cast<int>(grid), 256, 0, 1, pdl, s);
}

cudaError_t launch_kv_copy(const PageCopyParams &p, cudaStream_t s)
{
    const int64_t vecs = (2 * static_cast<int64_t>(p.kv_heads) * p.head_dim / 8) << p.page_shift;
    const int64_t units = p.n * ((vecs + COPY_THREADS * COPY_VECS - 1) / (COPY_THREADS * COPY_VECS));
    const int64_t grid = units < COPY_GRID ? units : COPY_GRID;
    return launch_ex(p.head_dim == 128 ? ub_kv_copy_kernel<128> : ub_kv_copy_kernel<64>, p, static_cast<int>(grid),
                     COPY_THREADS, 0, 1, p.pdl != 0, s);
}

cudaError_t launch_kv_accept(AcceptParams p, cudaStream_t s)
{
    p.parts = (p.caches * p.kv_heads * p.head_dim / 8 + ACCEPT_THREADS - 1) / ACCEPT_THREADS;
    return launch_ex(p.head_dim == 128 ? ub_kv_accept_kernel<128> : ub_kv_accept_kernel<64>, p, p.b.n_seqs * p.parts,
                     ACCEPT_THREADS, 0, 1, p.pdl != 0, s);
}

}  // namespace ubk
