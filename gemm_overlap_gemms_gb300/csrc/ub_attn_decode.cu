// Attention of one new token per sequence over a paged key/value cache (decoding).
//
//   O[h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q[h] . k_j - m),   j < kv_len
//
// for every query head h of the token, k and v of key/value head h / group. m is the
// running maximum: the keys are read once, the partial (m, sum p, sum p v) of a set of
// keys being rescaled by exp(m_old - m_new) when a larger score appears, and two partials
// joined in the same way.
//
// Bound by HBM: the cache is read once for `group` query heads, 4 * group flops per 4
// bytes. The tensor cores are needed for their multiply rate at a group of 4 and more
// (fp32 units would do 27e12 multiply-adds/s of work at group 8 and 6.7 TB/s), not for
// throughput; mma.sync.m16n8k16 on 16 keys by 8 heads matches the shape (a tcgen05 tile
// would want 64 or 128 rows of heads, or the softmax across TMEM lanes), with keys as the
// MMA's rows in the first product, S^T = K q^T, and the head dimension as its rows in the
// second, O^T = V^T P^T, so that up to 8 heads of a group cost one column tile.
//
// Work split: the (sequence, head, 32-key tile) triples of the whole call are laid end to
// end and every CTA takes an equal, contiguous range, found on the device from kv_lens. So
// ragged lengths, one long sequence and many short ones all load every SM alike, without
// the host knowing a length. The end of an item (its warps' partials joined and written, the
// next queries loaded) counts as 12 tiles, which also keeps many items whole: 64 sequences of
// 100 to 600 keys, 8 key/value heads 22.8 us, counted as 4 tiles 23.9, as none 28.9; 128
// sequences of 20 to 400 keys, 4 heads 18.4, 19.5 and 30.9 us (6 to 16 tiles: within 3 %).
// The parts of an item that spans CTAs go to the workspace and are joined in CTA order
// (deterministic) once a counter per item says that all are there: up to JOIN_MOST parts by
// the CTA that comes last, more by all their CTAs, a share of the outputs each, so that no
// CTA reads all of a long sequence's parts.
//
// A CTA is four loading and four computing warps, one CTA on an SM. The loading warps fill a
// ring of 128 KB (a stage is one tile's keys and values) with TMA boxes of one page or one
// tile, whichever is smaller, every fourth tile each: a tile of four boxes takes a loading
// warp about 1000 cycles (measured), more than the 700 in which an SM's share of HBM delivers
// it. Each computing warp takes every fourth tile by itself with its own running maximum, so
// that no barrier separates tiles (860 cycles a tile); the four partials are joined in shared
// memory at the end of an item, while the ring goes on filling.
//
// Measured (GB300): 128 sequences, 583272 keys, 32 query heads, 8 key/value heads of 128 (2.39
// GB): 345 us, 6.9 TB/s, HBM-bound (a ring of 192 KB: 3 % slower, SMs drift further apart; 64
// KB: 18 % slower). One sequence of 131071 keys, one key/value head (67 MB): 18.7 us, of which
// 10 us stream; 3-4 us pass before the first tile lands, 5 us after the last (parts written,
// counted, joined). 64 sequences, 127938 keys, 2 key/value heads (131 MB): 29 us, 18 of them
// streaming. 15 sequences of 2900 keys, one key/value head, 8 query heads (22 MB, 10 parts
// each): 10.4 us. Four sequences of 300 keys, 8 heads: 7.4-9.4 us a call, bound by the host's side.
#include <cuda_bf16.h>

#include "ub_attn.h"
#include "ub_device.cuh"
#include "ub_internal.h"

namespace ubk {
namespace {

constexpr int KT = DECODE_KEYS;
constexpr int WARPS = 4;
constexpr int DEC_THREADS = 32 * 2 * WARPS;
// Parts that one CTA joins (30 sequences of 2750 keys, 5 parts each: 12.1 us, joined by all
// their CTAs 15.0; 15 sequences, 10 parts each: 10.4, joined by one 11.2), and how many it has
// in flight.
constexpr int JOIN_MOST = 8, JOIN_STEP = 4;
constexpr int MIN_TILES = 4;             // of a CTA, on average (one sequence of 2000 keys: 7.8 us; 16: 10.9 us)
// Tiles that a join costs: items of equal length, whole and split, 32 items of 16 tiles 7.0 and
// 7.8 us, of 22 8.2 and 8.1, of 31 9.8 and 9.1; 8 items of 22 8.3 and 8.5, of 31 9.9 and 8.7; 64
// items of 31 10.0 and 10.5; 128 of 31 10.2 and 13.6.
constexpr int JOIN_TILES = 19;

template <int D, int NT>
struct DecShape {
    static constexpr int TILE_BYTES = KT * D * 2;
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int HEADS = 8 * NT;
    static constexpr int O_ROW = D + 4;                           // padded: conflict-free writes
    static constexpr int MERGE_BYTES = WARPS * HEADS * O_ROW * 4;
    // A multiple of WARPS, so that a stage always belongs to the same warp: the loads of two
    // tiles may land in either order, and a warp that waited for the second fill of a stage
    // whose first fill (another warp's) has not landed would see the parity it waits for.
    static constexpr int STAGES = 131072 / STAGE_BYTES;
    static constexpr int SMEM = STAGES * STAGE_BYTES + MERGE_BYTES + 960;
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(STAGES >= WARPS && STAGES % WARPS == 0, "one warp per stage");
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t *r)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t *r)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma_16x8x16(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One box: rows of one page, all of the head dimension (64 columns after 64 columns).
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int row, int head, int page)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %3, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(row), "r"(head), "r"(page)
        : "memory");
}

// Counts one arrival; everything this CTA wrote before the barrier in front of it is visible
// to whoever sees the count, and what the others wrote before theirs to this thread.
__device__ __forceinline__ uint32_t arrive_acq_rel(uint32_t *counter)
{
    uint32_t old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
    return old;
}

__device__ __forceinline__ void bar_compute() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ int clamped_len(const SeqBatch &b, int seq)
{
    const int len = b.kv_lens[seq];
    const int64_t most = static_cast<int64_t>(b.table_width) << b.page_shift;
    return len < 0 ? 0 : (len > most ? static_cast<int>(most) : len);
}
__device__ __forceinline__ int tiles_of(int len) { return len > 0 ? (len + KT - 1) / KT : 1; }

// What an item counts in the split: its tiles and its end, which costs a CTA about as long as
// DECODE_ITEM_COST tiles.
__device__ __forceinline__ int cost_of(int len) { return tiles_of(len) + DECODE_ITEM_COST; }

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The equal split of `total` units (tiles and ends of items) over `ctas`: CTA c's first unit,
// and the CTA of a unit.
struct Split {
    int64_t base, rem;
    __device__ __forceinline__ int64_t first(int64_t c) const { return c * base + (c < rem ? c : rem); }
    __device__ __forceinline__ int owner(int64_t x) const
    {
        const int64_t cut = rem * (base + 1);
        return static_cast<int>(x < cut ? quotient(x, base + 1) : rem + quotient(x - cut, base));
    }
};

__device__ __forceinline__ int64_t warp_sum(int64_t v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// Sum and maximum of the sequences' costs (one warp). I: a type that holds the sum over all heads.
template <typename I>
__device__ __forceinline__ I total_cost(const SeqBatch &b, int lane, int own, int *most)
{
    I sum = own;
    int top = own;
    for (int i = lane + 32; i < b.n_seqs; i += 32) {
        const int n = cost_of(clamped_len(b, i));
        sum += n;
        top = n > top ? n : top;
    }
    *most = __reduce_max_sync(0xffffffffu, top);
    return warp_sum(sum);
}
// The sequence that holds unit `unit` of the call, and the units before it. own: the cost of
// sequence `lane` (0 past the last).
template <typename I>
__device__ __forceinline__ void find_seq(const SeqBatch &b, int lane, int own, I unit, int heads, int *seq, I *before)
{
    I seen = 0;  // units of the sequences before this batch of 32, over all heads
    for (int i0 = 0; i0 < b.n_seqs; i0 += 32) {
        I mine = i0 == 0 ? own : (i0 + lane < b.n_seqs ? cost_of(clamped_len(b, i0 + lane)) : 0);
        mine *= heads;
        I upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const I x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, seen + upto > unit);
        if (past != 0u) {
            const int l = __ffs(static_cast<int>(past)) - 1;
            *seq = i0 + l;
            *before = seen + __shfl_sync(0xffffffffu, upto - mine, l);
            return;
        }
        seen += __shfl_sync(0xffffffffu, upto, 31);
    }
    *seq = b.n_seqs;
    *before = seen;
}

// What a CTA does: its first item and tile, and how many units it takes (none: nothing).
struct Share {
    Split split;
    int64_t x, left;  // first unit of the whole call (not counted for whole items), units
    int seq, head, t0;
};
template <typename I>
__device__ __forceinline__ Share share_of(const SeqBatch &b, int lane, int heads, int cta, int grid)
{
    Share s{{0, 0}, 0, 0, 0, 0, 0};
    const int own = lane < b.n_seqs ? cost_of(clamped_len(b, lane)) : 0;
    int most;
    const I total = total_cost<I>(b, lane, own, &most) * heads;
    // A CTA per item where no item is much longer than an equal share would be: a share saves
    // the difference and costs a join. Else equal shares, of at least MIN_TILES units, or one
    // CTA per item where those are shorter (355 items of one tile: 8.7 us; on 44 CTAs 18.4).
    const int64_t n_items = static_cast<int64_t>(b.n_seqs) * heads;
    const bool whole_items = n_items <= grid && static_cast<int64_t>(most - DECODE_ITEM_COST - JOIN_TILES) * grid <=
                                                    total - n_items * DECODE_ITEM_COST;
    I ctas = whole_items ? static_cast<I>(n_items) : total / MIN_TILES;
    if (!whole_items && ctas < n_items) ctas = n_items < total ? static_cast<I>(n_items) : total;
    ctas = ctas < 1 ? 1 : (ctas > grid ? grid : ctas);
    if (cta >= ctas) return s;
    const I base = static_cast<I>(quotient(total, ctas));
    s.split = Split{base, total - base * ctas};
    if (whole_items) {
        s.seq = cta / heads;
        s.head = cta - s.seq * heads;
        s.left = tiles_of(clamped_len(b, s.seq));
        return s;
    }
    const I x = static_cast<I>(s.split.first(cta));
    I before;
    find_seq<I>(b, lane, own, x, heads, &s.seq, &before);
    const int cost = cost_of(clamped_len(b, s.seq)), tiles = cost - DECODE_ITEM_COST;
    s.x = x;
    s.left = s.split.first(cta + 1) - x;
    s.head = static_cast<int>(quotient(x - before, cost));
    s.t0 = static_cast<int>(x - before - static_cast<I>(s.head) * cost);
    if (s.t0 >= tiles) {  // behind the item's last tile: on to the next
        s.x += cost - s.t0;
        s.left -= cost - s.t0;
        s.t0 = 0;
        if (++s.head == heads) {
            s.head = 0;
            ++s.seq;
        }
    }
    return s;
}

template <int D, int NT>
__global__ void __launch_bounds__(DEC_THREADS, DECODE_CTAS_PER_SM)
    ub_attn_decode_kernel(const __grid_constant__ DecodeParams p)
{
    using Sh = DecShape<D, NT>;
    constexpr int S = Sh::STAGES;
    extern __shared__ __align__(1024) uint8_t base[];
    float *sm_o = reinterpret_cast<float *>(base + S * Sh::STAGE_BYTES);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + S * Sh::STAGE_BYTES + Sh::MERGE_BYTES);
    float *sm_m = reinterpret_cast<float *>(bars + 2 * S);                     // [WARPS][HEADS]
    float *sm_l = sm_m + WARPS * DECODE_HEADS;                                 // [WARPS][HEADS]
    int *sm_last = reinterpret_cast<int *>(sm_l + WARPS * DECODE_HEADS);
    static_assert(2 * S * 8 + 2 * WARPS * DECODE_HEADS * 4 + 8 <= 960, "barrier area");
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + S);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((smem_u32(base) & 1023u) != 0u) {  // the swizzled tiles need what the declaration asks for
        if (threadIdx.x == 0) atomicCAS(p.status_word(), 0, UB_ERR_ALIGN);
        return;
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        fence_mbar_init();
        prefetch_tmap(&p.tmK);
        prefetch_tmap(&p.tmV);
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    const SeqBatch &b = p.b;
    const int heads = p.kv_heads * p.head_blocks;  // items per sequence
    const Share sh = p.many_tiles ? share_of<int64_t>(b, lane, heads, blockIdx.x, gridDim.x)
                                  : share_of<int>(b, lane, heads, blockIdx.x, gridDim.x);
    if (sh.left <= 0) return;
    const Split split = sh.split;
    int seq = sh.seq, head = sh.head, t0 = sh.t0;
    int64_t x = sh.x, left = sh.left;
    const WaitCtx wc{p.abort_word, p.status_word(), p.timeout_ns, p.epoch};
    bool alive = true;
    uint32_t count = 0;  // tiles of this CTA so far: stage count % S, phase count / S
    const int tid = threadIdx.x, G = gridDim.x;
    const float sl = p.scale * 1.4426950408889634f;
    constexpr int SLOT = decode_slot_floats(D);
    auto slot_of = [&](int cta, int which) { return p.ws + (static_cast<int64_t>(which) * G + cta) * SLOT; };
    // Four outputs of head h0 + hh of sequence s, from the weighted sum and the sum of weights.
    auto finish = [&](int s, int h0, int hh, int d, float4 acc, float M, float L) {
        const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
        uint2 w;
        w.x = pack_bf16x2(__float_as_uint(acc.x * inv), __float_as_uint(acc.y * inv));
        w.y = pack_bf16x2(__float_as_uint(acc.z * inv), __float_as_uint(acc.w * inv));
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + s * p.o_row + (h0 + hh) * p.o_head + d) = w;
        if (p.lse && d == 0) p.lse[static_cast<int64_t>(s) * p.heads + h0 + hh] = M * p.scale + logf(L);
    };
    struct Pending {     // an item that other CTAs have parts of
        int64_t item0;
        int tiles, seq, h0, g;
    };
    Pending pend[2] = {{0, 0, 0, 0, 0}, {0, 0, 0, 0, 0}};  // begun before this CTA; going on after it

    uint32_t upto = 0;   // ... when the current item is done
    // A tile in shared memory: box after box, in a box 64 columns after 64 columns, there row
    // after row of 128 bytes.
    const int box = KT < (1 << b.page_shift) ? KT : (1 << b.page_shift);  // rows per box
    const int box_shift = __ffs(box) - 1;
    auto row_at = [&](int r) { return (((r >> box_shift) * (D / 64)) << box_shift) * 128 + (r & (box - 1)) * 128; };
    const int half_at = box * 128;
    int k_row[2], v_row[2];  // this lane's rows of the two fragments of 16 keys
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
        k_row[mt] = row_at(mt * 16 + (lane & 15));
        v_row[mt] = row_at(mt * 16 + (lane & 7) + ((lane >> 4) << 3));
    }
    while (left > 0 && seq < b.n_seqs) {
        const int len = clamped_len(b, seq);
        const int tiles = tiles_of(len);
        const int64_t item0 = x - t0;
        const int t1 = tiles - t0 < left ? tiles : t0 + static_cast<int>(left);
        const int64_t units = tiles + DECODE_ITEM_COST - t0 < left ? tiles + DECODE_ITEM_COST - t0 : left;
        upto += t1 - t0;
        const int kvh = head / p.head_blocks, hb = head - kvh * p.head_blocks;
        const int h0 = kvh * p.group + hb * DECODE_HEADS;     // first query head
        const int g = p.group - hb * DECODE_HEADS < DECODE_HEADS ? p.group - hb * DECODE_HEADS : DECODE_HEADS;

        if (warp >= WARPS) {
            // ---------------------------------------------------------------- loads
            const int boxes = KT / box;
            const int32_t *table = b.page_table + seq * b.table_row;
            const int pages = (len + (1 << b.page_shift) - 1) >> b.page_shift;
            int cached0 = 0, cached_n = 0;   // page ids [cached0, cached0 + cached_n), one per lane
            int ids = -1;
            for (int t = t0; t < t1 && alive; ++t, ++count) {
                if ((count & (WARPS - 1)) != static_cast<uint32_t>(warp - WARPS)) continue;
                const int stage = count % S;
                if (count >= S) alive = mbar_wait(empty0 + 8 * stage, ((count / S) - 1) & 1, wc);
                alive = __all_sync(0xffffffffu, alive);
                if (!alive) break;
                const int key0 = t * KT;
                const int page0 = key0 >> b.page_shift;
                const int valid = len - key0;
                const int n_box = valid <= 0 ? 0 : ((valid < KT ? valid : KT) + box - 1) / box;
                if (page0 + boxes > cached0 + cached_n) {
                    cached0 = page0;
                    cached_n = 32;
                    ids = cached0 + lane < pages ? table[cached0 + lane] : -1;
                    if (cached0 + lane < pages && (ids < 0 || ids >= b.num_pages)) {
                        atomicCAS(p.status_word(), 0, UB_ERR_ARG);
                        ids = -1;  // outside the tensor: the box is filled with zeros
                    }
                }
                const uint32_t bar = full0 + 8 * stage;
                int page[KT / 8];
#pragma unroll
                for (int bx = 0; bx < KT / 8; ++bx) page[bx] = __shfl_sync(0xffffffffu, ids, (page0 - cached0 + bx) & 31);
                const int row = boxes > 1 ? 0 : key0 & ((1 << b.page_shift) - 1);
                if (lane == 0) {
                    const uint32_t dst = smem_u32(base) + stage * Sh::STAGE_BYTES;
                    const int bytes = box * D * 2;
                    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(2 * n_box * bytes));
#pragma unroll
                    for (int bx = 0; bx < KT / 8; ++bx) {
                        if (bx >= n_box) break;
                        tma_load_5d(dst + bx * bytes, &p.tmK, bar, row, kvh, page[bx]);
                        tma_load_5d(dst + Sh::TILE_BYTES + bx * bytes, &p.tmV, bar, row, kvh, page[bx]);
                    }
                }
                __syncwarp();
            }
        } else {
            // ---------------------------------------------------------------- compute
            uint32_t qf[NT][D / 16][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int hh = nt * 8 + lane / 4;
                const uint32_t *qp = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.q) +
                                                                        seq * p.q_row + (h0 + hh) * p.q_head) +
                                     (lane & 3);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    qf[nt][ks][0] = hh < g ? qp[ks * 8] : 0u;
                    qf[nt][ks][1] = hh < g ? qp[ks * 8 + 4] : 0u;
                }
            }
            float o[D / 16][NT][4];
            float m[NT][2], l[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m[nt][0] = m[nt][1] = -INFINITY;
                l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                for (int d = 0; d < D / 16; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[d][nt][i] = 0.f;
            }
            for (int t = t0; t < t1; ++t, ++count) {
                if ((count & (WARPS - 1)) != static_cast<uint32_t>(warp)) continue;
                const int stage = count % S;
                if (alive) alive = mbar_wait(full0 + 8 * stage, (count / S) & 1, wc);
                alive = __all_sync(0xffffffffu, alive);
                if (!alive) break;
                const uint32_t kb = smem_u32(base) + stage * Sh::STAGE_BYTES, vb = kb + Sh::TILE_BYTES;
                const int valid = len - t * KT;
                if (valid < KT) {
                    // Rows past the length hold another call's bytes, perhaps not even numbers:
                    // their weight is zero, so their values must be finite.
                    for (int i = lane; i < KT * D / 8; i += 32) {
                        const int half = i / (KT * 8), r = (i / 8) % KT;
                        if (r >= valid) st_shared_v4(vb + half * half_at + row_at(r) + (i % 8) * 16, 0u, 0u, 0u, 0u);
                    }
                    __syncwarp();
                }
                float s[2][NT][4];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[mt][nt][i] = 0.f;
                // The keys' fragments are loaded ahead of the products that use them, and the first
                // half of the values' ahead of the softmax.
                {
                    uint32_t a[2][D / 16][4];
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) {
                            const int c = (ks * 2 + (lane >> 4)) & 7;
                            ldsm_x4(kb + (ks / 4) * half_at + k_row[mt] + ((c ^ (lane & 7)) << 4), a[mt][ks]);
                        }
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_16x8x16(s[mt][nt], a[mt][ks], qf[nt][ks][0], qf[nt][ks][1]);
                }
                uint32_t va[D / 32][2][4];
                auto load_v = [&](int d0) {
#pragma unroll
                    for (int d = 0; d < D / 32; ++d)
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) {
                            const int c = ((d0 + d) * 2 + ((lane >> 3) & 1)) & 7;
                            ldsm_x4_trans(vb + ((d0 + d) / 4) * half_at + v_row[mt] + ((c ^ (lane & 7)) << 4), va[d][mt]);
                        }
                };
                load_v(0);
                uint32_t pf[2][NT][2];
                bool moved = false;
                float f[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = m[nt][c];
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float &v = s[mt][nt][r * 2 + c];
                                if (mt * 16 + r * 8 + lane / 4 >= valid) v = -INFINITY;
                                mx = fmaxf(mx, v);
                            }
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        const float ref = mx == -INFINITY ? 0.f : mx;  // no key yet: every weight is zero
                        f[nt][c] = ex2((m[nt][c] - ref) * sl);
                        moved |= m[nt][c] != mx;
                        m[nt][c] = mx;
                        float sum = 0.f;
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float &v = s[mt][nt][r * 2 + c];
                                v = ex2(fmaf(v, sl, -ref * sl));
                                sum += v;
                            }
                        l[nt][c] = l[nt][c] * f[nt][c] + sum;
                    }
                // Weights in BF16, the type of the values they multiply (their sum stays fp32):
                // up to 2^-8 of each weight, as large as the rounding of the output.
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            pf[mt][nt][r] = transpose8(pack_bf16x2(__float_as_uint(s[mt][nt][2 * r]),
                                                                   __float_as_uint(s[mt][nt][2 * r + 1])));
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[d][nt][i] *= f[nt][i & 1];
                }
#pragma unroll
                for (int d0 = 0; d0 < D / 16; d0 += D / 32) {
                    if (d0 > 0) load_v(d0);
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int d = 0; d < D / 32; ++d)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_16x8x16(o[d0 + d][nt], va[d][mt], pf[mt][nt][0], pf[mt][nt][1]);
                }
                if (valid < KT) fence_proxy_async_shared();  // the zeroed rows before the next load's writes
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * stage);
            }
            count = upto;

            // The four warps' partials, joined in shared memory.
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], off);
                    const int hh = nt * 8 + (lane & 3) * 2 + c;
                    if (lane < 4) {
                        sm_m[warp * DECODE_HEADS + hh] = m[nt][c];
                        sm_l[warp * DECODE_HEADS + hh] = l[nt][c];
                    }
                }
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int hh = nt * 8 + (lane & 3) * 2 + (i & 1);
                        sm_o[(warp * Sh::HEADS + hh) * Sh::O_ROW + d * 16 + lane / 4 + (i >> 1) * 8] = o[d][nt][i];
                    }
            bar_compute();
            const bool whole = t0 == 0 && t1 == tiles;
            float *mine = slot_of(blockIdx.x, t0 == 0 ? 1 : 0);
            for (int u = tid; u < g * (D / 4); u += 32 * WARPS) {
                const int hh = u / (D / 4), d = (u - hh * (D / 4)) * 4;
                float M = sm_m[hh];
#pragma unroll
                for (int w = 1; w < WARPS; ++w) M = fmaxf(M, sm_m[w * DECODE_HEADS + hh]);
                const float ref = M == -INFINITY ? 0.f : M;
                float L = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float fw = ex2((sm_m[w * DECODE_HEADS + hh] - ref) * sl);
                    L += sm_l[w * DECODE_HEADS + hh] * fw;
                    const float4 v = *reinterpret_cast<const float4 *>(sm_o + (w * Sh::HEADS + hh) * Sh::O_ROW + d);
                    acc.x += v.x * fw;
                    acc.y += v.y * fw;
                    acc.z += v.z * fw;
                    acc.w += v.w * fw;
                }
                if (whole) {
                    finish(seq, h0, hh, d, acc, M, L);
                } else {
                    *reinterpret_cast<float4 *>(mine + hh * D + d) = acc;
                    if (d == 0) {
                        mine[DECODE_HEADS * D + hh] = M;
                        mine[DECODE_HEADS * (D + 1) + hh] = L;
                    }
                }
            }
            if (!whole && t0 != 0) pend[0] = Pending{item0, tiles, seq, h0, g};
            if (!whole && t0 == 0) pend[1] = Pending{item0, tiles, seq, h0, g};
            bar_compute();  // the shared partials are free again
        }
        if (!__all_sync(0xffffffffu, alive)) alive = false;
        x += units;
        left -= units;
        t0 = 0;
        if (++head == heads) {
            head = 0;
            ++seq;
        }
    }
    // The parts of split items, joined when the CTA's own tiles are done. Up to JOIN_MOST parts:
    // the last CTA to arrive joins them. More (all their CTAs are resident: one per SM, no more
    // than SMs): each waits for the others and joins its share of the outputs. A CTA arrives for
    // both its items before it waits for either, or the items would wait for one another in a row.
    if (warp < WARPS && (pend[0].tiles | pend[1].tiles) != 0) {
        uint32_t before[2] = {0u, 0u};  // how many times such an item has been complete: a count
                                        // that is never reset, and changes only after this CTA has arrived
#pragma unroll
        for (int which = 0; which < 2; ++which)
            if (pend[which].tiles != 0)
                before[which] = *static_cast<volatile uint32_t *>(p.times + split.owner(pend[which].item0));
        bar_compute();                  // this CTA's parts are written
        if (warp < 2 && lane == 0) {    // a warp for each
            const Pending it = warp == 0 ? pend[0] : pend[1];
            if (it.tiles != 0) {
                const int a = split.owner(it.item0), parts = split.owner(it.item0 + it.tiles - 1) - a + 1;
                const bool last = static_cast<int>(arrive_acq_rel(p.counters + a)) == parts - 1;
                if (last) {
                    p.counters[a] = 0u;  // zero again for the next call
                    if (parts > JOIN_MOST) st_release_u32(p.times + a, (warp == 0 ? before[0] : before[1]) + 1u);
                }
                sm_last[warp] = last ? 1 : 0;
            }
        }
        bar_compute();
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const Pending it = pend[which];
            if (it.tiles == 0) continue;
            const bool last = sm_last[which] != 0;
            const int a = split.owner(it.item0), z = split.owner(it.item0 + it.tiles - 1);
            const int parts = z - a + 1;
            const uint32_t *times = p.times + a;
            // part i's slot: 1 for the CTA in which the item begins, 0 for the others
            auto part = [&](int i) { return slot_of(a + i, i == 0 ? 1 : 0); };
            const int units = it.g * (D / 4);  // of four outputs
            if (parts <= JOIN_MOST) {
                if (!last) continue;
                for (int u = tid; u < units; u += 32 * WARPS) {
                    const int hh = u / (D / 4), d = (u - hh * (D / 4)) * 4;
                    float M = -INFINITY, L = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int i0 = 0; i0 < parts; i0 += JOIN_STEP) {
                        float4 v[JOIN_STEP];
                        float m[JOIN_STEP], l[JOIN_STEP], top = M;
#pragma unroll
                        for (int k = 0; k < JOIN_STEP; ++k) {
                            m[k] = -INFINITY;
                            l[k] = 0.f;
                            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (i0 + k >= parts) continue;
                            v[k] = __ldcg(reinterpret_cast<const float4 *>(part(i0 + k) + hh * D + d));
                            m[k] = __ldcg(part(i0 + k) + DECODE_HEADS * D + hh);
                            l[k] = __ldcg(part(i0 + k) + DECODE_HEADS * (D + 1) + hh);
                        }
#pragma unroll
                        for (int k = 0; k < JOIN_STEP; ++k) top = fmaxf(top, m[k]);
                        const float ref = top == -INFINITY ? 0.f : top;
                        const float f0 = ex2((M - ref) * sl);
                        L *= f0;
                        acc.x *= f0;
                        acc.y *= f0;
                        acc.z *= f0;
                        acc.w *= f0;
                        M = top;
#pragma unroll
                        for (int k = 0; k < JOIN_STEP; ++k) {
                            const float fw = ex2((m[k] - ref) * sl);
                            L += l[k] * fw;
                            acc.x += v[k].x * fw;
                            acc.y += v[k].y * fw;
                            acc.z += v[k].z * fw;
                            acc.w += v[k].w * fw;
                        }
                    }
                    finish(it.seq, it.h0, hh, d, acc, M, L);
                }
                continue;
            }
            if (!last) {
                WaitClock clk;
                for (uint32_t n = 1; alive; ++n) {
                    uint32_t v;
                    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(times) : "memory");
                    if (v != before[which]) break;
                    if ((n & 15u) == 0 && !clk.ok(wc)) alive = false;
                }
                alive = __all_sync(0xffffffffu, alive);
            }
            // Units of this CTA: `width` lanes each, as few as have all parts in flight at once.
            constexpr int U = 5;               // parts in flight per lane
            const int width_shift = parts <= 4 * U ? 2 : (parts <= 8 * U ? 3 : (parts <= 16 * U ? 4 : 5));
            const int width = 1 << width_shift, at_once = (32 * WARPS) >> width_shift;
            const int per = (units + parts - 1) / parts, i_cta = static_cast<int>(blockIdx.x) - a;
            const int end = (i_cta + 1) * per < units ? (i_cta + 1) * per : units;
            for (int u0 = i_cta * per; u0 < end && alive; u0 += at_once) {
                const int u = u0 + (tid >> width_shift);
                const int hh = u / (D / 4), d = (u - hh * (D / 4)) * 4;
                float M = -INFINITY, L = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int i0 = lane & (width - 1); i0 < parts && u < end; i0 += width * U) {
                    float4 v[U];
                    float m[U], l[U], top = M;
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        const int i = i0 + width * k;
                        m[k] = -INFINITY;
                        l[k] = 0.f;
                        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (i >= parts) continue;
                        v[k] = __ldcg(reinterpret_cast<const float4 *>(part(i) + hh * D + d));
                        m[k] = __ldcg(part(i) + DECODE_HEADS * D + hh);
                        l[k] = __ldcg(part(i) + DECODE_HEADS * (D + 1) + hh);
                    }
#pragma unroll
                    for (int k = 0; k < U; ++k) top = fmaxf(top, m[k]);
                    const float ref = top == -INFINITY ? 0.f : top;
                    const float f0 = ex2((M - ref) * sl);
                    L *= f0;
                    acc.x *= f0;
                    acc.y *= f0;
                    acc.z *= f0;
                    acc.w *= f0;
                    M = top;
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        const float fw = ex2((m[k] - ref) * sl);
                        L += l[k] * fw;
                        acc.x += v[k].x * fw;
                        acc.y += v[k].y * fw;
                        acc.z += v[k].z * fw;
                        acc.w += v[k].w * fw;
                    }
                }
                float top = M;
                for (int o = width >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float fw = ex2((M - (top == -INFINITY ? 0.f : top)) * sl);
                L *= fw;
                acc.x *= fw;
                acc.y *= fw;
                acc.z *= fw;
                acc.w *= fw;
                for (int o = width >> 1; o > 0; o >>= 1) {
                    L += __shfl_xor_sync(0xffffffffu, L, o);
                    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
                    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
                    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
                    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
                }
                if ((lane & (width - 1)) == 0 && u < end) finish(it.seq, it.h0, hh, d, acc, top, L);
            }
        }
    }
    // A wait ran out: the copies already issued land before the CTA gives its memory back.
    if (!alive) settle(200000);
}

}  // namespace

template <int D, int NT>
static cudaError_t launch_decode(const DecodeParams &p, int grid, cudaStream_t s)
{
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void *>(ub_attn_decode_kernel<D, NT>),
                                           DecShape<D, NT>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_ex(ub_attn_decode_kernel<D, NT>, p, grid, DEC_THREADS, DecShape<D, NT>::SMEM, 1, p.pdl != 0, s);
}

cudaError_t launch_attn_decode(const DecodeParams &p, int grid, cudaStream_t s)
{
    const bool wide = p.group > 8;
    if (p.head_dim == 128) return wide ? launch_decode<128, 2>(p, grid, s) : launch_decode<128, 1>(p, grid, s);
    return wide ? launch_decode<64, 2>(p, grid, s) : launch_decode<64, 1>(p, grid, s);
}

}  // namespace ubk
