// Attention of drafted tokens over a paged key/value cache: a tree of drafts for each sequence.
//
//   O_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale * q_i . k_j - m_i)
//
// over the keys j of the text (all, or those in the window and the sinks), of the ancestors of
// draft i and of itself, in one pass over the keys: a running maximum m and sum l per row, O
// rescaled when the maximum grows by more than 2^8 (see ub_attn_prompt.cu).
//
// Few rows over many keys: bound by HBM as long as the keys and values are read once. A q tile is
// 128 rows, token by token and in a token the query heads of one key/value head (any number of
// them up to 128: 128 / heads tokens). A work item is up to two q tiles of one sequence and
// key/value head. The tensor core takes S = Q K^T (128 rows x 128 keys, from shared memory) and
// O += P V (P from TMEM), and has two pipelines of S, softmax, P and O:
//  - an item of one q tile gives them alternate key tiles, so that the chain S -> softmax -> P V
//    of a tile (2200 cycles) hides behind the other's, and joins the two O in TMEM at its end;
//  - an item of two q tiles gives each its q tile, and both take every key tile.
// What a draft sees of the other drafts is found where it is needed, in the one or two key tiles
// that hold drafts: a thread walks from its row's draft up its parents and sets a bit per key.
// So a tree may have any number of drafts, and nothing is prepared or kept between calls.
//
// Work split: the (item, key tile) pairs of the whole call are laid end to end and every CTA
// takes an equal, contiguous range, found on the device from the starts and lengths, as in
// ub_attn_decode.cu. The parts of an item that spans CTAs go to the workspace and are joined, in
// CTA order, by all its CTAs, a share of the outputs each, once a counter says that all are there.
//
// Roles (12 warps, one CTA per SM):
//   warps 0-3, 4-7   softmax of pipeline 0 and 1, one thread per row; the item's end; joins
//   warp 8           loads (TMA): Q, then K and V tiles in a ring
//   warps 9, 10      MMA issue for pipeline 0 and 1
//   warp 11          zeroes the rows of V past a sequence's end in its last tile
#include <cuda_bf16.h>

#include "ub_attn.h"
#include "ub_attn_mma.cuh"
#include "ub_device.cuh"
#include "ub_internal.h"

namespace ubk {
namespace {

constexpr int TR_THREADS = 384;
constexpr int KEYS = TREE_KEYS, ROWS = TREE_ROWS;
// Registers per thread by role; their sum is what the block is launched with (384 x 168).
constexpr int SOFTMAX_REGS = 200, SINGLE_REGS = 104;
static_assert(2 * SOFTMAX_REGS + SINGLE_REGS == 3 * 168, "register split");
constexpr int TM_S = 0, TM_O = 256;      // TMEM columns: S_i at 128 i, O_i at 256 + 128 i
constexpr float RESCALE_LOG2 = 8.f;      // growth of the maximum (log2) that is put off
// What the end of an item (O joined and written, the next queries loaded) counts in the split, in
// key tiles; what a join costs; key tiles of a CTA, at least.
constexpr int ITEM_COST = 3, JOIN_TILES = 5, MIN_TILES = 2;

template <int D>
struct TreeShape {
    static constexpr int TILE_BYTES = KEYS * D * 2;
    static constexpr int HALF_BYTES = KEYS * 128;         // 64 columns of a tile
    static constexpr int STAGES = D == 128 ? 5 : 10;
    static constexpr int CONTROL = 2048 + 768;            // (m, l) of two tiles; barriers
    static constexpr int SMEM = (2 + STAGES) * TILE_BYTES + CONTROL;
    static_assert(SMEM <= 232448, "shared memory");
};

// A sequence of the call.
struct Seq {
    int start, n;   // first token, tokens
    int len, text;  // keys; those before the drafts (below zero: some drafts have no key)
    int lo;         // first key in the window of a draft that follows the text
    int near, far;  // its key tile; key tiles before it that hold sinks
    int tiles;      // key tiles in sight
    int blocks;     // items of a key/value head
    __device__ __forceinline__ int tile(int t) const { return t < far ? t : t - far + near; }
    // Units of an item in the split.
    __device__ __forceinline__ int span() const { return tiles > 1 ? tiles : 1; }
    __device__ __forceinline__ int cost() const { return span() + ITEM_COST; }
};
__device__ __forceinline__ Seq seq_of(const TreeParams &p, int s)
{
    Seq q;
    int a = p.b.seq_starts[s], z = p.b.seq_starts[s + 1];
    const int len = p.b.kv_lens[s];
    a = a < 0 ? 0 : (a > p.T ? p.T : a);
    z = z < a ? a : (z > p.T ? p.T : z);
    const int64_t most = static_cast<int64_t>(p.b.table_width) << p.b.page_shift;
    q.start = a;
    q.n = z - a;
    q.len = len < 0 ? 0 : (len > most ? static_cast<int>(most) : len);
    q.text = q.len - q.n;
    q.lo = p.window > 0 && q.text >= p.window ? q.text - p.window + 1 : 0;
    q.near = q.lo / KEYS;
    const int sunk = (p.sinks + KEYS - 1) / KEYS;
    q.far = sunk < q.near ? sunk : q.near;
    q.tiles = (q.len + KEYS - 1) / KEYS - q.near + q.far;
    q.blocks = (q.n + 2 * p.tokens - 1) / (2 * p.tokens);
    return q;
}

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}
__device__ __forceinline__ int64_t warp_sum(int64_t v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The equal split of `total` units over CTAs: CTA c's first unit, and the CTA of a unit.
struct Split {
    int64_t base, rem;
    __device__ __forceinline__ int64_t first(int64_t c) const { return c * base + (c < rem ? c : rem); }
    __device__ __forceinline__ int owner(int64_t x) const
    {
        const int64_t cut = rem * (base + 1);
        return static_cast<int>(x < cut ? quotient(x, base + 1) : rem + quotient(x - cut, base));
    }
};

// A CTA's way through its share of the call: the current item, and its key tiles [t0, t1).
struct Walk {
    const TreeParams &p;
    Split split;
    int64_t x, left;  // unit of the whole call at t0 (not counted for whole items), units to go
    int s, item;      // sequence, item of it
    int t0, t1;
    Seq q;

    __device__ __forceinline__ explicit Walk(const TreeParams &params) : p(params) {}
    __device__ __forceinline__ bool more() const { return left > 0 && s < p.b.n_seqs; }
    __device__ __forceinline__ void cut() { t1 = q.span() - t0 < left ? q.span() : t0 + static_cast<int>(left); }
    __device__ __forceinline__ void settle_on()  // an item of sequence s, or of the next that has one
    {
        while (s < p.b.n_seqs) {
            q = seq_of(p, s);
            if (item < q.blocks * p.units) break;
            item = 0;
            ++s;
        }
        cut();
    }
    __device__ __forceinline__ void next()
    {
        const int64_t units = q.cost() - t0 < left ? q.cost() - t0 : left;
        x += units;
        left -= units;
        t0 = 0;
        if (++item < q.blocks * p.units) {
            cut();
        } else if (left > 0) {
            item = 0;
            ++s;
            settle_on();
        }
    }
    __device__ __forceinline__ int unit() const { return item / q.blocks; }
    __device__ __forceinline__ int first_token() const { return (item % q.blocks) * 2 * p.tokens; }
    __device__ __forceinline__ int tokens() const  // of this item
    {
        const int n = q.n - first_token();
        return n < 2 * p.tokens ? n : 2 * p.tokens;
    }
    // Whole in this CTA; and how many key tiles of it there are to do (an item without keys: none).
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == q.span(); }
    __device__ __forceinline__ int todo() const { return q.tiles > 0 ? t1 - t0 : 0; }
};

// Sets out CTA `cta` of `grid` (one warp, all lanes alike).
__device__ void begin(Walk &w, int lane, int cta, int grid)
{
    const TreeParams &p = w.p;
    w.left = 0;
    w.s = w.item = w.t0 = w.t1 = 0;
    w.x = 0;
    w.split = Split{0, 0};
    // Sums over the sequences: items, and units of the split.
    Seq own;
    own.n = own.blocks = own.tiles = 0;
    if (lane < p.b.n_seqs) own = seq_of(p, lane);
    int64_t items = own.blocks, total = static_cast<int64_t>(own.blocks) * (own.blocks > 0 ? own.cost() : 0);
    int most = own.blocks > 0 ? own.span() : 0;
    for (int i = lane + 32; i < p.b.n_seqs; i += 32) {
        const Seq q = seq_of(p, i);
        if (q.blocks == 0) continue;
        items += q.blocks;
        total += static_cast<int64_t>(q.blocks) * q.cost();
        most = q.span() > most ? q.span() : most;
    }
    items = warp_sum(items) * p.units;
    total = warp_sum(total) * p.units;
    most = __reduce_max_sync(0xffffffffu, most);
    if (items == 0) return;
    // A CTA per item where no item is much longer than an equal share would be: a share saves the
    // difference and costs a join. Else equal shares, of at least MIN_TILES units, or a CTA per
    // item where those are shorter.
    const bool whole = items <= grid && static_cast<int64_t>(most - JOIN_TILES) * grid <= total - items * ITEM_COST;
    int64_t ctas = whole ? items : total / MIN_TILES;
    if (!whole && ctas < items) ctas = items;
    ctas = ctas > grid ? grid : ctas;
    if (cta >= ctas) return;
    const int64_t base = quotient(total, ctas);
    w.split = Split{base, total - base * ctas};
    const int64_t at = whole ? cta : w.split.first(cta);
    // The sequence that holds item or unit `at`, and those before it.
    int64_t seen = 0, before = 0;
    for (int i0 = 0; i0 < p.b.n_seqs; i0 += 32) {
        Seq q = own;
        if (i0 > 0 && i0 + lane < p.b.n_seqs) q = seq_of(p, i0 + lane);
        int64_t mine = 0;
        if (i0 + lane < p.b.n_seqs && q.blocks > 0) mine = static_cast<int64_t>(q.blocks) * p.units * (whole ? 1 : q.cost());
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, seen + upto > at);
        if (past != 0u) {
            const int l = __ffs(static_cast<int>(past)) - 1;
            w.s = i0 + l;
            before = seen + __shfl_sync(0xffffffffu, upto - mine, l);
            break;
        }
        seen += __shfl_sync(0xffffffffu, upto, 31);
    }
    w.q = seq_of(p, w.s);
    if (whole) {
        w.item = static_cast<int>(at - before);
        w.left = w.q.span();
    } else {
        w.x = at;
        w.left = w.split.first(cta + 1) - at;
        w.item = static_cast<int>(quotient(at - before, w.q.cost()));
        w.t0 = static_cast<int>(at - before - static_cast<int64_t>(w.item) * w.q.cost());
        if (w.t0 >= w.q.span()) {  // behind the item's last tile: on to the next
            w.x += w.q.cost() - w.t0;
            w.left -= w.q.cost() - w.t0;
            w.t0 = 0;
            ++w.item;
        }
    }
    w.settle_on();
}

// The low `n` bits (n may be below zero or past 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

// The draft that draft i of a sequence follows, -1: the text.
__device__ __forceinline__ int parent_of(const TreeParams &p, const Seq &q, int i)
{
    const int up = p.parents[q.start + i];
    if (up >= -1 && up < i) return up;
    atomicCAS(p.b.status, 0, UB_ERR_ARG);
    return -1;
}

// Which of the 128 keys from key0 on draft `i` at position `pos` sees (i < 0: a row of no draft).
__device__ void keys_seen(const TreeParams &p, const Seq &q, int i, int pos, int key0, uint32_t *bits)
{
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int first = key0 + 32 * w;
        bits[w] = low_bits(q.text - first);
        if (p.window > 0) bits[w] &= ~low_bits(pos - p.window + 1 - first) | low_bits(p.sinks - first);
    }
    const int gone = key0 - q.text;  // drafts before this tile, or before the cache
    const int least = gone > -q.text ? gone : -q.text;
    for (int d = 0; i >= 0 && i >= least; ++d) {
        const int c = i - gone;
        const bool seen = c < KEYS && (p.window == 0 || d < p.window || pos - d < p.sinks);
#pragma unroll
        for (int w = 0; w < 4; ++w)
            if (seen && (c >> 5) == w) bits[w] |= 1u << (c & 31);
        i = parent_of(p, q, i);
    }
    __syncwarp();
}

// An item that other CTAs have parts of, as its CTA keeps it for the join.
struct Pending {
    int64_t item0;            // its first unit
    int span, row0, n, unit;  // units, first token and tokens, unit of heads
};

template <int D>
__global__ void __launch_bounds__(TR_THREADS, 1) ub_attn_tree_kernel(const __grid_constant__ TreeParams p)
{
    using Sh = TreeShape<D>;
    constexpr int NST = Sh::STAGES, HALVES = D / 64;
    extern __shared__ __align__(1024) uint8_t base[];
    const uint32_t sm_q = smem_u32(base), sm_kv = sm_q + 2 * Sh::TILE_BYTES;
    float *sm_max = reinterpret_cast<float *>(base + (2 + NST) * Sh::TILE_BYTES);  // [2][128]
    float *sm_sum = sm_max + 256;                                                  // [2][128]
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm_sum + 256);
    const uint32_t kv_full = smem_u32(bars), v_raw = kv_full + 8 * NST, kv_empty = kv_full + 16 * NST,
                   misc = kv_full + 24 * NST;
    const uint32_t q_full = misc, q_empty = misc + 8, s_full = misc + 16, p_full = misc + 32, o_full = misc + 48,
                   o_empty = misc + 64, both = misc + 80, parts_done = misc + 88, join_go = misc + 96, drain = misc + 112;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(bars) + 24 * NST + 128);
    volatile uint32_t *issued = tmem_slot + 1;   // ring positions whose loads have been issued
    static_assert(24 * NST + 136 <= 768, "barrier area");

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if ((sm_q & 1023u) != 0u) {  // the swizzled tiles need what the declaration asks for
        if (threadIdx.x == 0) atomicCAS(p.b.status, 0, UB_ERR_ALIGN);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(kv_full + 8 * i, 1);
            mbar_init(v_raw + 8 * i, 1);
            mbar_init(kv_empty + 8 * i, 2);  // both pipelines, or one of them twice
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);               // both issuing warps
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 4);
            mbar_init(o_full + 8 * i, 1);
            mbar_init(o_empty + 8 * i, 8);   // all softmax warps
            mbar_init(join_go + 8 * i, 1);
            mbar_init(drain + 8 * i, 1);
        }
        *issued = 0u;
        mbar_init(both, 8);
        mbar_init(parts_done, 8);
        fence_mbar_init();
        prefetch_tmap(&p.tmQ);
        prefetch_tmap(&p.tmK);
        prefetch_tmap(&p.tmV);
    }
    // Rows of a q tile that no load writes are multiplied too, and must not hold huge numbers.
    if (p.tokens * p.unit_heads < ROWS) {
        for (int i = threadIdx.x; i < 2 * Sh::TILE_BYTES / 16; i += TR_THREADS) st_shared_v4(sm_q + 16 * i, 0u, 0u, 0u, 0u);
        fence_proxy_async_shared();
    }
    if (warp == 9) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    const WaitCtx wc{p.abort_word, p.b.status, p.timeout_ns, p.epoch};
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        alive = __all_sync(0xffffffffu, mbar_wait(bar, parity, wc)) != 0;
        return alive;
    };
    auto arrive = [&](uint32_t bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    Walk w(p);
    begin(w, lane, blockIdx.x, gridDim.x);

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        more_registers<SOFTMAX_REGS>();
        const int i = warp >> 2;                       // pipeline
        const int row = (warp & 3) * 32 + lane;
        const int row_token = row / p.unit_heads, row_head = row - row_token * p.unit_heads;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + TM_S + i * 128 + lanes, to = tmem + TM_O + i * 128 + lanes;
        const float sl = p.scale * 1.4426950408889634f;
        const int G = gridDim.x;
        uint32_t n_s = 0, n_o[2] = {0, 0};             // phases used
        Pending pend[2] = {{0, 0, 0, 0, 0}, {0, 0, 0, 0, 0}};  // begun before this CTA; going on after it
        auto store_lse = [&](int64_t token, int head, float m, float l) {
            if (p.lse) p.lse[token * p.heads + head] = l > 0.f ? m * p.scale + logf(l) : (l == 0.f ? -INFINITY : l);
        };
        for (uint32_t k = 0; w.more() && alive; ++k, w.next()) {
            const Seq &q = w.q;
            const int ntok = w.tokens(), todo = w.todo();
            const bool two = ntok > p.tokens;
            const int token = (two ? i * p.tokens : 0) + row_token;  // of the item
            const bool real = row_token < p.tokens && token < ntok;
            const int draft = real ? w.first_token() + token : -1;
            int pos = q.text;
            if (p.window > 0 && draft >= 0)
                for (int up = parent_of(p, q, draft); up >= 0; up = parent_of(p, q, up)) ++pos;
            __syncwarp();
            float m = -INFINITY, l = 0.f;
            for (int j = two ? 0 : i; j < todo; j += two ? 1 : 2) {
                const int key0 = q.tile(w.t0 + j) * KEYS;
                uint32_t bits[4];
                // some row does not see all of the tile: drafts, or keys left of a window
                const bool edge = key0 + KEYS > q.text || (p.window > 0 && key0 <= q.len - p.window && key0 + KEYS > p.sinks);
                if (edge) keys_seen(p, q, draft, pos, key0, bits);
                if (!wait(s_full + 8 * i, n_s & 1)) break;
                ++n_s;
                tc_fence_after();
                float s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, reinterpret_cast<uint32_t *>(s) + c * 32);
                tmem_wait_ld();
                if (edge) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (((bits[c >> 5] >> (c & 31)) & 1u) == 0u) s[c] = -INFINITY;
                }
                float mx[4] = {m, m, m, m};
#pragma unroll
                for (int c = 0; c < 128; c += 8)
#pragma unroll
                    for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], s[c + 2 * u], s[c + 2 * u + 1]);
                const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                // A first or much larger maximum (never from -inf to -inf: the difference is no number).
                const float grow = (top - m) * sl;
                const bool moves = grow > RESCALE_LOG2;
                const float f = moves ? ex2(-grow) : 1.f;
                m = moves ? top : m;
                // S of this tile being there, O of this pipeline's last tile is complete.
                if (j > (two ? 0 : i) && __any_sync(0xffffffffu, moves)) {
#pragma unroll
                    for (int c = 0; c < D; c += 16) {
                        uint32_t v[16];
                        tmem_ld16(to + c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < 16; ++u) v[u] = __float_as_uint(__uint_as_float(v[u]) * f);
                        tmem_st16(to + c, v);
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m * sl;  // no key yet: every weight is zero
                const uint64_t sl2 = pair_of(sl, sl), ref2 = pair_of(-ref, -ref);
                // Weights in BF16, the type of the values they multiply (kind::f16 wants one type for
                // both): up to 2^-8 of each, as large as the rounding of the output. Their sum takes
                // them unrounded, in fp32.
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int c0 = 0; c0 < 128; c0 += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const uint64_t x = fma2(pair_of(s[c0 + c], s[c0 + c + 1]), sl2, ref2);
                        const float e0 = ex2(low(x)), e1 = ex2(high(x));
                        sum[(c / 2) & 1] = add2(sum[(c / 2) & 1], pair_of(e0, e1));
                        pk[c / 2] = pack_bf16x2(__float_as_uint(e0), __float_as_uint(e1));
                    }
                    tmem_st16(ts + c0 / 2, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive(p_full + 8 * i);
                const uint64_t all = add2(sum[0], sum[1]);
                l = l * f + (low(all) + high(all));
            }
            if (!alive) break;

            // The item's end: both pipelines' maxima and sums, then their O.
            if (k > 0 && !wait(o_empty + 8 * i, (k - 1) & 1)) break;  // the last item's have been read
            sm_max[i * 128 + row] = m;
            sm_sum[i * 128 + row] = l;
            arrive(both);
            if (todo > 0 && !wait(o_full, n_o[0]++ & 1)) break;
            if (todo > (two ? 0 : 1) && !wait(o_full + 8, n_o[1]++ & 1)) break;
            if (!wait(both, k & 1)) break;
            tc_fence_after();
            const bool whole = w.whole();
            const int64_t out_token = static_cast<int64_t>(q.start) + w.first_token() + token;
            const int unit = w.unit(), kvh = unit / p.blocks;
            const int in_group = (unit - kvh * p.blocks) * p.unit_heads + row_head;
            const int head = kvh * p.group + in_group;
            const bool mine = real && in_group < p.group;
            // One q tile: the two pipelines' O of a row, joined; half of the columns each.
            float f0 = 1.f, f1 = 0.f, M = m, L = l;
            if (!two) {
                const float m0 = sm_max[row], m1 = sm_max[128 + row];
                M = fmaxf(m0, m1);
                const float ref = M == -INFINITY ? 0.f : M;
                f0 = ex2((m0 - ref) * sl);
                f1 = ex2((m1 - ref) * sl);
                L = sm_sum[row] * f0 + sm_sum[128 + row] * f1;
            }
            const int c0 = two || i == 0 ? 0 : D / 2, c1 = two || i == 1 ? D : D / 2;
            const int which = w.t0 == 0 ? 1 : 0, part_row = two ? i * 128 + row : row;
            const int64_t slot = static_cast<int64_t>(which) * G + blockIdx.x;
            float4 *part = reinterpret_cast<float4 *>(p.ws) + slot * (64 * D) + part_row;
            const float inv = 1.f / L;
#pragma unroll 1
            for (int c = c0; c < c1; c += 16) {
                float v[16];
                if (two) {
                    tmem_ld16(to + c, reinterpret_cast<uint32_t *>(v));
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = 0.f;
                    float u[16];
                    // a pipeline without a key tile has nothing there
                    if (todo > 0) {
                        tmem_ld16(tmem + TM_O + lanes + c, reinterpret_cast<uint32_t *>(u));
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = u[e] * f0;
                    }
                    if (todo > 1) {
                        tmem_ld16(tmem + TM_O + 128 + lanes + c, reinterpret_cast<uint32_t *>(u));
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] += u[e] * f1;
                    }
                }
                if (mine && whole) {
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + out_token * p.o_row + head * p.o_head + c;
#pragma unroll
                    for (int e = 0; e < 16; e += 8) {
                        uint32_t x[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            x[y] = L == 0.f ? 0u
                                            : pack_bf16x2(__float_as_uint(v[e + 2 * y] * inv), __float_as_uint(v[e + 2 * y + 1] * inv));
                        *reinterpret_cast<uint4 *>(dst + e) = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                } else if (mine) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) part[(c + e) / 4 * 256] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
                __syncwarp();
            }
            tc_fence_before();
            if (mine && (two || i == 0)) {
                if (whole) {
                    store_lse(out_token, head, M, L);
                } else {
                    p.ws_rows[slot * 512 + part_row] = M;
                    p.ws_rows[slot * 512 + 256 + part_row] = L;
                }
            }
            arrive(o_empty);
            arrive(o_empty + 8);
            if (!whole && w.t0 != 0) pend[0] = Pending{w.x - w.t0, q.span(), q.start + w.first_token(), ntok, unit};
            if (!whole && w.t0 == 0) pend[1] = Pending{w.x, q.span(), q.start + w.first_token(), ntok, unit};
        }

        // The parts of split items, joined when the CTA's own tiles are done: a CTA says that its
        // parts are there for both its items before it waits for either, so that no two items
        // wait for one another (all CTAs are resident: one per SM, no more than SMs).
        if ((pend[0].span | pend[1].span) != 0 && alive) {
            arrive(parts_done);
            if (warp < 2) {  // a warp for each
                const Pending it = warp == 0 ? pend[0] : pend[1];
                if (it.span != 0) {
                    const int a = w.split.owner(it.item0), parts = w.split.owner(it.item0 + it.span - 1) - a + 1;
                    // a count of the item's parts, and one, never reset, of how often all have come
                    uint32_t *counter = p.counters + a, *times = p.times + a;
                    if (wait(parts_done, 0) && lane == 0) {
                        const uint32_t before = *static_cast<volatile uint32_t *>(times);
                        uint32_t come;
                        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(come) : "l"(counter) : "memory");
                        if (come == static_cast<uint32_t>(parts - 1)) {
                            *counter = 0u;             // zero again for the next call
                            st_release_u32(times, before + 1u);
                        } else {
                            WaitClock clk;
                            for (uint32_t n = 1; alive; ++n) {
                                uint32_t v;
                                asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(times) : "memory");
                                if (v != before) break;
                                if ((n & 15u) == 0 && !clk.ok(wc)) alive = false;
                            }
                        }
                    }
                    alive = __all_sync(0xffffffffu, alive) != 0;
                    arrive(join_go + 8 * warp);
                }
            }
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const Pending it = pend[which];
                if (it.span == 0) continue;
                if (!alive || !wait(join_go + 8 * which, 0)) break;
                const int a = w.split.owner(it.item0), parts = w.split.owner(it.item0 + it.span - 1) - a + 1;
                const int kvh = it.unit / p.blocks, h0 = (it.unit - kvh * p.blocks) * p.unit_heads;
                const int rows = it.n * p.unit_heads, tile_rows = p.tokens * p.unit_heads;
                const int units = rows * (D / 4);      // of four outputs, rows fastest
                // Units of this CTA: `width` lanes each, as few as have all parts in flight at once.
                constexpr int U = 5;                   // parts in flight per lane
                int width_shift = 0;
                while (width_shift < 5 && (U << width_shift) < parts) ++width_shift;
                const int width = 1 << width_shift, at_once = 256 >> width_shift;
                const int per = (units + parts - 1) / parts, i_cta = static_cast<int>(blockIdx.x) - a;
                const int end = (i_cta + 1) * per < units ? (i_cta + 1) * per : units;
                for (int u0 = i_cta * per; u0 < end; u0 += at_once) {
                    const int u = u0 + (static_cast<int>(threadIdx.x) >> width_shift);
                    const int c4 = u / rows, r = u - c4 * rows;
                    const int part_row = r < tile_rows ? r : 128 + r - tile_rows;
                    float MM = -INFINITY, LL = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int i0 = lane & (width - 1); i0 < parts && u < end; i0 += width * U) {
                        float4 v[U];
                        float mm[U], ll[U], top = MM;
#pragma unroll
                        for (int e = 0; e < U; ++e) {
                            const int part = i0 + width * e;
                            mm[e] = -INFINITY;
                            ll[e] = 0.f;
                            v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (part >= parts) continue;
                            // slot 1 for the CTA in which the item begins, 0 for the others
                            const int64_t slot = static_cast<int64_t>(part == 0 ? G : 0) + a + part;
                            v[e] = __ldcg(reinterpret_cast<const float4 *>(p.ws) + slot * (64 * D) + c4 * 256 + part_row);
                            mm[e] = __ldcg(p.ws_rows + slot * 512 + part_row);
                            ll[e] = __ldcg(p.ws_rows + slot * 512 + 256 + part_row);
                        }
#pragma unroll
                        for (int e = 0; e < U; ++e) top = fmaxf(top, mm[e]);
                        const float ref = top == -INFINITY ? 0.f : top;
                        const float g0 = ex2((MM - ref) * sl);
                        LL *= g0;
                        acc.x *= g0;
                        acc.y *= g0;
                        acc.z *= g0;
                        acc.w *= g0;
                        MM = top;
#pragma unroll
                        for (int e = 0; e < U; ++e) {
                            const float g = ex2((mm[e] - ref) * sl);
                            LL += ll[e] * g;
                            acc.x += v[e].x * g;
                            acc.y += v[e].y * g;
                            acc.z += v[e].z * g;
                            acc.w += v[e].w * g;
                        }
                    }
                    float top = MM;
                    for (int o = width >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const float g = ex2((MM - (top == -INFINITY ? 0.f : top)) * sl);
                    LL *= g;
                    acc.x *= g;
                    acc.y *= g;
                    acc.z *= g;
                    acc.w *= g;
                    for (int o = width >> 1; o > 0; o >>= 1) {
                        LL += __shfl_xor_sync(0xffffffffu, LL, o);
                        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
                        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
                        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
                        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
                    }
                    const int tok = r / p.unit_heads, in_group = h0 + r - tok * p.unit_heads;
                    if ((lane & (width - 1)) != 0 || u >= end || in_group >= p.group) continue;
                    const int64_t out_token = static_cast<int64_t>(it.row0) + tok;
                    const int head = kvh * p.group + in_group;
                    const float inv = LL == 0.f ? 0.f : 1.f / LL;
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + out_token * p.o_row + head * p.o_head + 4 * c4;
                    *reinterpret_cast<uint2 *>(dst) =
                        make_uint2(pack_bf16x2(__float_as_uint(acc.x * inv), __float_as_uint(acc.y * inv)),
                                   pack_bf16x2(__float_as_uint(acc.z * inv), __float_as_uint(acc.w * inv)));
                    if (c4 == 0) store_lse(out_token, head, top, LL);
                }
            }
        }
    } else {
        // the four single warps
        fewer_registers<SINGLE_REGS>();
        if (warp == 8) {
            // -------------------------------------------------------- loads
            uint32_t c = 0;                            // ring position
            const int box = KEYS < (1 << p.b.page_shift) ? KEYS : (1 << p.b.page_shift), boxes = KEYS / box;
            for (uint32_t k = 0; w.more() && alive; ++k, w.next()) {
                const Seq &q = w.q;
                const bool two = w.tokens() > p.tokens;
                const int unit = w.unit(), kvh = unit / p.blocks;
                if (k > 0 && !wait(q_empty, (k - 1) & 1)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, (two ? 2 : 1) * HALVES * p.tokens * p.unit_heads * 128);
                    for (int t = 0; t < (two ? 2 : 1); ++t)
                        for (int hf = 0; hf < HALVES; ++hf)
                            tma_load_3d(sm_q + t * Sh::TILE_BYTES + hf * Sh::HALF_BYTES, &p.tmQ, q_full, hf * 64,
                                        kvh * p.group + (unit - kvh * p.blocks) * p.unit_heads,
                                        q.start + w.first_token() + t * p.tokens);
                }
                __syncwarp();
                const int32_t *table = p.b.page_table + w.s * p.b.table_row;
                const int pages = (q.len + (1 << p.b.page_shift) - 1) >> p.b.page_shift;
                int cached0 = 0, cached_n = 0, ids = -1;  // page ids, one per lane
                for (int j = 0; j < w.todo() && alive; ++j) {
                    const int kt = q.tile(w.t0 + j), key0 = kt * KEYS, ext = extent(q.len, kt);
                    const int n_box = (ext + box - 1) / box, page0 = key0 >> p.b.page_shift;
                    if (page0 + boxes > cached0 + cached_n) {
                        cached0 = page0;
                        cached_n = 32;
                        // a page that no row sees may be another sequence's by now, or nobody's
                        const int64_t first = static_cast<int64_t>(cached0 + lane) << p.b.page_shift;
                        const bool seen = cached0 + lane < pages &&
                                          (p.window == 0 || first + (int64_t(1) << p.b.page_shift) > q.lo || first < p.sinks);
                        ids = seen ? table[cached0 + lane] : -1;
                        if (seen && (ids < 0 || ids >= p.b.num_pages)) {
                            atomicCAS(p.b.status, 0, UB_ERR_ARG);
                            ids = -1;                  // outside the tensor: filled with zeros
                        }
                    }
                    for (int kind = 0; kind < 2 && alive; ++kind, ++c) {
                        const uint32_t st = c % NST;
                        if (c >= NST && !wait(kv_empty + 8 * st, (c / NST - 1) & 1)) break;
                        // The last tile of V goes through the zeroing warp when it ends inside 16 keys.
                        const bool fix = kind == 1 && ext > q.len - key0;
                        const uint32_t bar = (fix ? v_raw : kv_full) + 8 * st;
                        if (lane == 0) mbar_arrive_expect_tx(bar, n_box * HALVES * box * 128);
                        __syncwarp();
                        const int bx = lane / HALVES, hf = lane - bx * HALVES;
                        const int page = __shfl_sync(0xffffffffu, ids, (page0 - cached0 + bx) & 31);
                        if (bx < n_box)
                            tma_load_4d(sm_kv + st * Sh::TILE_BYTES + hf * Sh::HALF_BYTES + bx * box * 128,
                                        kind == 0 ? &p.tmK : &p.tmV, bar, hf * 64,
                                        boxes > 1 ? 0 : key0 & ((1 << p.b.page_shift) - 1), kvh, page);
                        __syncwarp();
                        if (lane == 0) *issued = c + 1;
                    }
                }
            }
        } else if (warp < 11) {
            // -------------------------------------------------------- MMA issue
            const int i = warp - 9;
            uint32_t c = 0, n_p = 0;
            const uint32_t tp = tmem + TM_S + i * 128, to = tmem + TM_O + i * 128;
            const uint64_t k_desc = smem_desc_sw128(sm_kv), v_desc = smem_desc_v(sm_kv, Sh::HALF_BYTES);
            constexpr uint32_t o_idesc = attn_idesc(D, true);
            // A pipeline skips the other's key tiles, and the ring may turn meanwhile: a barrier's
            // parity tells two turns apart only once the loads of this one have been issued.
            auto wait_kv = [&](uint32_t at) {
                bool there = __all_sync(0xffffffffu, static_cast<int32_t>(*issued - at) > 0) != 0;
                if (!there) {
                    WaitClock clk;
                    for (uint32_t n = 1; !there; ++n) {
                        there = __all_sync(0xffffffffu, static_cast<int32_t>(*issued - at) > 0) != 0;
                        if ((n & 15u) == 0 && !there && !__all_sync(0xffffffffu, clk.ok(wc))) return alive = false;
                    }
                }
                return wait(kv_full + 8 * (at % NST), (at / NST) & 1);
            };
            for (uint32_t k = 0; w.more() && alive; ++k, w.next()) {
                const bool two = w.tokens() > p.tokens;
                const int todo = w.todo(), len = w.q.len;
                const int last = two ? todo - 1 : todo - 1 - ((todo - 1 - i) & 1);  // this pipeline's; below zero: none
                const uint64_t q_desc = smem_desc_sw128(sm_q + (two ? i * Sh::TILE_BYTES : 0));
                if (!wait(q_full, k & 1)) break;
                if (last < 0) arrive(q_empty);
                // O of the last item has been read
                if (last < 0 && k > 0 && !wait(o_empty + 8 * i, (k - 1) & 1)) break;
                for (int j = 0; j < todo; ++j, c += 2) {
                    if (!two && (j & 1) != i) continue;
                    const uint32_t ks = c % NST, vs = (c + 1) % NST;
                    const int ext = extent(len, w.q.tile(w.t0 + j));
                    if (!wait_kv(c)) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t s_idesc = attn_idesc(ext, false);
                        const uint64_t kk = k_desc + ks * (Sh::TILE_BYTES / 16);
#pragma unroll
                        for (int s = 0; s < D / 16; ++s) {
                            const int o = (s / 4) * (Sh::HALF_BYTES / 16) + (s % 4) * 2;
                            umma_ss(tp, q_desc + o, kk + o, s_idesc, s > 0);
                        }
                        umma_commit(s_full + 8 * i);
                        umma_commit(kv_empty + 8 * ks);
                        if (!two) umma_commit(kv_empty + 8 * ks);
                        if (j == last) umma_commit(q_empty);
                    }
                    __syncwarp();
                    if (!wait(p_full + 8 * i, n_p & 1)) break;
                    ++n_p;
                    if (k > 0 && j == (two ? 0 : i) && !wait(o_empty + 8 * i, (k - 1) & 1)) break;
                    if (!wait_kv(c + 1)) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t v = v_desc + vs * (Sh::TILE_BYTES / 16);
                        for (int s = 0; s < ext / 16; ++s)
                            umma_ts(to, tp + s * 8, v + s * 128, o_idesc, j > (two ? 0 : i) || s > 0);
                        umma_commit(kv_empty + 8 * vs);
                        if (!two) umma_commit(kv_empty + 8 * vs);
                        if (j == last) umma_commit(o_full + 8 * i);
                    }
                    __syncwarp();
                }
            }
            // everything issued has completed before TMEM goes back
            if (elect_one()) {
                umma_commit(drain + 8 * i);
                mbar_wait_drain(drain + 8 * i, 0, p.timeout_ns);
            }
            __syncwarp();
        } else {
            // -------------------------------------------------------- the last keys of V
            uint32_t c = 0, used = 0;                  // ring position; phase bit per stage of v_raw
            for (; w.more() && alive; w.next()) {
                const int todo = w.todo(), len = w.q.len;
                const int kt = w.q.tile(w.t0 + todo - 1), valid = len - kt * KEYS;
                const int ext = todo > 0 ? extent(len, kt) : 0;
                if (ext > valid) {
                    const uint32_t st = (c + 2 * todo - 1) % NST;
                    if (!wait(v_raw + 8 * st, (used >> st) & 1)) break;
                    used ^= 1u << st;
                    const uint32_t v = sm_kv + st * Sh::TILE_BYTES;
                    for (int u = lane; u < (ext - valid) * (D / 8); u += 32) {
                        const int rr = valid + u / (D / 8), ch = u % (D / 8);
                        st_shared_v4(v + (ch / 8) * Sh::HALF_BYTES + rr * 128 + (ch % 8) * 16, 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_shared();
                    arrive(kv_full + 8 * st);
                }
                c += 2 * todo;
            }
        }
    }
    if (!alive) settle(200000);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_tree(const TreeParams &p, int grid, cudaStream_t s)
{
    const cudaError_t e = raise_smem_limit(reinterpret_cast<const void *>(ub_attn_tree_kernel<D>), TreeShape<D>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_ex(ub_attn_tree_kernel<D>, p, grid, TR_THREADS, TreeShape<D>::SMEM, 1, p.pdl != 0, s);
}

}  // namespace

cudaError_t launch_attn_tree(const TreeParams &p, int grid, cudaStream_t s)
{
    return p.head_dim == 128 ? launch_tree<128>(p, grid, s) : launch_tree<64>(p, grid, s);
}

}  // namespace ubk
