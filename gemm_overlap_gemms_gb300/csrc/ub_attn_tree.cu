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
// them up to 128: 128 / heads tokens). A work item is up to two q tiles (in short calls one) of
// one sequence and key/value head. The tensor core takes S = Q K^T (128 rows x 128 keys, from shared memory) and
// O += P V (P from TMEM), and has two pipelines of S, softmax, P and O:
//  - an item of one q tile gives them alternate key tiles, so that the chain S -> softmax -> P V
//    of a tile (2200 cycles) hides behind the other's, and joins the two O in TMEM at its end;
//  - an item of two q tiles gives each its q tile, and both take every key tile.
// What a draft sees of the other drafts is found where it is needed, in the key tiles that hold
// drafts: a bit per key, from the parents of 32 drafts at a time. The last tile comes first, so that a
// row's path goes on from tile to tile, and is looked up while the first keys are loaded. So a tree may
// have any number of drafts, and nothing is prepared or kept between calls.
//
// Work split: the (item, key tile) pairs of the whole call are laid end to end and every CTA
// takes an equal, contiguous range, found on the device from the starts and lengths, as in
// ub_attn_decode.cu; or every CTA takes whole items, where that costs less than the joins. The parts
// of an item that spans CTAs go to the workspace and are joined, in CTA order, by all its CTAs, a
// share of the outputs each, once a counter says that all are there.
//
// Measured (GB300): 32 sequences of 16 drafts over 8192 keys, 8 heads of 128 each way (1.07 GB): 170
// us, 6.3 TB/s, HBM-bound; heads of 64 98 us, 5.5 TB/s (an item's end, 3-4 us, weighs more). With 64
// drafts and 4 query heads to a key head, 256 rows on a key tile, 230 us (heads of 64: 161): a step
// of both pipelines, 2300 cycles, as in ub_attn_prompt.cu. 16 sequences of 16-64 drafts, 72945 keys
// (77 MB), 8 query heads on two: 38 us, of which 4 are schedule, 4 the first loads, 16 tiles, 4 the
// wait for all parts, 5-9 the join. Four sequences of 3-12 drafts, 1534 keys: 11 us,
// five dependent trips to memory, three key tiles and the output.
//
// Roles (12 warps, one CTA per SM):
//   warps 0-3, 4-7   softmax of pipeline 0 and 1, one thread per row; the item's end; joins
//   warp 8           loads (TMA) of Q and K tiles; of V tiles of heads of 64
//   warps 9, 10      MMA issue for pipeline 0 and 1
//   warp 11          schedule: this CTA's items; loads of V tiles of heads of 128
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
constexpr int SOFTMAX_REGS = 216, SINGLE_REGS = 72;
static_assert(2 * SOFTMAX_REGS + SINGLE_REGS == 3 * 168, "register split");
constexpr int ITEMS = 4;                 // items published ahead
constexpr int TM_S = 0, TM_O = 256;      // TMEM columns: S_i at 128 i (and P_i in its place), O_i at 256 + 128 i
constexpr float RESCALE_LOG2 = 8.f;      // growth of the maximum (log2) that is put off
// Units of the split, about 0.08 us: what a key tile takes in an item of one q tile and of two, heads
// of 64 and of 128; the end of an item (the pipelines run empty, O joined and written, the next
// queries loaded). From the times of CTAs of calls of mixed items: key tiles 0.5-0.6 and 1.1 us with
// heads of 64, 0.6-1.0 and 1.2 with heads of 128, ends 2-4 us.
__host__ __device__ constexpr int tile_units(int head_dim, bool two) { return two ? 15 : (head_dim == 64 ? 7 : 9); }
constexpr int ITEM_COST = 50;
// A join, more of them at once taking longer (their parts, and the latest of their CTAs). 8 query and
// 8 key/value heads of 128, 16 drafts over 2048 keys, joined and whole: 2 sequences (16 items) 16.3
// and 20.4 us, 4 18.4 and 20.8, 8 24.6 and 21.4; 16 of 64 drafts, 8 heads on 2 (64 items), 2048 keys
// 29.8 and 22.3, 3000 keys 37.5 and 28.8, 6000 keys 45.6 and 48.5.
__device__ __forceinline__ int join_units(int items) { return 80 + items; }
constexpr int MIN_UNITS = 24;            // of a CTA, at least: no less than any tile
// Units of a CTA up to which items of one q tile are preferred. 16 sequences of 64 drafts, 8 query
// and 2 key/value heads of 128, against items of two: 1024 keys 16.9 and 26.9 us, 2048 keys 29.9 and
// 28.4, 4096 keys (150 units) 37.4 and 43.3, 6000 keys (200) 46.6 and 50.8, 8192 keys (250) 60.5 and 56.8.
constexpr int SHORT_SHARE = 200;
static_assert(ITEM_COST <= TREE_MOST_UNITS && tile_units(128, true) <= MIN_UNITS, "units");

template <int D>
struct TreeShape {
    static constexpr int TILE_BYTES = KEYS * D * 2;
    static constexpr int HALF_BYTES = KEYS * 128;         // 64 columns of a tile
    static constexpr int K_STAGES = D == 128 ? 3 : 5, V_STAGES = D == 128 ? 2 : 5, STAGES = K_STAGES + V_STAGES;
    // A box takes the warp that loads it 80 cycles, and a tile of heads of 128 in pages of 16 rows
    // has 16 of them: as long as HBM takes for half of it. K and V have a warp each there (4 sequences
    // of few drafts: 13.2 to 11.6 us); with heads of 64 the second warp's waits take more issue slots
    // from the softmax than its loads save (64 sequences, 32 heads of 64: 172 us for 150).
    static constexpr bool TWO_LOADERS = D == 128;
    static constexpr int CONTROL = 2048 + 768;            // (m, l) of two tiles; barriers
    static constexpr int SMEM = (2 + STAGES) * TILE_BYTES + CONTROL;
    // The rows that a CTA joins: those of an item and one more of each part at most.
    static_assert((2 * ROWS + TREE_MOST_CTAS) * 4 * tree_part_row(D) <= (2 + STAGES) * TILE_BYTES, "memory of a join");
    static_assert(SMEM <= 232448, "shared memory");
};

// A sequence of the call.
struct Seq {
    int start, n;   // first token, tokens
    int len, text;  // keys; those before the drafts (below zero: some drafts have no key)
    int lo;         // first key in the window of a draft that follows the text
    int near, far;  // its key tile; key tiles before it that hold sinks
    int tiles;      // key tiles in sight, at least one
    int blocks;     // items of a key/value head
    int per;        // units of a key tile
    // Units of an item (2^24 tiles at most).
    __device__ __forceinline__ int span() const { return tiles * per; }
    __device__ __forceinline__ int cost() const { return span() + ITEM_COST; }
};
// height: tokens of an item
__device__ __forceinline__ Seq seq_from(const TreeParams &p, int a, int z, int len, int height)
{
    Seq q;
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
    q.tiles = q.len > 0 ? (q.len + KEYS - 1) / KEYS - q.near + q.far : 1;
    q.blocks = static_cast<int>(static_cast<uint32_t>(q.n + height - 1) / static_cast<uint32_t>(height));
    q.per = tile_units(p.head_dim, height > p.tokens && q.n > p.tokens);
    return q;
}
__device__ __forceinline__ Seq seq_of(const TreeParams &p, int s, int height)
{
    return seq_from(p, p.b.seq_starts[s], p.b.seq_starts[s + 1], p.b.kv_lens[s], height);
}
// Lane l's sequence.
__device__ __forceinline__ Seq from_lane(const Seq &q, int l)
{
    Seq r;
    r.start = __shfl_sync(0xffffffffu, q.start, l);
    r.n = __shfl_sync(0xffffffffu, q.n, l);
    r.len = __shfl_sync(0xffffffffu, q.len, l);
    r.text = __shfl_sync(0xffffffffu, q.text, l);
    r.lo = __shfl_sync(0xffffffffu, q.lo, l);
    r.near = __shfl_sync(0xffffffffu, q.near, l);
    r.far = __shfl_sync(0xffffffffu, q.far, l);
    r.tiles = __shfl_sync(0xffffffffu, q.tiles, l);
    r.blocks = __shfl_sync(0xffffffffu, q.blocks, l);
    r.per = __shfl_sync(0xffffffffu, q.per, l);
    return r;
}

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}
__device__ __forceinline__ int quotient(int a, int b) { return static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)); }
__device__ __forceinline__ int64_t warp_sum(int64_t v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

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

// A CTA's way through its share of the call: the current item, and its key tiles [t0, t1), those
// whose first unit lies in the share.
struct Walk {
    const TreeParams &p;
    Split split;
    int64_t x, left;  // first unit of the item here, units to go; whole items: items to go
    int off;          // units of the item that are others' (before x)
    bool by_items;    // whole items only
    int height;       // tokens of an item: one or two q tiles of them
    int s, item;      // sequence, item of it
    int t0, t1;
    Seq q;

    __device__ __forceinline__ explicit Walk(const TreeParams &params) : p(params) {}
    __device__ __forceinline__ bool more() const { return left > 0 && s < p.b.n_seqs; }
    __device__ __forceinline__ void cut()
    {
        if (by_items) {
            t0 = 0;
            t1 = q.tiles;
            return;
        }
        const uint32_t per = q.per, end = off + left < q.span() ? static_cast<int>(off + left) : q.span();
        t0 = static_cast<int>((off + per - 1) / per);
        t1 = static_cast<int>((end + per - 1) / per);
    }
    __device__ __forceinline__ void settle_on()  // an item of sequence s, or of the next that has one
    {
        while (s < p.b.n_seqs) {
            q = seq_of(p, s, height);
            if (item < q.blocks * p.units) break;
            item = 0;
            ++s;
        }
        cut();
    }
    __device__ __forceinline__ void next()
    {
        const int units = by_items ? 1 : (q.cost() - off < left ? q.cost() - off : static_cast<int>(left));
        x += units;
        left -= units;
        off = 0;
        if (++item < q.blocks * p.units) {
            cut();
        } else if (left > 0) {
            item = 0;
            ++s;
            settle_on();
        }
    }
    __device__ __forceinline__ int unit() const { return q.blocks == 1 ? item : item / q.blocks; }
    __device__ __forceinline__ int first_token() const { return (item - unit() * q.blocks) * height; }
    __device__ __forceinline__ int tokens() const  // of this item
    {
        const int n = q.n - first_token();
        return n < height ? n : height;
    }
    // Whole in this CTA; and how many key tiles of it there are to do (an item without keys: none).
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == q.tiles; }
    __device__ __forceinline__ int todo() const { return q.len > 0 ? t1 - t0 : 0; }
};

// Sets out CTA `cta` of `grid` (one warp, all lanes alike). I: a type that holds the units of the
// call. (It runs cold, and everything waits for it: 32-bit where they fit.)
template <typename I>
__device__ __forceinline__ void begin(Walk &w, int lane, int cta, int grid)
{
    const TreeParams &p = w.p;
    w.left = w.x = 0;
    w.off = w.s = w.item = w.t0 = w.t1 = 0;
    w.by_items = false;
    w.split = Split{0, 0};
    const int n_seqs = p.b.n_seqs;
    Seq own;
    I items, total;
    int most;
    w.height = 2 * p.tokens;
#pragma unroll 1
    for (;;) {
        // Sums over the sequences: items, and units of the split; q tiles.
        I tiles = 0;
        items = total = 0;
        most = 0;
        own = Seq{0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
        for (int i = lane; i < n_seqs; i += 32) {
            const Seq q = seq_of(p, i, w.height);
            if (i == lane) own = q;
            items += q.blocks;
            tiles += static_cast<uint32_t>(q.n + p.tokens - 1) / static_cast<uint32_t>(p.tokens);
            total += static_cast<I>(q.blocks) * q.cost();
            most = q.blocks > 0 && q.span() > most ? q.span() : most;
        }
        items = warp_sum(items) * p.units;
        tiles = warp_sum(tiles) * p.units;
        total = warp_sum(total) * p.units;
        most = __reduce_max_sync(0xffffffffu, most);
        if (items == 0) return;
        // Items of one q tile where those are no more than the CTAs and the shares are short: the
        // keys are then read twice, but a part that has to be joined is half as large.
        if (tiles > grid || tiles == items || total > static_cast<I>(grid) * SHORT_SHARE) break;
        w.height = p.tokens;
    }
    // Whole items, as many for each CTA, where the longest ones in every round would not take much
    // longer than equal shares: a share saves the difference and costs a join. Else equal shares,
    // of at least MIN_UNITS units.
    const I rounds = quotient(items + grid - 1, static_cast<I>(grid));
    w.by_items = static_cast<int64_t>(rounds) * most <= quotient(total - items * ITEM_COST, static_cast<I>(grid)) +
                 join_units(static_cast<int>(items < 96 ? items : 96));
    const I work = w.by_items ? items : total;
    I ctas = w.by_items ? items : total / MIN_UNITS;
    ctas = ctas < 1 ? 1 : (ctas > grid ? grid : ctas);
    if (cta >= ctas) return;
    const I base = quotient(work, ctas);
    w.split = Split{base, work - base * ctas};
    const I at = static_cast<I>(w.split.first(cta));
    // The sequence that holds item or unit `at`, and those before it.
    I seen = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < n_seqs; i0 += 32) {
        Seq q = own;
        if (i0 > 0) q = seq_of(p, i0 + lane < n_seqs ? i0 + lane : n_seqs - 1, w.height);
        I mine = i0 + lane < n_seqs ? static_cast<I>(q.blocks) * p.units * (w.by_items ? 1 : q.cost()) : 0, upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const I y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, seen + upto > at);
        if (past != 0u) {
            const int l = __ffs(static_cast<int>(past)) - 1;
            w.s = i0 + l;
            w.q = from_lane(q, l);
            seen += __shfl_sync(0xffffffffu, upto - mine, l);
            break;
        }
        seen += __shfl_sync(0xffffffffu, upto, 31);
    }
    w.x = at;
    w.left = w.split.first(cta + 1) - at;
    if (w.by_items) {
        w.item = static_cast<int>(at - seen);
    } else {
        w.item = static_cast<int>(quotient(at - seen, static_cast<I>(w.q.cost())));
        w.off = static_cast<int>(at - seen - static_cast<I>(w.item) * w.q.cost());
    }
    w.cut();
    if (w.t0 >= w.q.tiles) w.next();  // behind the first unit of the item's last tile: on to the next
}

// One item of a CTA as the schedule warp publishes it. The other warps read it where they use it,
// so that it takes no registers beside a row's scores.
struct Item {
    int seq;         // sequence; -1: no more items
    int row0, ntok;  // first token of the call, tokens
    int first;       // first draft
    int kvh, h0;     // key/value head; first query head, of those that share it
    int len, text;   // as in Seq
    int lo, near, far;
    int t0, todo;    // key tiles in sight: the first one, how many (0: the item has no keys)
    int whole;       // all of the item's
    // The last keys first: a row's path, which goes from its own draft up, is then taken once.
    __device__ __forceinline__ int tile(int j) const
    {
        const int t = t0 + todo - 1 - j;
        return t < far ? t : t - far + near;
    }
};
// An item that other CTAs have parts of, for the join.
struct Pending {
    int row0, n, kvh, h0;
    int a, parts;       // the CTA in which it begins, and how many have parts; 0: no such item
};

// The low `n` bits (n may be below zero or past 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

// A row's way along its path: the next draft of it that no tile so far has held (below zero: none
// left), and how many came before that one, the row's own among them.
struct Path {
    int draft, steps;
};
// Which of the 128 keys from key0 on each row of a warp sees; start: the token of the sequence's first
// draft, text: keys before its n drafts. The drafts are taken a word of 32 keys at a time, from the last:
// a lane has one of them, its ancestors within the word come from doubling steps along the parents,
// and the rows on it read them there and go on with the first ancestor before the word. So a path
// costs a few steps per word, however long it is (48 sequences, chains of 7-51 drafts in a window, 8
// heads: 27.7 us; each row walking by itself, a trip to memory for each ancestor: 40.4. One chain of
// 16384 drafts: 1.8 and 7.0 ms).
__device__ __forceinline__ void keys_seen(const TreeParams &p, int start, int n, int text, Path &path, int key0, int lane, uint32_t *bits)
{
    const int gone = key0 - text;  // drafts before this tile
    // A row's position is needed where its window ends; drafts further from it than that lie in
    // such tiles, too.
    const bool ends = p.window > 0 && key0 <= text + n - p.window;
    int pos = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) bits[w] = 0u;
#pragma unroll 1
    for (int pass = ends ? 0 : 1; pass < 2; ++pass) {  // to the end of the path, for the position; this tile's
        int i = path.draft, d = path.steps;
        const int low = pass == 0 || gone < 0 ? 0 : gone;
#pragma unroll 1
        for (;;) {
            const int top = __reduce_max_sync(0xffffffffu, i);
            if (top < low) break;
            const int from = gone + ((top - gone) & ~31), word = (from - gone) >> 5;
            const int least = from > 0 ? from : 0, mine = from + lane;  // the word's first draft, the lane's
            int up = mine >= 0 && mine < n ? p.parents[start + mine] : -1;
            if (up < -1 || (up >= mine && up >= 0)) {  // it does not come before its child: the text
                atomicCAS(p.b.status, 0, UB_ERR_ARG);
                up = -1;
            }
            uint32_t held = 1u << lane;
#pragma unroll
            for (int twice = 0; twice < 5 && __any_sync(0xffffffffu, up >= least); ++twice) {
                const uint32_t h = __shfl_sync(0xffffffffu, held, (up - from) & 31);
                const int u = __shfl_sync(0xffffffffu, up, (up - from) & 31);
                if (up >= least) held |= h, up = u;
            }
            const int at = i - from;
            held = __shfl_sync(0xffffffffu, held, at & 31);
            up = __shfl_sync(0xffffffffu, up, at & 31);
            if (i < least) continue;
            uint32_t see = pass == 1 ? held : 0u;
            if (p.window > 0 && word < 4 && d + __popc(held) > p.window)  // a path that leaves the window
                for (uint32_t rest = see, k = d; rest != 0u; ++k) {
                    const uint32_t last = 0x80000000u >> __clz(rest);
                    rest ^= last;
                    if (static_cast<int>(k) >= p.window && pos - static_cast<int>(k) >= p.sinks) see ^= last;
                }
#pragma unroll
            for (int w = 0; w < 4; ++w) bits[w] |= w == word ? see : 0u;
            d += __popc(held);
            i = up < least ? up : -1;                  // (always below: 32 drafts are five steps)
        }
        if (pass == 0)
            pos = text + d - 1;
        else
            path = Path{i, d};
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int first = key0 + 32 * w;
        uint32_t old = low_bits(text - first);
        if (ends) old &= ~low_bits(pos - p.window + 1 - first) | low_bits(p.sinks - first);
        bits[w] |= old;
    }
}

__device__ __forceinline__ void store_lse(const TreeParams &p, int64_t token, int head, float m, float l)
{
    if (p.lse) p.lse[token * p.heads + head] = l > 0.f ? m * p.scale + logf(l) : (l == 0.f ? -INFINITY : l);
}

// 16 bytes from global to shared memory, past L1.
__device__ __forceinline__ void copy16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// A part of a split item in the workspace: 256 rows of D columns, maximum and sum (and two words).
template <int D>
struct PartRow {
    static constexpr int FLOATS = tree_part_row(D);
    static constexpr int BYTES = 4 * FLOATS;
};

// The join of a CTA's rows [first, first + n) of an item: its parts' rows one after the other at
// `mem`, with their weights in the place of the maxima. A lane has columns [col, col + 4) of rows r0,
// r0 + 8 * 128 / D and so on.
template <int D>
struct JoinRows {
    const TreeParams &p;
    const Pending &it;
    const float *mem;
    int first, n, r0, col;
    template <int ROWS_AT_ONCE>
    __device__ __forceinline__ void run() const
    {
        constexpr int STEP = 8 * (128 / D);
        const int step = n * PartRow<D>::FLOATS;  // from part to part
#pragma unroll 1
        for (int r1 = r0; r1 < n; r1 += STEP * ROWS_AT_ONCE) {
            float4 acc[ROWS_AT_ONCE];
            const float *at[ROWS_AT_ONCE];
#pragma unroll
            for (int e = 0; e < ROWS_AT_ONCE; ++e) {
                acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                at[e] = mem + (r1 + e * STEP < n ? r1 + e * STEP : r1) * PartRow<D>::FLOATS;
            }
#pragma unroll(8 / ROWS_AT_ONCE)
            for (int q = 0; q < it.parts; ++q) {
#pragma unroll
                for (int e = 0; e < ROWS_AT_ONCE; ++e) {
                    const float4 v = *reinterpret_cast<const float4 *>(at[e] + q * step + col);
                    const float f = at[e][q * step + D];
                    acc[e].x += v.x * f;
                    acc[e].y += v.y * f;
                    acc[e].z += v.z * f;
                    acc[e].w += v.w * f;
                }
            }
#pragma unroll
            for (int e = 0; e < ROWS_AT_ONCE; ++e) {
                const int r = r1 + e * STEP, tok = (first + r) / p.unit_heads;
                const int in_group = it.h0 + first + r - tok * p.unit_heads;
                if (r >= n || in_group >= p.group) continue;
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + (static_cast<int64_t>(it.row0) + tok) * p.o_row +
                                     (it.kvh * p.group + in_group) * p.o_head + col;
                *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(__float_as_uint(acc[e].x), __float_as_uint(acc[e].y)),
                                                             pack_bf16x2(__float_as_uint(acc[e].z), __float_as_uint(acc[e].w)));
            }
        }
    }
};

template <int D>
__global__ void __launch_bounds__(TR_THREADS, 1) ub_attn_tree_kernel(const __grid_constant__ TreeParams p)
{
    using Sh = TreeShape<D>;
    constexpr int NST = Sh::STAGES, KST = Sh::K_STAGES, VST = Sh::V_STAGES, HALVES = D / 64;
    extern __shared__ __align__(1024) uint8_t base[];
    const uint32_t sm_q = smem_u32(base), sm_kv = sm_q + 2 * Sh::TILE_BYTES;
    float *sm_max = reinterpret_cast<float *>(base + (2 + NST) * Sh::TILE_BYTES);  // [2][128]
    float *sm_sum = sm_max + 256;                                                  // [2][128]
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm_sum + 256);
    const uint32_t kv_full = smem_u32(bars), kv_empty = kv_full + 8 * NST, misc = kv_full + 16 * NST;
    const uint32_t q_full = misc, q_empty = misc + 8, s_full = misc + 16, p_full = misc + 32, o_full = misc + 48,
                   o_empty = misc + 64, both = misc + 80, parts_done = misc + 88, join_go = misc + 96, drain = misc + 112,
                   joined = misc + 128;
    const uint32_t it_full = misc + 136, it_empty = it_full + 8 * ITEMS;
    Item *items = reinterpret_cast<Item *>(reinterpret_cast<uint8_t *>(bars) + 16 * NST + 136 + 16 * ITEMS);
    Pending *pend = reinterpret_cast<Pending *>(items + ITEMS);  // begun before this CTA; going on after it
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(pend + 2);
    volatile uint32_t *issued = tmem_slot + 1;   // key tiles whose loads have been issued, of K and of V
    volatile uint32_t *turn = issued + 2;        // steps that the issuer of each pipeline has done
    static_assert(16 * NST + 136 + 16 * ITEMS + sizeof(Item) * ITEMS + sizeof(Pending) * 2 + 20 <= 768, "barrier area");

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if ((sm_q & 1023u) != 0u) {  // the swizzled tiles need what the declaration asks for
        if (threadIdx.x == 0) atomicCAS(p.b.status, 0, UB_ERR_ALIGN);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(kv_full + 8 * i, 1);
            mbar_init(kv_empty + 8 * i, 2);  // both pipelines, or one of them twice
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);               // both issuing warps
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 4);    // P written, O rescaled
            mbar_init(o_full + 8 * i, 1);
            mbar_init(o_empty + 8 * i, 8);   // all softmax warps
            mbar_init(join_go + 8 * i, 1);
            mbar_init(drain + 8 * i, 1);
        }
        for (int i = 0; i < ITEMS; ++i) {
            mbar_init(it_full + 8 * i, 1);
            mbar_init(it_empty + 8 * i, 11);  // every warp but the schedule's
        }
        pend[0].parts = pend[1].parts = 0;
        issued[0] = issued[1] = turn[0] = turn[1] = 0u;
        mbar_init(both, 8);
        mbar_init(parts_done, 8);
        mbar_init(joined, 8);
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
    // Waits for the k-th item of this CTA; false at the end, or when a wait ran out.
    auto there = [&](uint32_t k) {
        return wait(it_full + 8 * (k % ITEMS), (k / ITEMS) & 1) && *static_cast<volatile int *>(&items[k % ITEMS].seq) >= 0;
    };

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
        for (uint32_t k = 0; there(k); ++k) {
            const Item &it = items[k % ITEMS];
            const int todo = it.todo;
            const bool two = it.ntok > p.tokens;
            const int token = (two ? i * p.tokens : 0) + row_token;  // of the item
            const bool real = row_token < p.tokens && token < it.ntok;
            Path path{real ? it.first + token : -1, 0};
            float m = -INFINITY, l = 0.f;
            for (int j = two ? 0 : i; j < todo; j += two ? 1 : 2) {
                // Some row does not see all of the tile: drafts, or keys left of a window. The walks run
                // while S is computed.
                const int key0 = it.tile(j) * KEYS;
                const bool edge = key0 + KEYS > it.text || (p.window > 0 && key0 <= it.len - p.window && key0 + KEYS > p.sinks);
                uint32_t bits[4];
                if (edge) keys_seen(p, it.row0 - it.first, it.len - it.text, it.text, path, key0, lane, bits);
                if (!wait(s_full + 8 * i, n_s & 1)) break;
                ++n_s;
                tc_fence_after();
                float s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, reinterpret_cast<uint32_t *>(s) + c * 32);
                tmem_wait_ld();
                if (edge) {
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        if (__any_sync(0xffffffffu, bits[w] != 0xffffffffu)) {
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if ((bits[w] & (1u << c)) == 0u) s[32 * w + c] = -INFINITY;
                        }
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
            const bool whole = it.whole != 0;
            const int64_t out_token = static_cast<int64_t>(it.row0) + token;
            const int in_group = it.h0 + row_head, head = it.kvh * p.group + in_group;
            const bool mine = real && in_group < p.group;
            // One q tile: the two pipelines' O of a row, joined; half of the columns each.
            float f0 = 1.f, f1 = 1.f, M = m, L = l;
            if (!two) {
                const float m0 = sm_max[row], m1 = sm_max[128 + row];
                M = fmaxf(m0, m1);
                const float ref = M == -INFINITY ? 0.f : M;
                f0 = ex2((m0 - ref) * sl);
                f1 = ex2((m1 - ref) * sl);
                L = sm_sum[row] * f0 + sm_sum[128 + row] * f1;
            }
            const int c0 = two || i == 0 ? 0 : D / 2, c1 = two || i == 1 ? D : D / 2;
            const int which = it.t0 == 0 ? 1 : 0, part_row = two ? i * 128 + row : row;
            const int64_t slot = static_cast<int64_t>(which) * G + blockIdx.x;
            float *part = p.ws + (slot * 256 + part_row) * PartRow<D>::FLOATS;
            const float inv = 1.f / L;
            // a pipeline without a key tile has nothing there
            const bool has0 = two ? i == 0 : todo > 0, has1 = two ? i == 1 : todo > 1;
#pragma unroll 2
            for (int c = c0; c < c1; c += 16) {
                float v[16], u[16];
                if (has0) tmem_ld16(tmem + TM_O + lanes + c, reinterpret_cast<uint32_t *>(v));
                if (has1) tmem_ld16(tmem + TM_O + 128 + lanes + c, reinterpret_cast<uint32_t *>(u));
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = (has0 ? v[e] * f0 : 0.f) + (has1 ? u[e] * f1 : 0.f);
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
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<float4 *>(part + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
                __syncwarp();
            }
            tc_fence_before();
            if (mine && (two || i == 0)) {
                if (whole) {
                    store_lse(p, out_token, head, M, L);
                } else {
                    *reinterpret_cast<float2 *>(part + D) = make_float2(M, L);
                }
            }
            arrive(o_empty);
            arrive(o_empty + 8);
            arrive(it_empty + 8 * (k % ITEMS));
        }

        // The parts of split items, joined when the CTA's own tiles are done: a CTA says that its
        // parts are there for both its items before it waits for either, so that no two items
        // wait for one another (all CTAs are resident: one per SM, no more than SMs). Each CTA
        // joins its share of the item's rows, of all parts, which it copies into the ring's memory.
        if (alive && (pend[0].parts | pend[1].parts) != 0) {
            arrive(parts_done);
            if (warp < 2) {  // a warp for each
                const Pending it = pend[warp];
                if (it.parts != 0) {
                    // a count of the item's parts, and one, never reset, of how often all have come
                    uint32_t *counter = p.counters + it.a, *times = p.times + it.a;
                    if (wait(parts_done, 0) && lane == 0) {
                        const uint32_t before = *static_cast<volatile uint32_t *>(times);
                        uint32_t come;
                        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(come) : "l"(counter) : "memory");
                        if (come == static_cast<uint32_t>(it.parts - 1)) {
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
            // This CTA's rows of an item: [first, first + n), and where they are in shared memory, part
            // after part. Those of both items at once, where there is room.
            auto share = [&](const Pending &it, int &first, int &n) {
                const int rows = it.n * p.unit_heads, per = it.parts > 0 ? (rows + it.parts - 1) / it.parts : 0;
                first = (static_cast<int>(blockIdx.x) - it.a) * per;
                n = it.parts == 0 || first >= rows ? 0 : (rows - first < per ? rows - first : per);
            };
            int first0, n0, first1, n1;
            share(pend[0], first0, n0);
            share(pend[1], first1, n1);
            const int size0 = n0 * pend[0].parts * PartRow<D>::BYTES, size1 = n1 * pend[1].parts * PartRow<D>::BYTES;
            uint32_t n_joined = 0;
            const bool at_once = size0 + size1 <= (2 + NST) * Sh::TILE_BYTES;
#pragma unroll 1
            for (int round = 0; round < (at_once ? 1 : 2) && alive; ++round) {
#pragma unroll 1
                for (int which = at_once ? 0 : round; which < (at_once ? 2 : round + 1); ++which) {
                    const Pending it = pend[which];
                    const int first = which == 0 ? first0 : first1, n = which == 0 ? n0 : n1, tile_rows = p.tokens * p.unit_heads;
                    if (it.parts == 0 || !wait(join_go + 8 * which, 0)) continue;
                    // A row for each warp, of every part, or a part.
                    const uint32_t mem = sm_q + (at_once && which == 1 ? size0 : 0) + lane * 16;
                    const bool few = n < 8;
#pragma unroll 1
                    for (int part = few ? warp : 0; part < it.parts; part += few ? 8 : 1) {
                        // slot 1 for the CTA in which the item begins, 0 for the others
                        const int64_t slot = static_cast<int64_t>(part == 0 ? G : 0) + it.a + part;
                        const float *rows = p.ws + slot * 256 * PartRow<D>::FLOATS + lane * 4;
                        const uint32_t to = mem + part * n * PartRow<D>::BYTES;
#pragma unroll 2
                        for (int r = few ? 0 : warp; r < n; r += few ? 1 : 8) {
                            const int of = first + r, part_row = of < tile_rows ? of : 128 + of - tile_rows;
                            const float *from = rows + part_row * PartRow<D>::FLOATS;
                            if (lane < PartRow<D>::BYTES / 16) copy16(to + r * PartRow<D>::BYTES, from);
                            if (lane + 32 < PartRow<D>::BYTES / 16) copy16(to + r * PartRow<D>::BYTES + 512, from + 128);
                        }
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                arrive(joined);
                if (!alive || !wait(joined, n_joined++ & 1)) break;
#pragma unroll 1
                for (int which = at_once ? 0 : round; which < (at_once ? 2 : round + 1); ++which) {
                    const Pending it = pend[which];
                    const int first = which == 0 ? first0 : first1, n = which == 0 ? n0 : n1;
                    if (it.parts == 0) continue;
                    float *mem = reinterpret_cast<float *>(base + (at_once && which == 1 ? size0 : 0));
                    const int step = n * PartRow<D>::FLOATS;    // from part to part
                    // A row's weights of its parts, in place of their maxima: by a lane for each part,
                    // or, where there are many rows, by a lane for each row.
                    const bool many = n > 32;
                    const int by = many ? 1 : 32, q0 = many ? 0 : lane;
#pragma unroll 1
                    for (int r = many ? threadIdx.x : warp; r < n; r += many ? 256 : 8) {
                        float *at = mem + r * PartRow<D>::FLOATS + D;
                        float M = -INFINITY, L = 0.f;
#pragma unroll 4
                        for (int q = q0; q < it.parts; q += by) M = fmaxf(M, at[q * step]);
                        if (!many)
                            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
                        for (int q = q0; q < it.parts; q += by) L += at[q * step + 1] * ex2((at[q * step] - ref) * sl);
                        if (!many)
                            for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
                        const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll 4
                        for (int q = q0; q < it.parts; q += by) at[q * step] = ex2((at[q * step] - ref) * sl) * inv;
                        const int tok = (first + r) / p.unit_heads, in_group = it.h0 + first + r - tok * p.unit_heads;
                        if (q0 == 0 && in_group < p.group)
                            store_lse(p, static_cast<int64_t>(it.row0) + tok, it.kvh * p.group + in_group, M, L);
                    }
                    __syncwarp();
                    arrive(joined);
                    if (!wait(joined, n_joined++ & 1)) break;
                    // Then four columns of a row by a lane, several rows at once where there are many.
                    constexpr int SIDE = 128 / D;
                    const JoinRows<D> rows{p, it, mem, first, n, warp * SIDE + lane / (D / 4), (lane & (D / 4 - 1)) * 4};
                    if (n > 8 * SIDE)
                        rows.template run<4>();
                    else
                        rows.template run<1>();
                    __syncwarp();
                }
                if (at_once) break;
                arrive(joined);                                // the memory is free again
                if (!wait(joined, n_joined++ & 1)) break;
            }
        }
    } else {
        // the four single warps
        fewer_registers<SINGLE_REGS>();
        // The key tiles of an item, of K (kind 0), V (1) or both, into their rings: `c` are before them.
        auto load_tiles = [&](const Item &it, int from, int to, uint32_t &c) {
            const int box = KEYS < (1 << p.b.page_shift) ? KEYS : (1 << p.b.page_shift), boxes = KEYS / box;
            const int len = it.len, todo = it.todo;
            const int32_t *table = p.b.page_table + it.seq * p.b.table_row;
            const int pages = (len + (1 << p.b.page_shift) - 1) >> p.b.page_shift;
            int cached0 = INT32_MAX, ids = -1;         // page ids, one per lane
            for (int j = 0; j < todo; ++j, ++c) {
                const int kt = it.tile(j), key0 = kt * KEYS, ext = extent(len, kt);
                const int n_box = (ext + box - 1) / box, page0 = key0 >> p.b.page_shift;
                if (page0 < cached0) {                 // this tile's pages, and those before it
                    cached0 = page0 + boxes > 32 ? page0 + boxes - 32 : 0;
                    // a page that no row sees may be another sequence's by now, or nobody's
                    const int64_t first = static_cast<int64_t>(cached0 + lane) << p.b.page_shift;
                    const bool seen = cached0 + lane < pages &&
                                      (p.window == 0 || first + (int64_t(1) << p.b.page_shift) > it.lo || first < p.sinks);
                    ids = seen ? table[cached0 + lane] : -1;
                    if (seen && (ids < 0 || ids >= p.b.num_pages)) {
                        atomicCAS(p.b.status, 0, UB_ERR_ARG);
                        ids = -1;                      // outside the tensor: filled with zeros
                    }
                }
                for (int kind = from; kind < to; ++kind) {
                    const uint32_t stages = kind == 0 ? KST : VST, lap = c / stages;
                    const uint32_t st = c - lap * stages + (kind == 0 ? 0 : KST), bar = kv_full + 8 * st;
                    if (lap > 0 && !wait(kv_empty + 8 * st, (lap - 1) & 1)) return;
                    if (lane == 0) mbar_arrive_expect_tx(bar, n_box * HALVES * box * 128);
                    __syncwarp();
                    const int bx = lane / HALVES, hf = lane - bx * HALVES;
                    const int page = __shfl_sync(0xffffffffu, ids, (page0 - cached0 + bx) & 31);
                    if (bx < n_box)
                        tma_load_4d(sm_kv + st * Sh::TILE_BYTES + hf * Sh::HALF_BYTES + bx * box * 128,
                                    kind == 0 ? &p.tmK : &p.tmV, bar, hf * 64,
                                    boxes > 1 ? 0 : key0 & ((1 << p.b.page_shift) - 1), it.kvh, page);
                    __syncwarp();
                    if (lane == 0) issued[kind] = c + 1;
                }
            }
        };
        if (warp == 8) {
            // -------------------------------------------------------- loads
            uint32_t c = 0;
            for (uint32_t k = 0; there(k); ++k) {
                const Item &it = items[k % ITEMS];
                const bool two = it.ntok > p.tokens;
                if (k > 0 && !wait(q_empty, (k - 1) & 1)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, (two ? 2 : 1) * HALVES * p.tokens * p.unit_heads * 128);
                    for (int t = 0; t < (two ? 2 : 1); ++t)
                        for (int hf = 0; hf < HALVES; ++hf)
                            tma_load_3d(sm_q + t * Sh::TILE_BYTES + hf * Sh::HALF_BYTES, &p.tmQ, q_full, hf * 64,
                                        it.kvh * p.group + it.h0, it.row0 + t * p.tokens);
                }
                __syncwarp();
                load_tiles(it, 0, Sh::TWO_LOADERS ? 1 : 2, c);
                if (!alive) break;
                arrive(it_empty + 8 * (k % ITEMS));
            }
        } else if (warp < 11) {
            // -------------------------------------------------------- MMA issue
            // Step by step: O += P V of a tile, then S of the pipeline's next one. The pipelines take
            // turns, so that one's MMAs run during the other's softmax: without turns the two fall
            // into step and leave the tensor core and the arithmetic idle by turns (32 sequences of 64
            // drafts over 8192 keys, 4 query heads to a key head: 272 against 231 us, heads of 64: 224
            // against 173, when this was chosen). But a turn does not wait for keys that have not landed.
            const int i = warp - 9;
            uint32_t c = 0, n_p = 0, step = 0;
            const uint32_t ts = tmem + TM_S + i * 128, to = tmem + TM_O + i * 128;
            const uint64_t k_desc = smem_desc_sw128(sm_kv), v_desc = smem_desc_v(sm_kv, Sh::HALF_BYTES);
            constexpr uint32_t o_idesc = attn_idesc(D, true);
            // A pipeline skips the other's key tiles, and the ring may turn meanwhile: a barrier's
            // parity tells two turns apart only once the loads of this one have been issued.
            auto poll = [&](const volatile uint32_t *word, uint32_t least) {  // until *word >= least
                bool come = __all_sync(0xffffffffu, static_cast<int32_t>(*word - least) >= 0) != 0;
                if (come) return true;
                WaitClock clk;
                for (uint32_t n = 1; !come; ++n) {
                    come = __all_sync(0xffffffffu, static_cast<int32_t>(*word - least) >= 0) != 0;
                    if ((n & 15u) == 0 && !come && !__all_sync(0xffffffffu, clk.ok(wc))) return alive = false;
                }
                return true;
            };
            auto wait_k = [&](uint32_t at) { return poll(issued, at + 1) && wait(kv_full + 8 * (at % KST), (at / KST) & 1); };
            auto wait_v = [&](uint32_t at) {
                return poll(issued + 1, at + 1) && wait(kv_full + 8 * (KST + at % VST), (at / VST) & 1);
            };
            auto landed = [&](uint32_t at) {           // K
                return __all_sync(0xffffffffu, static_cast<int32_t>(*issued - at) > 0 &&
                                                   mbar_test(kv_full + 8 * (at % KST), (at / KST) & 1)) != 0;
            };
            auto pass = [&](uint32_t step) {
                if (lane == 0) turn[i] = step;
                __syncwarp();
            };
            for (uint32_t k = 0; there(k); ++k) {
                // Broadcast from lane 0, so that the compiler knows them to be the same in every lane:
                // descriptors then stay in uniform registers, and an issue costs less than the MMA.
                auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
                const Item &it = items[k % ITEMS];
                const bool two = same(it.ntok) > p.tokens;
                const int todo = same(it.todo), len = same(it.len), t0 = same(it.t0), far = same(it.far), gap = same(it.near) - far;
                const int stride = two ? 1 : 2, j0 = two ? 0 : i;
                const uint64_t q_desc = smem_desc_sw128(sm_q + (two ? i * Sh::TILE_BYTES : 0));
                auto tile_of = [&](int j) { const int t = t0 + todo - 1 - j; return t < far ? t : t + gap; };
                if (!wait(q_full, k & 1)) break;
                // O of the last item has been read before this one's first product.
                if (j0 >= todo) {
                    arrive(q_empty);
                    if (k > 0 && !wait(o_empty + 8 * i, (k - 1) & 1)) break;
                }
                const int steps = two ? todo : (todo + 1) / 2;  // of either pipeline
#pragma unroll 1
                for (int n = -1; n < steps; ++n) {
                    const int j = j0 + n * stride, next = j + stride;
                    bool passed = n < 0;               // the other pipeline may have its turn
                    if (n >= 0) ++step;
                    if (n >= 0 && j < todo) {
                        const uint32_t st = KST + (c + j) % VST, freed = kv_empty + 8 * st;
                        const uint64_t v = v_desc + st * (Sh::TILE_BYTES / 16);
                        const int kt = tile_of(j), ext = extent(len, kt), valid = len - kt * KEYS;
                        if (k > 0 && n == 0 && !wait(o_empty + 8 * i, (k - 1) & 1)) break;
                        if (!wait_v(c + j)) break;
                        if (ext > valid) {
                            // What is past the sequence's end has the weight zero, and may hold anything:
                            // zeros take its place (two q tiles: by both issuers, whoever comes first).
                            const uint32_t mem = sm_kv + st * Sh::TILE_BYTES;
                            for (int u = lane; u < (ext - valid) * (D / 8); u += 32) {
                                const int r = valid + u / (D / 8), ch = u % (D / 8);
                                st_shared_v4(mem + (ch / 8) * Sh::HALF_BYTES + r * 128 + (ch % 8) * 16, 0u, 0u, 0u, 0u);
                            }
                            fence_proxy_async_shared();
                            __syncwarp();
                        }
                        if (!poll(turn + (1 - i), step - 1 + i)) break;
                        if (!wait(p_full + 8 * i, n_p & 1)) break;
                        ++n_p;
                        tc_fence_after();
                        if (elect_one()) {
                            if (ext == KEYS) {
#pragma unroll
                                for (int s = 0; s < KEYS / 16; ++s) umma_ts(to, ts + s * 8, v + s * 128, o_idesc, n > 0 || s > 0);
                            } else {  // the sequence's last keys
                                for (int s = 0; s < ext / 16; ++s) umma_ts(to, ts + s * 8, v + s * 128, o_idesc, n > 0 || s > 0);
                            }
                            umma_commit(freed);
                            if (!two) umma_commit(freed);
                            if (next >= todo) umma_commit(o_full + 8 * i);
                        }
                        __syncwarp();
                    }
                    if (next >= todo || !landed(c + next)) {
                        if (!passed) pass(step);
                        passed = true;
                        if (next >= todo) continue;
                        if (!wait_k(c + next)) break;
                    }
                    {   // S of key tile `next`, which has landed
                        const uint32_t st = (c + next) % KST, freed = kv_empty + 8 * st;
                        const uint32_t s_idesc = attn_idesc(extent(len, tile_of(next)), false);
                        const uint64_t kk = k_desc + st * (Sh::TILE_BYTES / 16);
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int s = 0; s < D / 16; ++s) {
                                const int o = (s / 4) * (Sh::HALF_BYTES / 16) + (s % 4) * 2;
                                umma_ss(ts, q_desc + o, kk + o, s_idesc, s > 0);
                            }
                            umma_commit(s_full + 8 * i);
                            umma_commit(freed);
                            if (!two) umma_commit(freed);
                            if (next + stride >= todo) umma_commit(q_empty);
                        }
                        __syncwarp();
                    }
                    if (!passed) pass(step);
                }
                if (!alive) break;
                c += todo;
                arrive(it_empty + 8 * (k % ITEMS));
            }
            // everything issued has completed before TMEM goes back
            if (elect_one()) {
                umma_commit(drain + 8 * i);
                mbar_wait_drain(drain + 8 * i, 0, p.timeout_ns);
            }
            __syncwarp();
        } else {
            // -------------------------------------------------------- schedule
            Walk w(p);
            if (p.many_units)
                begin<int64_t>(w, lane, blockIdx.x, gridDim.x);
            else
                begin<int>(w, lane, blockIdx.x, gridDim.x);
            auto publish = [&](uint32_t k) {
                if (k >= ITEMS && !wait(it_empty + 8 * (k % ITEMS), (k / ITEMS - 1) & 1)) return;
                if (lane == 0) {
                    Item it;
                    it.seq = -1;
                    if (w.more()) {
                        const int first = w.first_token(), unit = w.unit(), kvh = p.blocks == 1 ? unit : unit / p.blocks;
                        it = Item{w.s, w.q.start + first, w.tokens(), first, kvh,
                                  (unit - kvh * p.blocks) * p.unit_heads, w.q.len, w.q.text, w.q.lo, w.q.near, w.q.far,
                                  w.t0, w.todo(), w.whole() ? 1 : 0};
                        if (!it.whole) {
                            const int64_t item0 = w.x - w.off;
                            const int a = w.split.owner(item0);
                            pend[w.t0 == 0 ? 1 : 0] =
                                Pending{it.row0, it.ntok, it.kvh, it.h0, a, w.split.owner(item0 + w.q.span() - w.q.per) - a + 1};
                        }
                    }
                    items[k % ITEMS] = it;
                }
                arrive(it_full + 8 * (k % ITEMS));
            };
            uint32_t c = 0;
            publish(0);
            for (uint32_t k = 0; w.more() && alive; ++k) {
                // read again: it takes no registers beside the loads
                if (Sh::TWO_LOADERS && k > 0) w.q = seq_of(p, w.s, w.height);
                w.next();
                publish(k + 1);                        // before this one's loads may have to wait
                if constexpr (Sh::TWO_LOADERS)
                    if (alive) load_tiles(items[k % ITEMS], 1, 2, c);
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
