// Causal attention of packed prompts, or of chunks of prompts over the paged cache.
//
//   O_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale * q_i . k_j - m_i),  j <= pos_i
//
// in one pass over the keys: a running maximum m and sum l per row, and O rescaled by
// exp(m_old - m_new) when the maximum grows. The rescaling is put off while the maximum
// has grown by less than 2^8: the weights then stay below 2^8, which neither BF16 nor the
// fp32 sums mind, and the division by l at the end cancels the choice of m.
//
// A work item is 256 rows, two q tiles of 128: consecutive tokens of one sequence, and,
// where query heads share a key/value head, a power of two of those heads per token (row =
// token * pack + head). Where items of 128 rows, one q tile, are no more than the CTAs, they
// are the items (882 tokens, 12 heads: 18 against 20 us; in calls of more items the second
// tile runs in the first one's pauses and saves reading keys and values twice). Per 128 keys and
// q tile the tensor core computes S = Q K^T (128 x 128, both operands from shared memory) and
// O += P V (P from TMEM, V read MN-major); the softmax in between is per TMEM lane, one thread
// per row, without shuffles.
//
// WINDOW: a row sees the keys j > pos - window and j < sinks. An item then has the key tiles of
// its rows' windows and of the sinks only, whatever its position: items are of one length, and
// the schedule orders them by the keys that they reach all the same.
//
// Roles (16 warps, one CTA per SM, persistent over items):
//   warps 0-3, 4-7   softmax of q tile 0 and 1: S from TMEM, P back into the columns of S
//   warps 8-11       epilogue: O / l to memory, while the next item's first tiles run
//   warp 12          loads (TMA): Q, then K and V tiles in a ring
//   warps 13, 14     MMA issue for q tile 0 and 1: S, then per key tile O and the next S
//   warp 15          schedule: the CTA's items, longest first over the whole call; and
//                    zeroes the rows of V past a sequence's end in its last tile (their
//                    weights are zero, their values may be anything)
// The two q tiles alternate, so that the tensor core works on one while the softmax of
// the other runs. TMEM: S_0, S_1 (128 columns each), O_0, O_1.
//
// Only the keys that a q tile needs are multiplied: the last key tile of a q tile is cut
// to 16 keys (N of the first product, K of the second).
//
// What bounds it (GB300): a step of 128 keys for both q tiles is 2048 cycles of MMAs (heads
// of 128) against 2420 measured in a long sequence (2200 for one q tile alone); the difference
// is the chain S -> softmax (1150 cycles, 870 of them its instructions; exp2 runs at 4 cycles
// per warp and SM quarter) -> P V -> next S, which the other tile's MMAs cover only in part.
// TMEM holds no third tile. One sequence of 16384 tokens, 8 query heads, 2 key/value heads:
// 329-342 us, 1.61-1.67 PFLOP/s; tensor pipe active in 80 % of the cycles. Shorter prompts: the first
// item is known 1.6 us after the grid ahead has finished, and the call ends with its longest
// item (8037 tokens in four sequences, 8 heads each way: 42 us, of which the 24 key tiles of
// the longest item take 36). Heads of 64: half the MMAs, the same softmax: 2440 cycles a step.
// Windows: one sequence of 8160 tokens, 8 heads of 128, window 1024 and 4 sinks (11 key tiles an
// item): 42 us. A CTA takes 7 us to its first scores, 15 us for an item's steps (1.2-1.4 each, the
// masked ones up to 2) and 4-5 from one item's last weights to the next one's first scores: Q has
// one place in shared memory, and the code of an item's ends runs cold.
#include <cuda_bf16.h>
#include <limits.h>

#include "ub_attn.h"
#include "ub_attn_mma.cuh"
#include "ub_device.cuh"
#include "ub_internal.h"

namespace ubk {
namespace {

constexpr int PR_THREADS = 512;
constexpr int ITEMS = 4;                 // schedule ring
constexpr int DONE = 16;                 // barriers of the ring's releases: more than can be unseen
// Registers per thread by role; their sum is what the block is launched with (512 x 128).
constexpr int SOFTMAX_REGS = 176, EPILOGUE_REGS = 88, SINGLE_REGS = 72;
static_assert(2 * SOFTMAX_REGS + EPILOGUE_REGS + SINGLE_REGS == 4 * 128, "register split");
constexpr int TM_S = 0, TM_O = 256;      // TMEM columns: S_i at 128 i, O_i at 256 + 128 i
// Heads of 128: the weights of the first PART steps of 16 keys are handed over while the rest
// are computed (16384 tokens: 337 against 350 us; heads of 64, whose products are half as
// long, lose by it: 78 against 75 us for chunks over a cache).
constexpr int PART = 4;
constexpr float RESCALE_LOG2 = 8.f;      // growth of the maximum (log2) that is put off

template <int D>
struct PromptShape {
    static constexpr int TILE_BYTES = PROMPT_KEYS * D * 2;
    static constexpr int HALF_BYTES = PROMPT_KEYS * 128;  // 64 columns of a tile
    static constexpr int STAGES = D == 128 ? 5 : 10;
    static constexpr int SMEM = (2 + STAGES) * TILE_BYTES + 2048 + 1024;
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(STAGES < DONE, "an unseen release per ring position at most");
};

// One work item.
struct Item {
    int row0;    // first token (row of q); -1: no more items
    int ntok;    // tokens
    int off;     // position of the first token
    int len;     // keys of the sequence
    int src;     // first key row (packed) or sequence (paged)
    int unit;
    int j0, j1;  // its key tiles, of those in sight (a piece of a split item: a part of them)
    int slot;    // first workspace slot of a split item; -1: not split
    int piece, pieces;
    int n;       // key tiles of the whole item
};
constexpr Item kNoItem = {-1, 0, 0, 0, 0, 0, 0, 0, -1, 0, 1, 0};
// First key tile of piece i of an item of n tiles.
__device__ __forceinline__ int piece_begin(int n, int i, int pieces)
{
    const int base = n / pieces, rem = n - base * pieces;
    return i * base + (i < rem ? i : rem);
}

// The keys that the rows of an item see together: all up to the last row, or (WINDOW) from the
// window of the first row on, and the first `sinks`. Key tiles are counted along those that hold
// such a key.
template <bool WINDOW>
struct Sight {
    int lo;    // first key of the first row's window
    int near;  // its key tile
    int far;   // key tiles before it that hold sinks
    __device__ __forceinline__ int gap() const { return WINDOW ? near - far : 0; }
    // The key tile that is the j-th in sight.
    __device__ __forceinline__ int tile(int j) const { return WINDOW && j >= far ? j + (near - far) : j; }
};
template <bool WINDOW>
__device__ __forceinline__ Sight<WINDOW> sight(const PromptParams &p, int off)
{
    Sight<WINDOW> s{0, 0, 0};
    if (WINDOW) {
        s.lo = off >= p.window ? off - p.window + 1 : 0;
        s.near = s.lo / PROMPT_KEYS;
        const int sunk = (p.sinks + PROMPT_KEYS - 1) / PROMPT_KEYS;
        s.far = sunk < s.near ? sunk : s.near;
    }
    return s;
}

// The lowest n bits.
__device__ __forceinline__ uint32_t bits_below(int n)
{
    return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

struct Range2 {
    int lim[2];  // keys that q tile i reaches
    int n[2];    // its key tiles, of those of the item or piece
    int tok[2];  // its tokens
    int nmax;
    int limmax;
};
// gap: key tiles out of sight before the last ones
__device__ __forceinline__ Range2 ranges(const Item &it, int tpt, int gap)
{
    Range2 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int tok = it.ntok - i * tpt;
        tok = tok < 0 ? 0 : (tok > tpt ? tpt : tok);
        int lim = tok > 0 ? it.off + i * tpt + tok : 0;
        lim = lim < 0 ? 0 : (lim > it.len ? it.len : lim);
        r.tok[i] = tok;
        r.lim[i] = lim;
        const int n = (lim + PROMPT_KEYS - 1) / PROMPT_KEYS - (lim > 0 ? gap : 0), most = it.j1 - it.j0;
        r.n[i] = n - it.j0 < 0 ? 0 : (n - it.j0 > most ? most : n - it.j0);
    }
    r.nmax = r.n[0] > r.n[1] ? r.n[0] : r.n[1];
    r.limmax = r.lim[0] > r.lim[1] ? r.lim[0] : r.lim[1];
    return r;
}
// What the schedule warp publishes: ready for use, as code that runs once per item is cold, and all
// roles would run it at the same time (four sequences in windows, as below: 37.5 to 35.3 us; one
// sequence of 16384 tokens 302 to 298).
template <bool WINDOW>
struct Work : Item {
    Sight<WINDOW> in;
    Range2 r;
};
// The same values, known to be the same in every lane.
__device__ __forceinline__ Range2 uniform(Range2 r)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r.lim[i] = __shfl_sync(0xffffffffu, r.lim[i], 0);
        r.n[i] = __shfl_sync(0xffffffffu, r.n[i], 0);
    }
    r.nmax = r.n[0] > r.n[1] ? r.n[0] : r.n[1];
    return r;
}
// ---------------------------------------------------------------- schedule

struct SeqInfo {
    int start, n, len, off;
};
__device__ __forceinline__ SeqInfo seq_info(const PromptParams &p, int s)
{
    SeqInfo q;
    int a = p.b.seq_starts[s], z = p.b.seq_starts[s + 1];
    a = a < 0 ? 0 : (a > p.T ? p.T : a);
    z = z < a ? a : (z > p.T ? p.T : z);
    q.start = a;
    q.n = z - a;
    if (p.paged) {
        const int64_t most = static_cast<int64_t>(p.b.table_width) << p.b.page_shift;
        const int len = p.b.kv_lens[s];
        q.len = len < 0 ? 0 : (len > most ? static_cast<int>(most) : len);
    } else {
        q.len = q.n;
    }
    q.off = q.len - q.n;
    return q;
}
// Of the `nt` items (token tiles of 1 << shift tokens) of a sequence, those that reach at
// least `c` key tiles.
__device__ __forceinline__ int reaching(int nt, int len, int off, int c, int shift)
{
    const int x = (c - 1) * PROMPT_KEYS;
    const uint32_t t = x < off ? 0u : (static_cast<uint32_t>(x) - static_cast<uint32_t>(off)) >> shift;
    const int n = nt - (t < static_cast<uint32_t>(nt) ? static_cast<int>(t) : nt);
    return c <= 0 ? nt : (len <= x ? 0 : n);
}
__device__ __forceinline__ int items_from(const SeqInfo &q, int c, int shift)
{
    return reaching((q.n + (1 << shift) - 1) >> shift, q.len, q.off, c, shift);
}

// The work items of a call in the order "most key tiles first" (ties: by sequence, then by
// tile), without a list: one warp counts the items of at least c key tiles over all
// sequences, 32 levels c at once (one per lane, the sequences broadcast one by one), and so
// finds the level of a rank. Up to 32 sequences stay in registers, one per lane; beyond, they
// are read again for every count (from L1).
struct Schedule {
    const PromptParams &p;
    int lane, shift, n_seqs, cmax, tiles;
    SeqInfo own;

    __device__ __forceinline__ SeqInfo info(int i0) const
    {
        if (i0 == 0) return own;
        return i0 + lane < n_seqs ? seq_info(p, i0 + lane) : SeqInfo{0, 0, 0, 0};
    }
    __device__ __forceinline__ void measure()  // cmax, tiles
    {
        int most = 0, sum = 0;
        for (int i0 = 0; i0 < n_seqs; i0 += 32) {
            const SeqInfo q = info(i0);
            const int n = q.n > 0 ? static_cast<int>((static_cast<uint32_t>(q.len) + PROMPT_KEYS - 1) / PROMPT_KEYS) : 0;
            most = n > most ? n : most;
            sum += items_from(q, 0, shift);
        }
        cmax = __reduce_max_sync(0xffffffffu, most);
        tiles = __reduce_add_sync(0xffffffffu, sum);
    }
    // Key tiles of all items together, about (each sequence's run evenly from its first item's
    // to its last item's).
    __device__ __forceinline__ float work() const
    {
        float sum = 0.f;
        for (int i0 = 0; i0 < n_seqs; i0 += 32) {
            const SeqInfo q = info(i0);
            const int first = q.off + (1 << shift) < q.len ? q.off + (1 << shift) : q.len;
            sum += 0.5f * items_from(q, 0, shift) * ((first > 0 ? first : 0) + q.len) * (1.f / PROMPT_KEYS);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        return sum;
    }
    // Items of at least c key tiles, for each lane's own c. (One copy of the code: it runs cold,
    // before anything else of the call can start.)
    __device__ __noinline__ int counts(int c) const
    {
        int sum = 0;
        c = c <= cmax ? c : cmax + 1;  // no item has more; the keys of c tiles stay within 32 bits
        for (int i0 = 0; i0 < n_seqs; i0 += 32) {
            const SeqInfo q = info(i0);
            const int m = n_seqs - i0 < 32 ? n_seqs - i0 : 32;
            const int nt = items_from(q, 0, shift);
#pragma unroll 4
            for (int i = 0; i < m; ++i)
                sum += reaching(__shfl_sync(0xffffffffu, nt, i), __shfl_sync(0xffffffffu, q.len, i),
                                __shfl_sync(0xffffffffu, q.off, i), c, shift);
        }
        return sum;
    }
    // *level: the key tiles of the item
    __device__ __noinline__ Item at(int g, int *level) const
    {
        // The largest level lo with count(lo) > g, in strides that fall to 1; the last pass
        // covers lo + 1 too, so that 31 levels at most may be left for it: level 31 takes two.
        int lo = 0, stride = cmax <= 30 ? 1 : (cmax <= 62 ? 2 : (cmax + 32) / 32), k, n;
        for (;; stride = stride <= 31 ? 1 : (stride + 30) / 31) {
            n = counts(lo + lane * stride);
            k = 31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, n > g) | 1u));
            lo += k * stride;
            if (stride == 1) break;
        }
        int r = g - __shfl_sync(0xffffffffu, n, k + 1);
        *level = lo;
        Item it = kNoItem;
        for (int i0 = 0; i0 < n_seqs; i0 += 32) {
            const SeqInfo q = info(i0);
            const int from = items_from(q, lo, shift), mine = from - items_from(q, lo + 1, shift);
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, upto > r);
            if (past != 0u) {
                const int l = __ffs(static_cast<int>(past)) - 1;
                const int tile = items_from(q, 0, shift) - from + (r - (upto - mine));
                const int t0 = tile << shift;
                it.row0 = __shfl_sync(0xffffffffu, q.start + t0, l);
                it.ntok = __shfl_sync(0xffffffffu, q.n - t0 < (1 << shift) ? q.n - t0 : 1 << shift, l);
                it.off = __shfl_sync(0xffffffffu, q.off + t0, l);
                it.len = __shfl_sync(0xffffffffu, q.len, l);
                it.src = __shfl_sync(0xffffffffu, p.paged ? i0 + lane : q.start, l);
                return it;
            }
            r -= __shfl_sync(0xffffffffu, upto, 31);
        }
        return it;
    }
};

// Few rows over many keys (a call of fewer items than CTAs): items of more than `limit` key
// tiles are cut into `pieces` pieces each, as even as the number of CTAs allows, which is one
// piece or whole item for each: the pieces' CTAs then join their item together. With more
// items than CTAs nothing is split (windows: the last round may be, see plan_of), nor where no item
// has more than MIN_SPLIT key tiles: the join takes about 6 us, a key tile 1.1 (four chunks of 16 tokens, 12 query and 4 key/value
// heads of 128, split against whole: 1280 keys 21.2 and 18.2 us, 1536 keys 20.3 and 20.5, 2048
// keys 21.9 and 25.1, 4096 keys 28.4 and 44.0).
struct Plan {
    int pieces;          // 1: nothing is split
    uint32_t split_end;  // ranks [0, split_end): pieces of the split items, item by item
    uint32_t total;      // ... then the whole items
    int n_split;         // token tiles (of each unit) that are split
    uint32_t whole;      // not 0: ranks [0, whole) are whole items, the pieces of the rest follow
};
constexpr int MIN_SPLIT = PROMPT_WHOLE_KEYS / PROMPT_KEYS;
// Key tiles of a piece, at least, where the CTAs would allow shorter ones. It matters to a few
// rows over keys that just pay for a split; 16 tokens, 8 query heads on one of 128, pieces of at
// least 3, 5 and 8 tiles: 2000 keys 13.8, 14.5 and 19.7 us, 3000 keys 13.8, 16.1 and 19.8, 6000
// keys 15.4, 17.0 and 20.1; 300 and 1 tokens over 1409 and 3000 keys, heads of 64: 15.8, 15.9 and
// 18.1; 20000 keys, 8 heads each way: 27.0 with any of them.
constexpr int MIN_PIECE = 5;
// With a window the key tiles of an item are at most `cap`, whatever it reaches.
template <bool WINDOW>
__device__ Plan plan_of(const Schedule &sc, int units, int ctas, int slots, int cap)
{
    Plan pl{1, 0u, static_cast<uint32_t>(sc.tiles) * units, 0, 0u};
    const int cmax = WINDOW && sc.cmax > cap ? cap : sc.cmax;
    if (cmax <= MIN_SPLIT) return pl;
    if (pl.total >= static_cast<uint32_t>(ctas)) {
        // Windows make items of one length, of which one more than fill the CTAs takes as long as
        // twice as many: the items of an incomplete last round are split where two CTAs or more can
        // share each of them and the longest of them reaches more than MIN_SPLIT key tiles, in sight or
        // not (of one or two rounds: of more rounds the last is a small part).
        const uint32_t rounds = pl.total / ctas, left = pl.total - rounds * ctas;
        if (!WINDOW || rounds > 2u || left == 0u) return pl;
        uint32_t pieces = static_cast<uint32_t>(ctas) / left;
        if (pieces * MIN_PIECE > static_cast<uint32_t>(cmax)) pieces = cmax / MIN_PIECE;
        if (pieces * left > static_cast<uint32_t>(slots)) pieces = slots / left;
        if (pieces < 2u || static_cast<uint32_t>(sc.counts(MIN_SPLIT + 1)) * units <= pl.total - left) return pl;
        pl.pieces = static_cast<int>(pieces);
        pl.whole = pl.total - left;
        pl.total = pl.whole + left * pieces;
        return pl;
    }
    // 32 limits at once, from an even share up to the longest item, closer together near the
    // first; of those that give no more pieces than there are CTAs and slots, the one of the
    // shortest longest piece.
    float work = sc.work();
    if (WINDOW) work = fminf(work, static_cast<float>(sc.tiles) * cap);
    int limit = static_cast<int>(work * units / ctas) + 1;
    limit = limit < MIN_PIECE ? MIN_PIECE : limit;
    limit += static_cast<int>(static_cast<float>(cmax - limit) * static_cast<float>(sc.lane * sc.lane) * (1.f / 1024.f));
    const int n = sc.counts(limit + 1), pieces = (cmax + limit - 1) / limit;
    const float split = static_cast<float>(n) * units * pieces;
    const bool fits = limit < cmax && split <= slots && split + static_cast<float>(sc.tiles - n) * units <= ctas;
    const int longest = (cmax + pieces - 1) / pieces;
    const int best = __reduce_min_sync(0xffffffffu, fits ? longest : INT_MAX);
    if (best == INT_MAX) return pl;
    const int pick = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, fits && longest == best))) - 1;
    pl.pieces = __shfl_sync(0xffffffffu, pieces, pick);
    pl.n_split = __shfl_sync(0xffffffffu, n, pick);
    pl.split_end = static_cast<uint32_t>(pl.n_split * units * pl.pieces);
    pl.total += static_cast<uint32_t>(pl.n_split * units * (pl.pieces - 1));
    return pl;
}
template <bool WINDOW>
__device__ Item item_of(const Schedule &sc, const Plan &pl, int units, uint32_t g)
{
    uint32_t rank = g;   // among the items; fewer than 2^32: T * heads rows
    int piece = 0, pieces = 1, slot = -1;
    if (WINDOW && pl.whole > 0u) {
        if (g >= pl.whole) {
            pieces = pl.pieces;
            rank = (g - pl.whole) / static_cast<uint32_t>(pieces);
            piece = static_cast<int>(g - pl.whole - rank * pieces);
            slot = static_cast<int>(rank) * pieces;
            rank += pl.whole;
        }
    } else if (g < pl.split_end) {
        pieces = pl.pieces;
        rank = g / static_cast<uint32_t>(pieces);
        piece = static_cast<int>(g - rank * pieces);
        slot = static_cast<int>(rank) * pieces;
    } else if (pl.pieces > 1) {
        rank = g - static_cast<uint32_t>(pl.n_split * units * (pl.pieces - 1));
    }
    const uint32_t tile = rank / static_cast<uint32_t>(units);
    int level;
    Item it = sc.at(static_cast<int>(tile), &level);
    it.unit = static_cast<int>(rank - tile * units);
    it.j0 = 0;
    if (WINDOW && level > 0) level -= sight<WINDOW>(sc.p, it.off).gap();
    it.j1 = it.n = level;
    if (pieces > 1) {
        it.j0 = piece_begin(level, piece, pieces);
        it.j1 = piece_begin(level, piece + 1, pieces);
        it.slot = slot;
        it.piece = piece;
        it.pieces = pieces;
    }
    return it;
}

// ---------------------------------------------------------------- kernel

template <int D, bool WINDOW>
__global__ void __launch_bounds__(PR_THREADS, 1) ub_attn_prompt_kernel(const __grid_constant__ PromptParams p)
{
    using Sh = PromptShape<D>;
    constexpr int NST = Sh::STAGES;
    constexpr bool EARLY = D == 128;
    extern __shared__ __align__(1024) uint8_t base[];
    const uint32_t sm_q = smem_u32(base), sm_kv = sm_q + 2 * Sh::TILE_BYTES;
    float *sm_sum = reinterpret_cast<float *>(base + (2 + NST) * Sh::TILE_BYTES);  // [2][128]
    float *sm_max = sm_sum + 256;                                                  // [2][128]
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm_max + 256);
    const uint32_t b0 = smem_u32(bars);
    const uint32_t kv_full = b0, v_raw = b0 + 8 * NST, kv_done = b0 + 16 * NST;
    const uint32_t misc = b0 + 16 * NST + 8 * DONE;
    const uint32_t q_full = misc, q_empty = misc + 16, s_full = misc + 32, p_full = misc + 48, p_part = misc + 152, o_empty = misc + 64,
                   l_full = misc + 80, l_empty = misc + 96, o_full = misc + 112, drain = misc + 128, want = misc + 144,
                   parts_done = misc + 168, join_go = misc + 176,
                   it_full = misc + 184, it_empty = it_full + 8 * ITEMS;
    auto *items = reinterpret_cast<Work<WINDOW> *>(reinterpret_cast<uint8_t *>(bars) + 16 * NST + 8 * DONE + 184 + 16 * ITEMS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(items + ITEMS);
    volatile uint32_t *turn = tmem_slot + 1;     // steps that the issuer of each q tile has done
    static_assert(16 * NST + 8 * DONE + 184 + 16 * ITEMS + sizeof(Work<WINDOW>) * ITEMS + 12 <= 1024, "barrier area");

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if ((sm_q & 1023u) != 0u) {  // the swizzled tiles need what the declaration asks for
        if (threadIdx.x == 0) atomicCAS(p.b.status, 0, UB_ERR_ALIGN);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(kv_full + 8 * i, 1);
            mbar_init(v_raw + 8 * i, 1);
        }
        for (int i = 0; i < DONE; ++i) mbar_init(kv_done + 8 * i, 2);  // both issuing warps
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 1);
            mbar_init(q_empty + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_part + 8 * i, 4);    // the first PART steps of P written, O rescaled
            mbar_init(p_full + 8 * i, 4);
            mbar_init(o_empty + 8 * i, 4);
            mbar_init(l_full + 8 * i, 4);
            mbar_init(l_empty + 8 * i, 4);
            mbar_init(o_full + 8 * i, 1);
        }
        mbar_init(drain, 1);
        mbar_init(drain + 8, 1);
        mbar_init(want, 1);
        mbar_init(parts_done, 4);
        mbar_init(join_go, 1);
        turn[0] = turn[1] = 0;
        for (int i = 0; i < ITEMS; ++i) {
            mbar_init(it_full + 8 * i, 1);
            mbar_init(it_empty + 8 * i, 15);  // every warp but the schedule's
        }
        fence_mbar_init();
        prefetch_tmap(&p.tmQ);
        prefetch_tmap(&p.tmK);
        prefetch_tmap(&p.tmV);
    }
    if (warp == 13) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (warp != 15) {
        pdl_wait();
        pdl_trigger();
    }

    const WaitCtx wc{p.abort_word, p.b.status, p.timeout_ns, p.epoch};
    const int pack = 1 << p.pack_shift;
    const int tpt = PROMPT_ROWS >> p.pack_shift;  // tokens per q tile
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        alive = __all_sync(0xffffffffu, mbar_wait(bar, parity, wc)) != 0;
        return alive;
    };
    auto arrive = [&](uint32_t bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // The k-th item of this CTA; false at the end (or when a wait ran out).
    auto next_item = [&](uint32_t k, Work<WINDOW> &it) {
        const uint32_t slot = k % ITEMS;
        if (!wait(it_full + 8 * slot, (k / ITEMS) & 1)) return false;
        it = items[slot];
        arrive(it_empty + 8 * slot);
        return it.row0 >= 0;
    };

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        more_registers<SOFTMAX_REGS>();
        const int i = warp >> 2;                       // q tile
        const int row = (warp & 3) * 32 + lane;
        const uint32_t ts = tmem + TM_S + i * 128 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const float sl = p.scale * 1.4426950408889634f;
        uint32_t n_s = 0, n_l = 0;                     // phases used
        Work<WINDOW> it;
        uint32_t k = 0;
        for (; next_item(k, it); ++k) {
            const Sight<WINDOW> in = it.in;
            const int n = i == 0 ? it.r.n[0] : it.r.n[1];
            if (n == 0) continue;
            const int token = i * tpt + (row >> p.pack_shift);
            int reach = it.off + token + 1;            // keys this row sees
            reach = reach > it.len ? it.len : reach;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j) {
                if (!wait(s_full + 8 * i, n_s & 1)) break;
                ++n_s;
                tc_fence_after();
                float s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, reinterpret_cast<uint32_t *>(s) + c * 32);
                tmem_wait_ld();
                const int key0 = in.tile(it.j0 + j) * PROMPT_KEYS, cols = reach - key0;
                // Columns past the row, and those between the sinks and its window: 32 at a time, where
                // a row of the warp has any (four sequences of 8037 tokens together, 8 heads, window
                // 1024: 37.5 us; every column compared: 41.4).
                const int from = WINDOW ? p.sinks - key0 : 0, to = WINDOW ? it.off + token - p.window + 1 - key0 : 0;
                if (__any_sync(0xffffffffu, cols < PROMPT_KEYS || (WINDOW && to > 0 && from < PROMPT_KEYS))) {
#pragma unroll
                    for (int c0 = 0; c0 < 128; c0 += 32) {
                        uint32_t seen = bits_below(cols - c0);
                        if (WINDOW) seen &= bits_below(from - c0) | ~bits_below(to - c0);
                        if (__any_sync(0xffffffffu, seen != 0xffffffffu)) {
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(seen & (1u << c))) s[c0 + c] = -INFINITY;
                        }
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
                // S of this tile being there, O of the last tile is complete.
                if (j > 0 && __any_sync(0xffffffffu, moves)) {
                    const uint32_t to = ts + (TM_O - TM_S);
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
                    if ((EARLY && c0 + 32 == PART * 16) || c0 == 96) {
                        tmem_wait_st();
                        tc_fence_before();
                        arrive((c0 == 96 ? p_full : p_part) + 8 * i);
                    }
                }
                const uint64_t both = add2(sum[0], sum[1]);
                l = l * f + (low(both) + high(both));
            }
            if (!alive) break;
            if (!wait(l_empty + 8 * i, (n_l & 1) ^ 1)) break;
            ++n_l;
            sm_sum[i * 128 + row] = l;
            sm_max[i * 128 + row] = m;
            arrive(l_full + 8 * i);
        }
        // A split item is the last one of its CTA (without windows the only one) and of the CTAs of
        // its other pieces. When all pieces' parts are there, each CTA joins a share: 16 columns of
        // 128 rows at a time.
        it = items[k > 0 ? (k - 1) % ITEMS : 0];
        if (it.slot >= 0 && alive) {
            if (warp == 0) {
                // a count of the item's pieces, and one, never reset, of how often all have come
                uint32_t *counter = p.counters + it.slot / it.pieces, *times = counter + PROMPT_SLOTS / 2;
                if (wait(parts_done, 0) && lane == 0) {
                    const uint32_t before = *static_cast<volatile uint32_t *>(times);
                    uint32_t come;
                    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(come) : "l"(counter) : "memory");
                    if (come == static_cast<uint32_t>(it.pieces - 1)) {
                        *counter = 0u;                 // zero again for the next call
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
                arrive(join_go);
            }
            if (alive && wait(join_go, 0)) {
                const int gap = it.in.gap();
                const Range2 r = it.r;
                const int per = D / 16;                // units of a q tile
                for (int u = it.piece + it.pieces * i; u < 2 * per; u += 2 * it.pieces) {
                    const int t = u / per, c = (u - t * per) * 16;
                    const int rows_tok = t == 0 ? r.tok[0] : r.tok[1], lim = t == 0 ? r.lim[0] : r.lim[1];
                    if (rows_tok == 0) continue;
                    // key tiles that q tile t reaches
                    const int n = (lim + PROMPT_KEYS - 1) / PROMPT_KEYS - (lim > 0 ? gap : 0);
                    const float *rows = p.ws_rows + static_cast<int64_t>(it.slot) * 512 + t * 128 + row;
                    const float4 *cols = reinterpret_cast<const float4 *>(p.ws) + static_cast<int64_t>(it.slot) * (64 * D) +
                                         c / 4 * 256 + t * 128 + row;
                    float M = -INFINITY, L = 0.f, acc[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
                    for (int q0 = 0; q0 < it.pieces; q0 += 4) {
                        float4 v[4][4];
                        float m[4], l[4], top = M;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int b = piece_begin(it.n, q0 + q, it.pieces);
                            m[q] = -INFINITY;          // no such part, or no key of this q tile in it
                            l[q] = 0.f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[q][e] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (q0 + q >= it.pieces || b >= n || piece_begin(it.n, q0 + q + 1, it.pieces) == b) continue;
                            m[q] = __ldcg(rows + (q0 + q) * 512);
                            l[q] = __ldcg(rows + (q0 + q) * 512 + 256);
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[q][e] = __ldcg(cols + static_cast<int64_t>(q0 + q) * (64 * D) + e * 256);
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) top = fmaxf(top, m[q]);
                        const float ref = top == -INFINITY ? 0.f : top, f0 = ex2((M - ref) * sl);
                        M = top;
                        L *= f0;
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[e] *= f0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float f = ex2((m[q] - ref) * sl);
                            L += l[q] * f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                acc[4 * e] += v[q][e].x * f;
                                acc[4 * e + 1] += v[q][e].y * f;
                                acc[4 * e + 2] += v[q][e].z * f;
                                acc[4 * e + 3] += v[q][e].w * f;
                            }
                        }
                    }
                    const int token = t * tpt + (row >> p.pack_shift);
                    const int h = (it.unit << p.pack_shift) + (row & (pack - 1));
                    if (token >= it.ntok) continue;
                    const float inv = 1.f / L;
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + (it.row0 + token) * p.o_row + h * p.o_head + c;
#pragma unroll
                    for (int e = 0; e < 16; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            w[x] = L == 0.f ? 0u
                                            : pack_bf16x2(__float_as_uint(acc[e + 2 * x] * inv), __float_as_uint(acc[e + 2 * x + 1] * inv));
                        *reinterpret_cast<uint4 *>(dst + e) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (p.lse && c == 0)
                        p.lse[static_cast<int64_t>(it.row0 + token) * p.heads + h] =
                            L > 0.f ? M * p.scale + logf(L) : (L == 0.f ? -INFINITY : L);
                }
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------ epilogue
        fewer_registers<EPILOGUE_REGS>();
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t n_o[2] = {0, 0};
        Work<WINDOW> it;
        for (uint32_t k = 0; next_item(k, it); ++k) {
            const Range2 r = it.r;
            // A split item's part: [columns / 4][256 rows][4] fp32 and the rows' maxima and sums.
            float4 *part_o = reinterpret_cast<float4 *>(p.ws) + static_cast<int64_t>(it.slot + it.piece) * (64 * D) + row;
            float *part_m = p.ws_rows + static_cast<int64_t>(it.slot + it.piece) * 512 + row;
            // One row's 32 columns from c on, times f, or zeros.
            auto store = [&](int i, int c, const float *v, float f, bool none) {
                const int token = i * tpt + (row >> p.pack_shift);
                const int h = (it.unit << p.pack_shift) + (row & (pack - 1));
                if (token >= it.ntok) return;
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + (it.row0 + token) * p.o_row + h * p.o_head + c;
#pragma unroll
                for (int u = 0; u < 32; u += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = none ? 0u : pack_bf16x2(__float_as_uint(v[u + 2 * e] * f), __float_as_uint(v[u + 2 * e + 1] * f));
                    *reinterpret_cast<uint4 *>(dst + u) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            };
            auto store_lse = [&](int i, float m, float l) {
                const int token = i * tpt + (row >> p.pack_shift);
                const int h = (it.unit << p.pack_shift) + (row & (pack - 1));
                if (p.lse && token < it.ntok)
                    p.lse[static_cast<int64_t>(it.row0 + token) * p.heads + h] =
                        l > 0.f ? m * p.scale + logf(l) : (l == 0.f ? -INFINITY : l);
            };
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (r.tok[i] == 0 || !alive) continue;
                if (r.n[i] == 0) {
                    if (it.slot >= 0) continue;        // no key in this piece: not a part of this q tile
                    const float zero[32] = {};
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) store(i, c, zero, 0.f, true);
                    store_lse(i, -INFINITY, 0.f);
                    continue;
                }
                if (!wait(l_full + 8 * i, n_o[i] & 1)) continue;
                const float l = sm_sum[i * 128 + row], m = sm_max[i * 128 + row];
                arrive(l_empty + 8 * i);
                if (!wait(o_full + 8 * i, n_o[i] & 1)) continue;
                ++n_o[i];
                tc_fence_after();
                const float inv = 1.f / l;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float v[32];
                    tmem_ld32(tmem + TM_O + i * 128 + lanes + c, reinterpret_cast<uint32_t *>(v));
                    tmem_wait_ld();
                    if (it.slot < 0) {
                        store(i, c, v, inv, l == 0.f);
                    } else {
                        float4 *to = part_o + i * 128 + c / 4 * 256;
#pragma unroll
                        for (int u = 0; u < 32; u += 4) to[u / 4 * 256] = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
                    }
                }
                tc_fence_before();
                arrive(o_empty + 8 * i);
                if (it.slot < 0) {
                    store_lse(i, m, l);
                } else {
                    part_m[i * 128] = m;
                    part_m[i * 128 + 256] = l;
                }
            }
            if (!alive) break;
            if (it.slot < 0) continue;
            arrive(parts_done);                        // the softmax warps join it
        }
    } else {
      // the four single warps
      fewer_registers<SINGLE_REGS>();
      if (warp == 12) {
        // ------------------------------------------------------------ loads
        uint32_t c = 0, n_q[2] = {0, 0};               // ring position, Q loads so far
        uint32_t n_done = 0, freed = 0;                // releases seen; ring positions that they freed
        uint32_t two = 0, n_ends = 0;                  // bit of each release to come: frees two positions
        Work<WINDOW> it;
        const int box = PROMPT_KEYS < (1 << p.b.page_shift) ? PROMPT_KEYS : (1 << p.b.page_shift);
        constexpr int HALVES = D / 64;
        for (uint32_t k = 0;; ++k) {
            if (k >= 2) arrive(want);                  // every load of item k - 1 has been issued
            if (!next_item(k, it)) break;
            const Sight<WINDOW> in = it.in;
            const Range2 r = it.r;
            const int kvh = (it.unit << p.pack_shift) / p.group;
            const int32_t *table = p.paged ? p.b.page_table + it.src * p.b.table_row : nullptr;
            const int pages = p.paged ? (it.len + (1 << p.b.page_shift) - 1) >> p.b.page_shift : 0;
            int cached0 = 0, cached_n = 0, ids = -1;   // page ids, one per lane
            auto load_q = [&](int i) {
                if ((i == 0 ? r.n[0] : r.n[1]) == 0) return;
                const int n = i == 0 ? n_q[0]++ : n_q[1]++;
                if (n > 0 && !wait(q_empty + 8 * i, (n - 1) & 1)) return;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full + 8 * i, Sh::TILE_BYTES);
                    for (int hf = 0; hf < HALVES; ++hf)
                        tma_load_3d(sm_q + i * Sh::TILE_BYTES + hf * Sh::HALF_BYTES, &p.tmQ, q_full + 8 * i, hf * 64,
                                    it.unit << p.pack_shift, it.row0 + i * tpt);
                }
                __syncwarp();
            };
            for (int j = 0; j < 2 || j < r.nmax; ++j) {
                if (j < 2) load_q(j);
                if (!alive || j >= r.nmax) continue;
                const int kt = in.tile(it.j0 + j), key0 = kt * PROMPT_KEYS;
                // every key that is multiplied is loaded (pages past the length as zeros)
                const int n_box = p.paged ? (extent(r.limmax, kt) + box - 1) / box : 1;
                const int page0 = key0 >> p.b.page_shift;
                const int boxes = PROMPT_KEYS / box;
                if (p.paged && page0 + boxes > cached0 + cached_n) {
                    cached0 = page0;
                    cached_n = 32;
                    // a page that no row sees may be another sequence's by now, or nobody's
                    const int64_t first = static_cast<int64_t>(cached0 + lane) << p.b.page_shift;
                    const bool seen = cached0 + lane < pages &&
                                      (!WINDOW || first + (int64_t(1) << p.b.page_shift) > in.lo || first < p.sinks);
                    ids = seen ? table[cached0 + lane] : -1;
                    if (seen && (ids < 0 || ids >= p.b.num_pages)) {
                        atomicCAS(p.b.status, 0, UB_ERR_ARG);
                        ids = -1;                      // outside the tensor: filled with zeros
                    }
                }
#pragma unroll
                for (int kind = 0; kind < 2 && alive; ++kind, ++c) {
                    const uint32_t st = c % NST;
                    while (c - freed >= NST && wait(kv_done + 8 * (n_done % DONE), (n_done / DONE) & 1)) {
                        freed += 1u + ((two >> (n_done % 32)) & 1u);
                        ++n_done;
                    }
                    if (!alive) break;
                    // The MMA warp releases K of tile 0, then V of each tile with K of the next.
                    if (kind == 0 || j == r.nmax - 1) {
                        const uint32_t at = n_ends++ % 32;
                        two = (two & ~(1u << at)) | (static_cast<uint32_t>(kind == 0 && j > 0) << at);
                    }
                    // The last tile of V goes through the zeroing warp when it ends inside 16 keys.
                    const bool fix = kind == 1 && j == r.nmax - 1 && extent(r.limmax, kt) > it.len - key0;
                    const uint32_t bar = (fix ? v_raw : kv_full) + 8 * st;
                    const CUtensorMap *map = kind == 0 ? &p.tmK : &p.tmV;
                    const uint32_t dst = sm_kv + st * Sh::TILE_BYTES;
                    if (lane == 0)
                        mbar_arrive_expect_tx(bar, p.paged ? n_box * HALVES * box * 128 : Sh::TILE_BYTES);
                    __syncwarp();
                    if (p.paged) {
                        const int bx = lane / HALVES, hf = lane - bx * HALVES;
                        const int page = __shfl_sync(0xffffffffu, ids, (page0 - cached0 + bx) & 31);
                        if (bx < n_box)
                            tma_load_4d(dst + hf * Sh::HALF_BYTES + bx * box * 128, map, bar, hf * 64,
                                        boxes > 1 ? 0 : key0 & ((1 << p.b.page_shift) - 1), kvh, page);
                    } else if (lane < HALVES) {
                        tma_load_3d(dst + lane * Sh::HALF_BYTES, map, bar, lane * 64, kvh, it.src + key0);
                    }
                    __syncwarp();
                }
            }
            if (!alive) break;
        }
    } else if (warp < 15) {
        // ------------------------------------------------------------ MMA issue
        // A warp per q tile. The whole warp walks the tiles and one elected lane issues, on values
        // that are the same in every lane (broadcast from lane 0, so that the compiler knows):
        // descriptors then stay in uniform registers, and an issue costs less than the MMA takes.
        // The two warps take turns, step by step: one waits for its weights while the other's
        // MMAs are being taken by the tensor core, and the tiles stay half a period apart.
        const int i = warp - 13;
        uint32_t c = 0, n_done = 0, n_q = 0, n_p = 0, step = 0;
        const uint32_t tp = tmem + TM_S + i * 128, to = tmem + TM_O + i * 128;
        const uint64_t q_desc = smem_desc_sw128(sm_q + i * Sh::TILE_BYTES), k_desc = smem_desc_sw128(sm_kv),
                       v_desc = smem_desc_v(sm_kv, Sh::HALF_BYTES);
        // Every tile of the ring is waited for, used or not: phases are seen one by one.
        auto wait_kv = [&](uint32_t cs) { return wait(kv_full + 8 * (cs % NST), (cs / NST) & 1); };
        auto in_turn = [&](uint32_t g) {
            const volatile uint32_t *other = turn + (1 - i);
            bool mine = __all_sync(0xffffffffu, static_cast<int32_t>(*other - g) >= 0) != 0;
            if (mine) return true;
            WaitClock clk;
            for (uint32_t n = 1; !mine; ++n) {
                mine = __all_sync(0xffffffffu, static_cast<int32_t>(*other - g) >= 0) != 0;
                if ((n & 15u) == 0 && !mine && !__all_sync(0xffffffffu, clk.ok(wc))) return alive = false;
            }
            return true;
        };
        Work<WINDOW> it;
        for (uint32_t k = 0; next_item(k, it); ++k) {
            Sight<WINDOW> in = it.in;
            if (WINDOW) in.near = __shfl_sync(0xffffffffu, in.near, 0), in.far = __shfl_sync(0xffffffffu, in.far, 0);
            const Range2 r = uniform(it.r);
            const int n = i == 0 ? r.n[0] : r.n[1], lim = i == 0 ? r.lim[0] : r.lim[1];
            const int j0 = __shfl_sync(0xffffffffu, it.j0, 0);
            if (n > 0) {
                if (!wait(q_full + 8 * i, n_q & 1)) break;
                ++n_q;
            }
            // Step j: O += P V of tile j, then S of tile j + 1. Ring: V of tile j at c - 1, K of
            // tile j + 1 at c.
            for (int j = -1; j < r.nmax; ++j, c += 2) {
                const bool has_v = j >= 0, has_k = j + 1 < r.nmax;
                const bool pv = has_v && j < n, s_next = has_k && j + 1 < n;
                if (has_v && !wait_kv(c - 1)) break;
                if (has_k && !wait_kv(c)) break;
                if (j == 0 && pv && !wait(o_empty + 8 * i, n_q & 1)) break;  // n_q - 1 items written out
                ++step;
                if (!in_turn(step - 1 + i)) break;
                const uint64_t v = v_desc + ((c - 1) % NST) * (Sh::TILE_BYTES / 16);
                const uint64_t kk = k_desc + (c % NST) * (Sh::TILE_BYTES / 16);
                const int steps = pv ? extent(lim, in.tile(j0 + j)) / 16 : 0;
                const uint32_t s_idesc = attn_idesc(s_next ? extent(lim, in.tile(j0 + j + 1)) : 16, false);
                constexpr uint32_t o_idesc = attn_idesc(D, true);
                if (pv) {
                    if (EARLY) {
                        if (!wait(p_part + 8 * i, n_p & 1)) break;
                        tc_fence_after();
                        if (steps == PROMPT_KEYS / 16 && elect_one()) {
#pragma unroll
                            for (int s = 0; s < PART; ++s) umma_ts(to, tp + s * 8, v + s * 128, o_idesc, j > 0 || s > 0);
                        }
                        __syncwarp();
                    }
                    if (!wait(p_full + 8 * i, n_p & 1)) break;
                    ++n_p;
                }
                tc_fence_after();
                if (elect_one()) {
                    if (steps == PROMPT_KEYS / 16) {
#pragma unroll
                        for (int s = EARLY ? PART : 0; s < PROMPT_KEYS / 16; ++s)
                            umma_ts(to, tp + s * 8, v + s * 128, o_idesc, j > 0 || s > 0);
                    } else {  // the sequence's last keys
                        for (int s = 0; s < steps; ++s) umma_ts(to, tp + s * 8, v + s * 128, o_idesc, j > 0 || s > 0);
                    }
                    if (s_next) {
#pragma unroll
                        for (int s = 0; s < D / 16; ++s) {
                            const int o = (s / 4) * (Sh::HALF_BYTES / 16) + (s % 4) * 2;
                            umma_ss(tp, q_desc + o, kk + o, s_idesc, s > 0);
                        }
                        umma_commit(s_full + 8 * i);
                        if (j + 2 == n) umma_commit(q_empty + 8 * i);
                    }
                    turn[i] = step;
                    if (pv && j == n - 1) umma_commit(o_full + 8 * i);
                    if (has_v || has_k) umma_commit(kv_done + 8 * (n_done % DONE));
                }
                __syncwarp();
                if (has_v || has_k) ++n_done;
            }
            if (!alive) break;
            c -= 2;  // nmax + 1 steps over 2 nmax tiles
        }
        // everything issued has completed before TMEM goes back
        if (elect_one()) {
            umma_commit(drain + 8 * i);
            mbar_wait_drain(drain + 8 * i, 0, p.timeout_ns);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ schedule
        // The first item is looked up twice, at first in a call of made-up numbers and before the
        // grid ahead has finished: the code is in the instruction cache by the time that this
        // call's numbers may be read, and everything else waits for the first item.
        Schedule sched{p, lane, 0, 1, 0, 0, {0, lane == 0 ? 65536 : 0, lane == 0 ? 65536 : 0, 0}};
        Plan plan;
        Item it;
#pragma unroll 1
        for (int real = 0; real < 2; ++real) {
            if (real) {
                pdl_wait();
                pdl_trigger();
                sched.n_seqs = p.b.n_seqs;
                sched.own = lane < p.b.n_seqs ? seq_info(p, lane) : SeqInfo{0, 0, 0, 0};
            }
            // Items of one q tile where those are no more than the CTAs and are not split, of two
            // elsewhere.
            sched.shift = 7 - p.pack_shift;
            int cap = INT_MAX;
            for (;; ++sched.shift) {
                sched.measure();
                // key tiles in sight of an item: its rows' windows, and the sinks
                if (WINDOW)
                    cap = static_cast<int>((static_cast<int64_t>(p.window) + (1 << sched.shift) + 2 * PROMPT_KEYS - 3) / PROMPT_KEYS) +
                          (p.sinks + PROMPT_KEYS - 1) / PROMPT_KEYS;
                if (sched.shift == 8 - p.pack_shift ||
                    (static_cast<uint32_t>(sched.tiles) * p.units <= gridDim.x && (sched.cmax <= MIN_SPLIT || cap <= MIN_SPLIT)))
                    break;
            }
            plan = plan_of<WINDOW>(sched, p.units, gridDim.x, p.slots, cap);
            it = kNoItem;
            if (blockIdx.x < plan.total) it = item_of<WINDOW>(sched, plan, p.units, blockIdx.x);
        }
        // Longest first. The first two items of each CTA are dealt forth and back over the CTAs,
        // the rest by tickets, drawn when the loads of the item before have been issued.
        auto publish = [&](uint32_t k, Item it) {
            if (k >= ITEMS && !wait(it_empty + 8 * (k % ITEMS), (k / ITEMS - 1) & 1)) return;
            if (lane == 0) {
                Work<WINDOW> &w = items[k % ITEMS];
                static_cast<Item &>(w) = it;
                w.in = sight<WINDOW>(p, it.off);
                w.r = ranges(it, tpt, w.in.gap());
            }
            arrive(it_full + 8 * (k % ITEMS));
        };
        auto draw = [&](uint32_t k) {
            uint32_t g = 2 * gridDim.x - 1 - blockIdx.x;
            if (WINDOW && plan.whole > 0u) {
                // a piece of the last round is its CTA's last item: all is dealt, nothing drawn
                if (k >= 2) g = k * gridDim.x + blockIdx.x;
            } else if (k >= 2) {
                uint32_t ticket = 0;
                if (lane == 0) ticket = atomicAdd(p.tickets, 1u);
                g = 2 * gridDim.x + __shfl_sync(0xffffffffu, ticket, 0);
            }
            Item drawn = kNoItem;
            if (g < plan.total) drawn = item_of<WINDOW>(sched, plan, p.units, g);
            publish(k, drawn);
            return drawn;
        };
        uint32_t c = 0, used = 0;                      // ring position; phase bit per stage of v_raw
        publish(0, it);
        Item it1 = it;
        if (it.row0 >= 0) it1 = draw(1);
        for (uint32_t k = 0; it.row0 >= 0 && alive; ++k) {
            // it: item k, it1: item k + 1, published before the zeroing of item k is waited for
            if (k >= 1) {
                if (!wait(want, (k - 1) & 1)) break;
                it1 = draw(k + 1);
                if (!alive) break;
            }
            const Sight<WINDOW> in = items[k % ITEMS].in;
            const Range2 r = items[k % ITEMS].r;
            const int j = r.nmax - 1, kt = in.tile(it.j0 + j), valid = it.len - kt * PROMPT_KEYS;
            const int ext = r.nmax > 0 ? extent(r.limmax, kt) : 0;
            if (ext > valid) {
                const uint32_t st = (c + 2 * j + 1) % NST;
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
            c += 2 * r.nmax;
            it = it1;
        }
      }
    }

    if (!alive) settle(200000);  // a wait ran out: copies already issued land first
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 13) tmem_dealloc(tmem, 512);
    // The last CTA of the call leaves the tickets at zero.
    if (threadIdx.x == 0 && atomicAdd(p.tickets + 1, 1u) == gridDim.x - 1) p.tickets[0] = p.tickets[1] = 0u;
}

template <int D, bool WINDOW>
cudaError_t launch_prompt(const PromptParams &p, int grid, cudaStream_t s)
{
    const cudaError_t e =
        raise_smem_limit(reinterpret_cast<const void *>(ub_attn_prompt_kernel<D, WINDOW>), PromptShape<D>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_ex(ub_attn_prompt_kernel<D, WINDOW>, p, grid, PR_THREADS, PromptShape<D>::SMEM, 1, p.pdl != 0, s);
}

}  // namespace

cudaError_t launch_attn_prompt(const PromptParams &p, int grid, cudaStream_t s)
{
    if (p.window > 0) return p.head_dim == 128 ? launch_prompt<128, true>(p, grid, s) : launch_prompt<64, true>(p, grid, s);
    return p.head_dim == 128 ? launch_prompt<128, false>(p, grid, s) : launch_prompt<64, false>(p, grid, s);
}

}  // namespace ubk
