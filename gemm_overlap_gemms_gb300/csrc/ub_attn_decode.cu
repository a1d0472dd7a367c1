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
// the host knowing a length. An item (sequence, head) that spans CTAs is joined by the CTA
// that finishes last: each part goes to the workspace, a counter per item tells who came
// last, and parts are added in CTA order (deterministic). Above 16 parts the join has two
// levels, groups of 16 consecutive parts first, so that no CTA reads all of them.
//
// A CTA is a loading warp and four computing warps, two CTAs on an SM. The loading warp
// fills a ring of stages (one tile's keys and values) with TMA boxes of one page or one
// tile, whichever is smaller; each computing warp takes every fourth tile by itself with
// its own running maximum, so that no barrier separates tiles; the four partials are
// joined in shared memory at the end of an item.
#include <cuda_bf16.h>

#include "ub_attn.h"
#include "ub_device.cuh"
#include "ub_internal.h"

namespace ubk {
namespace {

constexpr int KT = DECODE_KEYS;
constexpr int WARPS = 4;
constexpr int DEC_THREADS = 32 * (WARPS + 1);
constexpr int JOIN_GROUP = 16;           // parts per first-level join

template <int D, int NT>
struct DecShape {
    static constexpr int TILE_BYTES = KT * D * 2;
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int HEADS = 8 * NT;
    static constexpr int O_ROW = D + 4;                           // padded: conflict-free writes
    static constexpr int MERGE_BYTES = WARPS * HEADS * O_ROW * 4;
    // As many stages as fit twice on an SM (115,712 bytes per CTA with the reserve).
    static constexpr int STAGES_FIT = (115712 - 2048 - MERGE_BYTES) / STAGE_BYTES;
    // A multiple of WARPS, so that a stage always belongs to the same warp: the loads of two
    // tiles may land in either order, and a warp that waited for the second fill of a stage
    // whose first fill (another warp's) has not landed would see the parity it waits for.
    static constexpr int STAGES = STAGES_FIT < 8 ? STAGES_FIT / WARPS * WARPS : 8;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + MERGE_BYTES + 768;
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

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int row,
                                            int head, int page)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(row), "r"(head), "r"(page)
        : "memory");
}

__device__ __forceinline__ float4 ld_cg4(const float *p)
{
    float4 v;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ float ld_cg(const float *p)
{
    float v;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void bar_compute() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ int clamped_len(const SeqBatch &b, int seq)
{
    const int len = b.kv_lens[seq];
    const int64_t most = static_cast<int64_t>(b.table_width) << b.page_shift;
    return len < 0 ? 0 : (len > most ? static_cast<int>(most) : len);
}
__device__ __forceinline__ int tiles_of(int len) { return len > 0 ? (len + KT - 1) / KT : 1; }

// The equal split of `total` tiles over `ctas`: CTA c's first tile, and the CTA of a tile.
struct Split {
    int64_t base, rem;
    __device__ __forceinline__ int64_t first(int64_t c) const { return c * base + (c < rem ? c : rem); }
    __device__ __forceinline__ int owner(int64_t x) const
    {
        const int64_t cut = rem * (base + 1);
        return static_cast<int>(x < cut ? x / (base + 1) : rem + (x - cut) / base);
    }
};

// Sum of all lengths' tiles, and the sequence that holds per-head tile `x` (one warp).
__device__ __forceinline__ int64_t total_tiles(const SeqBatch &b, int lane)
{
    int64_t sum = 0;
    for (int i = lane; i < b.n_seqs; i += 32) sum += tiles_of(clamped_len(b, i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}
__device__ __forceinline__ void find_seq(const SeqBatch &b, int lane, int64_t tile, int heads, int *seq, int64_t *before)
{
    int64_t seen = 0;  // tiles of the sequences before this batch of 32, over all heads
    for (int i0 = 0; i0 < b.n_seqs; i0 += 32) {
        const int64_t mine =
            i0 + lane < b.n_seqs ? static_cast<int64_t>(tiles_of(clamped_len(b, i0 + lane))) * heads : 0;
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, seen + upto > tile);
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

template <int D, int NT>
__global__ void __launch_bounds__(DEC_THREADS, DECODE_CTAS_PER_SM)
    ub_attn_decode_kernel(const __grid_constant__ DecodeParams p)
{
    using Sh = DecShape<D, NT>;
    constexpr int S = Sh::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *sm_o = reinterpret_cast<float *>(base + S * Sh::STAGE_BYTES);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + S * Sh::STAGE_BYTES + Sh::MERGE_BYTES);
    float *sm_m = reinterpret_cast<float *>(bars + 2 * S);                     // [WARPS][HEADS]
    float *sm_l = sm_m + WARPS * DECODE_HEADS;                                 // [WARPS][HEADS]
    int *sm_last = reinterpret_cast<int *>(sm_l + WARPS * DECODE_HEADS);
    static_assert(2 * S * 8 + 2 * WARPS * DECODE_HEADS * 4 + 4 <= 768, "barrier area");
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + S);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
    const int64_t total = total_tiles(b, lane) * heads;
    // No CTA gets fewer than MIN_TILES tiles: below, one more part to join costs more than
    // the tiles it takes off the others.
    constexpr int MIN_TILES = 4;
    int64_t ctas = total / MIN_TILES;
    ctas = ctas < 1 ? 1 : (ctas > gridDim.x ? gridDim.x : ctas);
    if (blockIdx.x >= ctas) return;
    const Split split{total / ctas, total % ctas};
    const int64_t x0 = split.first(blockIdx.x), x1 = split.first(blockIdx.x + 1);

    int seq;
    int64_t before;
    find_seq(b, lane, x0, heads, &seq, &before);
    const WaitCtx wc{p.abort_word, p.status_word(), p.timeout_ns, p.epoch};
    bool alive = true;
    uint32_t count = 0;  // tiles of this CTA so far: stage count % S, phase count / S

    for (int64_t x = x0; x < x1 && seq < b.n_seqs;) {
        const int len = clamped_len(b, seq);
        const int tiles = tiles_of(len);
        const int head = static_cast<int>((x - before) / tiles);
        const int64_t item0 = before + static_cast<int64_t>(head) * tiles;
        const int t0 = static_cast<int>(x - item0);
        const int t1 = item0 + tiles < x1 ? tiles : static_cast<int>(x1 - item0);
        const int kvh = head / p.head_blocks, hb = head - kvh * p.head_blocks;
        const int h0 = kvh * p.group + hb * DECODE_HEADS;     // first query head
        const int g = p.group - hb * DECODE_HEADS < DECODE_HEADS ? p.group - hb * DECODE_HEADS : DECODE_HEADS;

        if (warp == WARPS) {
            // ---------------------------------------------------------------- loads
            const int box = KT < (1 << b.page_shift) ? KT : (1 << b.page_shift);  // rows per box
            const int boxes = KT / box;
            constexpr int HALVES = D / 64;
            const int32_t *table = b.page_table + seq * b.table_row;
            const int pages = (len + (1 << b.page_shift) - 1) >> b.page_shift;
            int cached0 = 0, cached_n = 0;   // page ids [cached0, cached0 + cached_n), one per lane
            int ids = -1;
            for (int t = t0; t < t1 && alive; ++t, ++count) {
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
                if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n_box) * HALVES * 2 * box * 128);
                __syncwarp();
                // lane = (K or V, box, half)
                const int kind = lane / (boxes * HALVES), rest = lane - kind * boxes * HALVES;
                const int bx = rest / HALVES, half = rest - bx * HALVES;
                const int page = __shfl_sync(0xffffffffu, ids, (page0 - cached0 + bx) & 31);
                if (kind < 2 && bx < n_box)
                    tma_load_4d(smem_u32(base) + stage * Sh::STAGE_BYTES + kind * Sh::TILE_BYTES + half * KT * 128 +
                                    bx * box * 128,
                                kind == 0 ? &p.tmK : &p.tmV, bar, half * 64,
                                boxes > 1 ? 0 : key0 & ((1 << b.page_shift) - 1), kvh, page);
            }
        } else {
            // ---------------------------------------------------------------- compute
            uint32_t qf[NT][D / 16][2];
            const float sl = p.scale * 1.4426950408889634f;
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
                        if (r >= valid) st_shared_v4(vb + half * KT * 128 + r * 128 + (i % 8) * 16, 0u, 0u, 0u, 0u);
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
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const int r = mt * 16 + (lane & 15);
                        const int c = (ks * 2 + (lane >> 4)) & 7;
                        uint32_t a[4];
                        ldsm_x4(kb + (ks / 4) * KT * 128 + r * 128 + ((c ^ (r & 7)) << 4), a);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_16x8x16(s[mt][nt], a, qf[nt][ks][0], qf[nt][ks][1]);
                    }
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
                        f[nt][c] = exp2f((m[nt][c] - ref) * sl);
                        moved |= m[nt][c] != mx;
                        m[nt][c] = mx;
                        float sum = 0.f;
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float &v = s[mt][nt][r * 2 + c];
                                v = exp2f(fmaf(v, sl, -ref * sl));
                                sum += v;
                            }
                        l[nt][c] = l[nt][c] * f[nt][c] + sum;
                    }
                // Weights in BF16, the type of the values they multiply (their sum stays fp32):
                // 2^-9 of each weight, as large as the rounding of the output.
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
                for (int d = 0; d < D / 16; ++d)
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const int r = mt * 16 + (lane & 7) + ((lane >> 4) << 3);
                        const int c = (d * 2 + ((lane >> 3) & 1)) & 7;
                        uint32_t a[4];
                        ldsm_x4_trans(vb + (d / 4) * KT * 128 + r * 128 + ((c ^ (r & 7)) << 4), a);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_16x8x16(o[d][nt], a, pf[mt][nt][0], pf[mt][nt][1]);
                    }
                if (valid < KT) fence_proxy_async_shared();  // the zeroed rows before the next load's writes
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * stage);
            }
            count = static_cast<uint32_t>(x - x0) + (t1 - t0);

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
            const int tid = threadIdx.x;
            constexpr int SLOT = decode_slot_floats(D);
            const int G = gridDim.x;
            auto slot_of = [&](int cta, int which) { return p.ws + (static_cast<int64_t>(which) * G + cta) * SLOT; };
            auto finish = [&](int hh, int d, float4 acc, float M, float L) {
                const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
                uint2 w;
                w.x = pack_bf16x2(__float_as_uint(acc.x * inv), __float_as_uint(acc.y * inv));
                w.y = pack_bf16x2(__float_as_uint(acc.z * inv), __float_as_uint(acc.w * inv));
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + seq * p.o_row +
                                           (h0 + hh) * p.o_head + d) = w;
                if (p.lse && d == 0) p.lse[static_cast<int64_t>(seq) * p.heads + h0 + hh] = M * p.scale + logf(L);
            };
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
                    const float fw = exp2f((sm_m[w * DECODE_HEADS + hh] - ref) * sl);
                    L += sm_l[w * DECODE_HEADS + hh] * fw;
                    const float4 v = *reinterpret_cast<const float4 *>(sm_o + (w * Sh::HEADS + hh) * Sh::O_ROW + d);
                    acc.x += v.x * fw;
                    acc.y += v.y * fw;
                    acc.z += v.z * fw;
                    acc.w += v.w * fw;
                }
                if (whole) {
                    finish(hh, d, acc, M, L);
                } else {
                    *reinterpret_cast<float4 *>(mine + hh * D + d) = acc;
                    if (d == 0) {
                        mine[DECODE_HEADS * D + hh] = M;
                        mine[DECODE_HEADS * (D + 1) + hh] = L;
                    }
                }
            }
            if (!whole) {
                // The last of an item's parts to arrive joins them, in groups of JOIN_GROUP.
                // Counters: group 0 at CTA a, a later group at its first CTA (a CTA is inside at
                // most one item that began before it), the groups of the item at CTA a; the
                // joined groups' slots likewise.
                const int a = split.owner(item0), z = split.owner(item0 + tiles - 1);
                const int parts = z - a + 1, groups = (parts + JOIN_GROUP - 1) / JOIN_GROUP;
                const int gi = (static_cast<int>(blockIdx.x) - a) / JOIN_GROUP;
                auto arrive = [&](uint32_t *counter, int n) {
                    __threadfence();
                    bar_compute();
                    if (tid == 0) {
                        const bool last = atomicAdd(counter, 1u) == static_cast<uint32_t>(n - 1);
                        if (last) *counter = 0u;  // zero again for the next call
                        __threadfence();
                        *sm_last = last ? 1 : 0;
                    }
                    bar_compute();
                    return *sm_last != 0;
                };
                // Part i of n at `part(i)`; joined into `to`, or the output.
                auto join = [&](int n, auto part, float *to) {
                    for (int u = tid; u < g * (D / 4); u += 32 * WARPS) {
                        const int hh = u / (D / 4), d = (u - hh * (D / 4)) * 4;
                        float M = -INFINITY;
                        for (int i = 0; i < n; ++i) M = fmaxf(M, ld_cg(part(i) + DECODE_HEADS * D + hh));
                        const float ref = M == -INFINITY ? 0.f : M;
                        float L = 0.f;
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                        for (int i = 0; i < n; ++i) {
                            const float *q = part(i);
                            const float fw = exp2f((ld_cg(q + DECODE_HEADS * D + hh) - ref) * sl);
                            L += ld_cg(q + DECODE_HEADS * (D + 1) + hh) * fw;
                            const float4 v = ld_cg4(q + hh * D + d);
                            acc.x += v.x * fw;
                            acc.y += v.y * fw;
                            acc.z += v.z * fw;
                            acc.w += v.w * fw;
                        }
                        if (!to) {
                            finish(hh, d, acc, M, L);
                        } else {
                            *reinterpret_cast<float4 *>(to + hh * D + d) = acc;
                            if (d == 0) {
                                to[DECODE_HEADS * D + hh] = M;
                                to[DECODE_HEADS * (D + 1) + hh] = L;
                            }
                        }
                    }
                };
                const int first = a + gi * JOIN_GROUP;
                const int n = parts - gi * JOIN_GROUP < JOIN_GROUP ? parts - gi * JOIN_GROUP : JOIN_GROUP;
                // a part's slot: 1 for the CTA in which the item begins, 0 for the others
                auto part1 = [&](int i) { return slot_of(first + i, first + i == a ? 1 : 0); };
                if (arrive(p.counters + (gi == 0 ? 0 : G) + first, n)) {
                    if (groups == 1) {
                        join(n, part1, nullptr);
                    } else {
                        join(n, part1, slot_of(first, gi == 0 ? 2 : 3));
                        if (arrive(p.counters + 2 * G + a, groups)) {
                            auto part2 = [&](int i) { return slot_of(a + i * JOIN_GROUP, i == 0 ? 2 : 3); };
                            join(groups, part2, nullptr);
                        }
                    }
                }
            }
            bar_compute();  // the shared partials are free again
        }
        if (!__all_sync(0xffffffffu, alive)) alive = false;
        x += t1 - t0;
        if (item0 + tiles == x && head == heads - 1) {
            before += static_cast<int64_t>(tiles) * heads;
            ++seq;
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
