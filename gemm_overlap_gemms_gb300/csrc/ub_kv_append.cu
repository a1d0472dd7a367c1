// Position rotation of queries and keys, and the append of keys and values to a paged
// cache, in one pass over the QKV projection's output.
//
// Token t of sequence s (n_s new tokens, L_s tokens in the cache after them) has position
// pos = L_s - n_s + t - seq_starts[s]. Its query and key heads are rotated in pairs,
//     (a, b) -> (a cos - b sin, b cos + a sin),   cos, sin = table[pos][j],  j < rot / 2,
// the pair j being elements (j, j + rot/2) of the head, or (2j, 2j + 1) when interleaved;
// elements from rot on are copied. The query goes to q_out, the key and the value to row
// pos % page_size of page page_table[s][pos / page_size]. The arithmetic is fp32, with one
// rounding to BF16.
//
// Bound by HBM: every byte is read once and written once. A warp owns a token: it finds
// the token's sequence with one round of loads (each lane compares some of the starts and
// the warp counts the votes: no chain of dependent loads as in a binary search), keeps its
// lane's cos and sin in registers, and walks the token's heads, a lane moving the two
// 16-byte vectors that the rotation pairs. With few tokens the heads of a token are dealt
// over several warps instead, so that the loads of a decoding step are all in flight at
// once.
//
// Measured (GB300): 16166 tokens, 32 + 8 + 8 heads of 128 (401 MB): 64 us, 6.3 TB/s; 8145 tokens,
// 8 + 8 + 8 heads (104 MB): 20.4 us, 5.1 TB/s, of which about 4 us are launch and ramp. CTAs of
// 128 threads (of 256: 68 us) and four heads in flight per lane (two: 66 us, eight: 73 us);
// loading the first heads ahead of the token's place costs registers, and so warps: 77 us.
// Four tokens: 2.4 us of GPU time, 9.5-10.8 us a call, bound by the host's side of it.
#include <cuda_bf16.h>

#include "ub_attn.h"
#include "ub_device.cuh"
#include "ub_internal.h"

namespace ubk {
namespace {

constexpr int APPEND_THREADS = 128;

__device__ __forceinline__ void unpack8(const uint4 &x, float *f)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rotate the pair of vectors (x, y) of one lane. Half-split: element i of x pairs with
// element i of y. Interleaved: neighbours inside each vector; c / s then hold the four
// pairs of x, then the four of y.
__device__ __forceinline__ void rotate(uint4 &x, uint4 &y, const float *c, const float *s, bool interleaved)
{
    float a[8], b[8];
    unpack8(x, a);
    unpack8(y, b);
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
            a[2 * i] = a0 * c[i] - a1 * s[i];
            a[2 * i + 1] = a1 * c[i] + a0 * s[i];
            b[2 * i] = b0 * c[4 + i] - b1 * s[4 + i];
            b[2 * i + 1] = b1 * c[4 + i] + b0 * s[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a0 = a[i], b0 = b[i];
            a[i] = a0 * c[i] - b0 * s[i];
            b[i] = b0 * c[i] + a0 * s[i];
        }
    }
    x = pack8(a);
    y = pack8(b);
}

template <int D>
__global__ void __launch_bounds__(APPEND_THREADS) ub_kv_append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int SLOTS = D / 16;        // lanes per head, two 16-byte vectors each
    constexpr int HL = 32 / SLOTS;       // heads a warp moves at once
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (APPEND_THREADS / 32) + (threadIdx.x >> 5);
    const int t = static_cast<int>(unit / p.parts);
    const int part = static_cast<int>(unit - static_cast<int64_t>(t) * p.parts);
    pdl_wait();
    pdl_trigger();
    if (t >= p.T) return;

    // The token's sequence: how many sequences end at or before t.
    int seq = 0;
    for (int i = 0; i < p.b.n_seqs; i += 32) {
        const bool past = i + lane < p.b.n_seqs && p.b.seq_starts[i + lane + 1] <= t;
        seq += __popc(__ballot_sync(0xffffffffu, past));
    }
    if (seq >= p.b.n_seqs) return;       // a row after the last sequence
    // A sequence ends at T at the latest, for the positions as for the attention over them.
    const int64_t start = p.b.seq_starts[seq], end = min(p.b.seq_starts[seq + 1], p.T);
    if (t < start || t >= end) return;   // starts out of order: no sequence
    const int64_t pos = p.b.kv_lens[seq] - (end - start) + (t - start);
    if (pos < 0 || (p.rot > 0 && pos >= p.max_pos)) {
        if (lane == 0) atomicCAS(p.b.status, 0, UB_ERR_ARG);
        return;
    }
    const int64_t slot_page = pos >> p.b.page_shift;
    const int64_t row = pos & ((int64_t(1) << p.b.page_shift) - 1);
    int64_t page = -1;
    if (slot_page < p.b.table_width) page = p.b.page_table[seq * p.b.table_row + slot_page];
    const bool cached = page >= 0 && page < p.b.num_pages;
    if (!cached && lane == 0) atomicCAS(p.b.status, 0, UB_ERR_ARG);

    const int slot = lane % SLOTS, hl = lane / SLOTS;
    const int half = p.rot / 16;         // 16-byte vectors of half the rotated part
    const bool turns = slot < half;
    const int v0 = turns && !p.interleaved ? slot : 2 * slot;
    const int v1 = turns && !p.interleaved ? slot + half : 2 * slot + 1;
    float c[8], s[8];
    if (turns) {
        const float4 *cp = reinterpret_cast<const float4 *>(p.cos + pos * (p.rot / 2) + slot * 8);
        const float4 *sp = reinterpret_cast<const float4 *>(p.sin + pos * (p.rot / 2) + slot * 8);
        *reinterpret_cast<float4 *>(c) = cp[0];
        *reinterpret_cast<float4 *>(c + 4) = cp[1];
        *reinterpret_cast<float4 *>(s) = sp[0];
        *reinterpret_cast<float4 *>(s + 4) = sp[1];
    }

    const int total = p.heads + 2 * p.kv_heads;
    const int step = HL * p.parts;
    constexpr int U = 4;                 // heads in flight per lane
    for (int h0 = part * HL + hl; h0 < total; h0 += U * step) {
        uint4 x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * step;
            if (h >= total) continue;
            const __nv_bfloat16 *src;
            if (h < p.heads)
                src = static_cast<const __nv_bfloat16 *>(p.q) + t * p.q_row + h * p.q_head;
            else if (h < p.heads + p.kv_heads)
                src = static_cast<const __nv_bfloat16 *>(p.k) + t * p.k_row + (h - p.heads) * p.k_head;
            else
                src = static_cast<const __nv_bfloat16 *>(p.v) + t * p.v_row + (h - p.heads - p.kv_heads) * p.v_head;
            x[u] = *reinterpret_cast<const uint4 *>(src + v0 * 8);
            y[u] = *reinterpret_cast<const uint4 *>(src + v1 * 8);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * step;
            if (h >= total) continue;
            const bool is_v = h >= p.heads + p.kv_heads;
            if (turns && !is_v) rotate(x[u], y[u], c, s, p.interleaved != 0);
            __nv_bfloat16 *dst;
            if (h < p.heads) {
                dst = static_cast<__nv_bfloat16 *>(p.q_out) + t * p.o_row + h * p.o_head;
            } else {
                if (!cached) continue;
                if (!is_v)
                    dst = static_cast<__nv_bfloat16 *>(p.k_cache) + page * p.kc_page + (h - p.heads) * p.kc_head +
                          row * p.kc_row;
                else
                    dst = static_cast<__nv_bfloat16 *>(p.v_cache) + page * p.vc_page +
                          (h - p.heads - p.kv_heads) * p.vc_head + row * p.vc_row;
            }
            *reinterpret_cast<uint4 *>(dst + v0 * 8) = x[u];
            *reinterpret_cast<uint4 *>(dst + v1 * 8) = y[u];
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t s)
{
    const int64_t warps = static_cast<int64_t>(p.T) * p.parts;
    const int per_cta = APPEND_THREADS / 32;
    const int64_t grid = (warps + per_cta - 1) / per_cta;
    return launch_ex(p.head_dim == 128 ? ub_kv_append_kernel<128> : ub_kv_append_kernel<64>, p, static_cast<int>(grid),
                     APPEND_THREADS, 0, 1, p.pdl != 0, s);
}

}  // namespace ubk
