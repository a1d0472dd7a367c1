// Host side of the attention operators declared in include/ub.h (ub_kv_append,
// ub_attn_prompt, ub_attn_decode, ub_attn_tree and their forms for windows and drafts, and
// ub_kv_accept, ub_kv_copy): argument checks, tensor maps, launches. Nothing of the token batch
// (lengths, page table, drafts) is read on the host.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include "ub_attn.h"
#include "ub_attn_host.h"
#include "ub_internal.h"

using namespace ubk;

namespace {

// One stride of a dimension of `extent`: that of a dimension of length 1 is never used, and
// is replaced by one that the tensor maps accept.
bool stride_ok(int64_t *stride, int64_t extent, int64_t unused)
{
    if (extent == 1) {
        *stride = unused;
        return true;
    }
    return *stride > 0 && *stride % 8 == 0 && *stride < (int64_t(1) << 38);
}

int check_heads(const char *fn, const char *name, ub_heads_t *x, int64_t tokens, int heads, int head_dim)
{
    if (!x->data) return fail_call(UB_ERR_ARG, "%s: %s is null", fn, name);
    if (!aligned16(x->data)) return fail_call(UB_ERR_ALIGN, "%s: %s is not 16-byte aligned", fn, name);
    if (!stride_ok(&x->head, heads, head_dim) || !stride_ok(&x->row, tokens, static_cast<int64_t>(heads) * head_dim))
        return fail_call(UB_ERR_ALIGN, "%s: %s has strides [%lld, %lld]: positive multiples of 8 are needed", fn, name,
                         (long long)x->row, (long long)x->head);
    return UB_OK;
}

int check_pages(const char *fn, const char *name, ub_pages_t *x, const ub_attn_t &a)
{
    if (!x->data) return fail_call(UB_ERR_ARG, "%s: %s is null", fn, name);
    if (!aligned16(x->data)) return fail_call(UB_ERR_ALIGN, "%s: %s is not 16-byte aligned", fn, name);
    const int64_t dense = static_cast<int64_t>(a.page_size) * a.head_dim;
    if (!stride_ok(&x->row, a.page_size, a.head_dim) || !stride_ok(&x->head, a.kv_heads, dense) ||
        !stride_ok(&x->page, a.num_pages, dense * a.kv_heads))
        return fail_call(UB_ERR_ALIGN, "%s: %s has strides [%lld, %lld, %lld]: positive multiples of 8 are needed", fn,
                         name, (long long)x->page, (long long)x->head, (long long)x->row);
    return UB_OK;
}

int check_cache_sizes(const char *fn, const ub_attn_t *a)
{
    if (a->page_size < 8 || a->page_size > 256 || (a->page_size & (a->page_size - 1)) != 0)
        return fail_call(UB_ERR_ARG, "%s: page size %d is not a power of two from 8 to 256", fn, a->page_size);
    if (a->num_pages <= 0 || a->table_width <= 0)
        return fail_call(UB_ERR_ZERO, "%s: %lld pages, %lld table entries per sequence", fn, (long long)a->num_pages,
                         (long long)a->table_width);
    if (a->num_pages > INT32_MAX || a->table_width * a->page_size > INT32_MAX - 256 || a->table_width > INT32_MAX)
        return fail_call(UB_ERR_ARG, "%s: cache of %lld pages, table of %lld entries: too large", fn,
                         (long long)a->num_pages, (long long)a->table_width);
    return UB_OK;
}

int check_caches(const char *fn, ub_attn_t *a)
{
    if (int rc = check_pages(fn, "k_cache", &a->k_cache, *a)) return rc;
    return check_pages(fn, "v_cache", &a->v_cache, *a);
}

int check_table(const char *fn, const ub_attn_t &a)
{
    if (!a.kv_lens || !a.page_table) return fail_call(UB_ERR_ARG, "%s: kv_lens or page_table is null", fn);
    if (a.n_seqs > 1 && a.table_row < a.table_width)
        return fail_call(UB_ERR_ARG, "%s: page_table rows of %lld entries, %lld apart", fn, (long long)a.table_width,
                         (long long)a.table_row);
    return UB_OK;
}

// What a row sees besides the causal rule, of at most `keys` keys: *window 0 if that is everything.
int check_window(const char *fn, int32_t window, int32_t sinks, int64_t keys, int *out_window, int *out_sinks)
{
    if (window < 0 || sinks < 0) return fail_call(UB_ERR_ARG, "%s: window %d, sinks %d", fn, window, sinks);
    const bool all = window == 0 || window >= keys || sinks >= keys;
    *out_window = all ? 0 : window;
    *out_sinks = all ? 0 : sinks;
    return UB_OK;
}

// The checks the attention operators share; *a becomes a copy with usable strides.
int check_common(const char *fn, ub_handle_t h, const ub_attn_t *in, bool cache, ub_attn_t *a)
{
    if (!h) return fail_call(UB_ERR_ARG, "null handle");
    if (!in) return fail_call(UB_ERR_ARG, "%s: null arguments", fn);
    if (in->size != sizeof(ub_attn_t))
        return fail_call(UB_ERR_ARG, "%s: argument struct of %u bytes, %zu expected", fn, in->size, sizeof(ub_attn_t));
    *a = *in;
    if (a->n_seqs <= 0 || a->heads <= 0 || a->kv_heads <= 0)
        return fail_call(UB_ERR_ZERO, "%s: %d sequences, %d heads, %d key/value heads", fn, a->n_seqs, a->heads, a->kv_heads);
    if (a->heads % a->kv_heads != 0 || a->heads > 65536)
        return fail_call(UB_ERR_ARG, "%s: %d heads are not a multiple of %d key/value heads", fn, a->heads, a->kv_heads);
    if (a->head_dim != 64 && a->head_dim != 128)
        return fail_call(UB_ERR_ARG, "%s: head dimension %d is neither 64 nor 128", fn, a->head_dim);
    if (!cache) return UB_OK;
    if (int rc = check_cache_sizes(fn, a)) return rc;
    if (int rc = check_table(fn, *a)) return rc;
    return check_caches(fn, a);
}

int check_scale(const char *fn, const ub_attn_t &a)
{
    if (!(a.scale > 0.f) || !isfinite(a.scale)) return fail_call(UB_ERR_ARG, "%s: scale %g", fn, a.scale);
    return UB_OK;
}

SeqBatch batch_of(const ub_attn_t &a, const HandleCall &c)
{
    SeqBatch b;
    memset(&b, 0, sizeof b);
    b.seq_starts = a.seq_starts;
    b.kv_lens = a.kv_lens;
    b.page_table = a.page_table;
    b.table_row = a.table_row;
    b.table_width = static_cast<int>(a.table_width);
    b.num_pages = static_cast<int>(a.num_pages);
    while ((1 << b.page_shift) < a.page_size) ++b.page_shift;
    b.n_seqs = a.n_seqs;
    b.status = c.status;
    return b;
}

int encode_pages(CUtensorMap *map, const ub_pages_t &x, const ub_attn_t &a, int box_rows)
{
    const uint64_t dims[4] = {static_cast<uint64_t>(a.head_dim), static_cast<uint64_t>(a.page_size),
                              static_cast<uint64_t>(a.kv_heads), static_cast<uint64_t>(a.num_pages)};
    const uint64_t strides[4] = {2, static_cast<uint64_t>(x.row) * 2, static_cast<uint64_t>(x.head) * 2,
                                 static_cast<uint64_t>(x.page) * 2};
    const uint32_t box[4] = {64, static_cast<uint32_t>(a.page_size < box_rows ? a.page_size : box_rows), 1, 1};
    return encode_nd(map, x.data, 4, dims, strides, box);
}

// The same with the head dimension as head_dim / 64 times 64 columns, whole in every box.
int encode_pages_whole(CUtensorMap *map, const ub_pages_t &x, const ub_attn_t &a, int box_rows)
{
    const uint64_t dims[5] = {64, static_cast<uint64_t>(a.page_size), static_cast<uint64_t>(a.head_dim / 64),
                              static_cast<uint64_t>(a.kv_heads), static_cast<uint64_t>(a.num_pages)};
    const uint64_t strides[5] = {2, static_cast<uint64_t>(x.row) * 2, 128, static_cast<uint64_t>(x.head) * 2,
                                 static_cast<uint64_t>(x.page) * 2};
    const uint32_t box[5] = {64, static_cast<uint32_t>(a.page_size < box_rows ? a.page_size : box_rows),
                             static_cast<uint32_t>(a.head_dim / 64), 1, 1};
    return encode_nd(map, x.data, 5, dims, strides, box);
}

// Packed tokens [T, heads, head_dim] in boxes of `box_heads` heads by `box_tokens` tokens.
int encode_tokens(CUtensorMap *map, const ub_heads_t &x, int64_t T, int heads, int head_dim, int box_heads, int box_tokens)
{
    const uint64_t dims[3] = {static_cast<uint64_t>(head_dim), static_cast<uint64_t>(heads), static_cast<uint64_t>(T)};
    const uint64_t strides[3] = {2, static_cast<uint64_t>(x.head) * 2, static_cast<uint64_t>(x.row) * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_tokens)};
    return encode_nd(map, x.data, 3, dims, strides, box);
}

int append_call(const char *fn, ub_handle_t h, const ub_attn_t *in, const int32_t *parents, void *stream)
{
    ub_attn_t a;
    if (int rc = check_common(fn, h, in, true, &a)) return rc;
    const int64_t T = handle_tokens(h);
    if (!a.seq_starts) return fail_call(UB_ERR_ARG, "%s: seq_starts is null", fn);
    if (a.rot_dim < 0 || a.rot_dim > a.head_dim || a.rot_dim % 16 != 0)
        return fail_call(UB_ERR_ARG, "%s: rot_dim %d is not a multiple of 16 up to %d", fn, a.rot_dim, a.head_dim);
    if (a.interleaved != 0 && a.interleaved != 1) return fail_call(UB_ERR_ARG, "%s: interleaved must be 0 or 1", fn);
    if (a.rot_dim > 0) {
        if (!a.cos || !a.sin || a.max_pos <= 0) return fail_call(UB_ERR_ARG, "%s: no rotation tables", fn);
        if (!aligned16(a.cos) || !aligned16(a.sin))
            return fail_call(UB_ERR_ALIGN, "%s: rotation tables not 16-byte aligned", fn);
    }
    if (int rc = check_heads(fn, "q", &a.q, T, a.heads, a.head_dim)) return rc;
    if (int rc = check_heads(fn, "k", &a.k, T, a.kv_heads, a.head_dim)) return rc;
    if (int rc = check_heads(fn, "v", &a.v, T, a.kv_heads, a.head_dim)) return rc;
    if (int rc = check_heads(fn, "out", &a.out, T, a.heads, a.head_dim)) return rc;
    DeviceScope g(handle_device(h));
    if (!g.ok) return fail_call(UB_ERR_CUDA, "%s: cannot select the handle's device", fn);
    Range range(fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    HandleCall c;
    if (int rc = handle_call(h, s, &c)) return rc;
    AppendParams p;
    memset(&p, 0, sizeof p);
    p.b = batch_of(a, c);
    p.parents = parents;
    p.q = a.q.data;
    p.k = a.k.data;
    p.v = a.v.data;
    p.q_out = a.out.data;
    p.k_cache = a.k_cache.data;
    p.v_cache = a.v_cache.data;
    p.q_row = a.q.row;
    p.q_head = a.q.head;
    p.k_row = a.k.row;
    p.k_head = a.k.head;
    p.v_row = a.v.row;
    p.v_head = a.v.head;
    p.o_row = a.out.row;
    p.o_head = a.out.head;
    p.kc_page = a.k_cache.page;
    p.kc_head = a.k_cache.head;
    p.kc_row = a.k_cache.row;
    p.vc_page = a.v_cache.page;
    p.vc_head = a.v_cache.head;
    p.vc_row = a.v_cache.row;
    p.cos = a.cos;
    p.sin = a.sin;
    p.max_pos = a.max_pos;
    p.T = static_cast<int>(T);
    p.heads = a.heads;
    p.kv_heads = a.kv_heads;
    p.head_dim = a.head_dim;
    p.rot = a.rot_dim;
    p.interleaved = a.interleaved;
    // Warps per token: one when the tokens alone fill the GPU (32 warps per SM), else enough
    // to do so, at most one per step of the token's heads.
    const int64_t steps = (a.heads + 2 * a.kv_heads + 512 / a.head_dim - 1) / (512 / a.head_dim);
    int64_t parts = (static_cast<int64_t>(c.sms) * 32 + T - 1) / T;
    p.parts = static_cast<int>(parts < steps ? parts : steps);
    p.pdl = c.pdl;
    bool timed = false;
    if (int rc = handle_prof_start(h, UB_OP_KV_APPEND, s, &timed)) return rc;
    const cudaError_t e = launch_kv_append(p, s);
    if (e != cudaSuccess) return cuda_failed(e, "append kernel launch");
    return handle_prof_stop(h, UB_OP_KV_APPEND, s, timed);
}

int prompt_call(const char *fn, ub_handle_t h, const ub_attn_t *in, int32_t window, int32_t sinks, void *stream)
{
    ub_attn_t a;
    const bool paged = in && in->page_size != 0;
    if (int rc = check_common(fn, h, in, paged, &a)) return rc;
    const int64_t T = handle_tokens(h);
    if (!a.seq_starts) return fail_call(UB_ERR_ARG, "%s: seq_starts is null", fn);
    if (int rc = check_scale(fn, a)) return rc;
    if (int rc = check_heads(fn, "q", &a.q, T, a.heads, a.head_dim)) return rc;
    if (!paged) {
        if (int rc = check_heads(fn, "k", &a.k, T, a.kv_heads, a.head_dim)) return rc;
        if (int rc = check_heads(fn, "v", &a.v, T, a.kv_heads, a.head_dim)) return rc;
    }
    if (int rc = check_heads(fn, "out", &a.out, T, a.heads, a.head_dim)) return rc;
    const int64_t keys = paged ? a.table_width * a.page_size : T;
    PromptParams p;
    memset(&p, 0, sizeof p);
    if (int rc = check_window(fn, window, sinks, keys, &p.window, &p.sinks)) return rc;
    DeviceScope g(handle_device(h));
    if (!g.ok) return fail_call(UB_ERR_CUDA, "%s: cannot select the handle's device", fn);
    Range range(fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    HandleCall c;
    if (int rc = handle_call(h, s, &c)) return rc;
    p.group = a.heads / a.kv_heads;
    // The query heads of a key/value head are packed into the rows of a q tile, as many as a
    // power of two of the group allows: they share the tile's keys and values, and a tile of
    // fewer tokens wastes less of the causal diagonal and of a short sequence.
    while (p.pack_shift < 7 && p.group % (2 << p.pack_shift) == 0) ++p.pack_shift;
    const int pack = 1 << p.pack_shift;
    if (int rc = encode_tokens(&p.tmQ, a.q, T, a.heads, a.head_dim, pack, PROMPT_ROWS / pack)) return rc;
    if (paged) {
        if (int rc = encode_pages(&p.tmK, a.k_cache, a, PROMPT_KEYS)) return rc;
        if (int rc = encode_pages(&p.tmV, a.v_cache, a, PROMPT_KEYS)) return rc;
    } else {
        if (int rc = encode_tokens(&p.tmK, a.k, T, a.kv_heads, a.head_dim, 1, PROMPT_KEYS)) return rc;
        if (int rc = encode_tokens(&p.tmV, a.v, T, a.kv_heads, a.head_dim, 1, PROMPT_KEYS)) return rc;
    }
    handle_count_maps(h, 3);
    p.b = batch_of(a, c);
    p.paged = paged ? 1 : 0;
    p.out = a.out.data;
    p.lse = a.lse;
    p.o_row = a.out.row;
    p.o_head = a.out.head;
    p.T = static_cast<int>(T);
    p.heads = a.heads;
    p.kv_heads = a.kv_heads;
    p.head_dim = a.head_dim;
    p.units = a.kv_heads * (p.group >> p.pack_shift);
    p.scale = a.scale;
    p.tickets = c.tickets;
    p.ws = c.ws;
    p.ws_rows = c.ws_rows;
    p.counters = c.piece_counters;
    const size_t slots = c.ws_floats / (2 * PROMPT_ROWS * static_cast<size_t>(a.head_dim));
    p.slots = static_cast<int>(slots < PROMPT_SLOTS ? slots : PROMPT_SLOTS);
    p.abort_word = c.abort_word;
    p.timeout_ns = c.timeout_ns;
    p.epoch = c.epoch;
    p.pdl = c.pdl;
    // One persistent CTA per SM, no more than there can be work items, unless they may have to
    // be split over their keys.
    const int64_t tokens = PROMPT_ROWS / pack;
    const int64_t most = (T / tokens + (a.n_seqs < T ? a.n_seqs : T)) * p.units;
    const int64_t grid = most < c.sms && keys <= PROMPT_WHOLE_KEYS ? most : c.sms;
    bool timed = false;
    if (int rc = handle_prof_start(h, UB_OP_ATTN_PROMPT, s, &timed)) return rc;
    const cudaError_t e = launch_attn_prompt(p, static_cast<int>(grid), s);
    if (e != cudaSuccess) return cuda_failed(e, "prompt attention kernel launch");
    return handle_prof_stop(h, UB_OP_ATTN_PROMPT, s, timed);
}

int decode_call(const char *fn, ub_handle_t h, const ub_attn_t *in, int32_t window, int32_t sinks, void *stream)
{
    ub_attn_t a;
    if (int rc = check_common(fn, h, in, true, &a)) return rc;
    const int64_t T = handle_tokens(h);
    if (int rc = check_scale(fn, a)) return rc;
    if (a.n_seqs > T)
        return fail_call(UB_ERR_CAPACITY, "%s: %d sequences exceed the %lld active tokens", fn, a.n_seqs, (long long)T);
    if (int rc = check_heads(fn, "q", &a.q, T, a.heads, a.head_dim)) return rc;
    if (int rc = check_heads(fn, "out", &a.out, T, a.heads, a.head_dim)) return rc;
    DecodeParams p;
    memset(&p, 0, sizeof p);
    if (int rc = check_window(fn, window, sinks, a.table_width * a.page_size, &p.window, &p.sinks)) return rc;
    DeviceScope g(handle_device(h));
    if (!g.ok) return fail_call(UB_ERR_CUDA, "%s: cannot select the handle's device", fn);
    Range range(fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    HandleCall c;
    if (int rc = handle_call(h, s, &c)) return rc;
    if (int rc = encode_pages_whole(&p.tmK, a.k_cache, a, DECODE_KEYS)) return rc;
    if (int rc = encode_pages_whole(&p.tmV, a.v_cache, a, DECODE_KEYS)) return rc;
    handle_count_maps(h, 2);
    p.b = batch_of(a, c);
    p.q = a.q.data;
    p.out = a.out.data;
    p.lse = a.lse;
    p.q_row = a.q.row;
    p.q_head = a.q.head;
    p.o_row = a.out.row;
    p.o_head = a.out.head;
    p.heads = a.heads;
    p.kv_heads = a.kv_heads;
    p.head_dim = a.head_dim;
    p.group = a.heads / a.kv_heads;
    p.head_blocks = (p.group + DECODE_HEADS - 1) / DECODE_HEADS;
    p.scale = a.scale;
    p.ws = c.ws;
    p.counters = c.join_counters;
    p.times = c.join_counters + c.join_words / DECODE_COUNTERS;
    p.abort_word = c.abort_word;
    p.timeout_ns = c.timeout_ns;
    p.epoch = c.epoch;
    p.pdl = c.pdl;
    // As many CTAs as fit, and no more than there can be tiles.
    int64_t grid = static_cast<int64_t>(c.sms) * DECODE_CTAS_PER_SM;
    const int64_t most = ((a.table_width * a.page_size + DECODE_KEYS - 1) / DECODE_KEYS) * a.n_seqs * a.kv_heads * p.head_blocks;
    p.many_tiles = most > INT32_MAX / (1 + DECODE_ITEM_COST) ? 1 : 0;
    if (grid > most) grid = most;
    if (DECODE_COUNTERS * grid > c.join_words || DECODE_SLOTS * grid * decode_slot_floats(a.head_dim) > static_cast<int64_t>(c.ws_floats))
        return fail_call(UB_ERR_ARG, "%s: workspace too small for %lld CTAs", fn, (long long)grid);
    bool timed = false;
    if (int rc = handle_prof_start(h, UB_OP_ATTN_DECODE, s, &timed)) return rc;
    const cudaError_t e = launch_attn_decode(p, static_cast<int>(grid), s);
    if (e != cudaSuccess) return cuda_failed(e, "decode attention kernel launch");
    return handle_prof_stop(h, UB_OP_ATTN_DECODE, s, timed);
}

int tree_call(const char *fn, ub_handle_t h, const ub_attn_t *in, const int32_t *parents, int32_t window, int32_t sinks,
              void *stream)
{
    ub_attn_t a;
    if (int rc = check_common(fn, h, in, true, &a)) return rc;
    const int64_t T = handle_tokens(h);
    if (!a.seq_starts || !parents) return fail_call(UB_ERR_ARG, "%s: seq_starts or parents is null", fn);
    if (int rc = check_scale(fn, a)) return rc;
    if (int rc = check_heads(fn, "q", &a.q, T, a.heads, a.head_dim)) return rc;
    if (int rc = check_heads(fn, "out", &a.out, T, a.heads, a.head_dim)) return rc;
    const int64_t keys = a.table_width * a.page_size;
    TreeParams p;
    memset(&p, 0, sizeof p);
    if (int rc = check_window(fn, window, sinks, keys, &p.window, &p.sinks)) return rc;
    DeviceScope g(handle_device(h));
    if (!g.ok) return fail_call(UB_ERR_CUDA, "%s: cannot select the handle's device", fn);
    Range range(fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    HandleCall c;
    if (int rc = handle_call(h, s, &c)) return rc;
    // All query heads of a key/value head share a q tile, in even sets where they are more than
    // its rows: they share its keys and values.
    p.group = a.heads / a.kv_heads;
    p.blocks = (p.group + TREE_ROWS - 1) / TREE_ROWS;
    p.unit_heads = (p.group + p.blocks - 1) / p.blocks;
    p.units = a.kv_heads * p.blocks;
    p.tokens = TREE_ROWS / p.unit_heads;
    if (int rc = encode_tokens(&p.tmQ, a.q, T, a.heads, a.head_dim, p.unit_heads, p.tokens)) return rc;
    if (int rc = encode_pages(&p.tmK, a.k_cache, a, TREE_KEYS)) return rc;
    if (int rc = encode_pages(&p.tmV, a.v_cache, a, TREE_KEYS)) return rc;
    handle_count_maps(h, 3);
    p.b = batch_of(a, c);
    p.parents = parents;
    p.out = a.out.data;
    p.lse = a.lse;
    p.o_row = a.out.row;
    p.o_head = a.out.head;
    p.T = static_cast<int>(T);
    p.heads = a.heads;
    p.kv_heads = a.kv_heads;
    p.head_dim = a.head_dim;
    p.scale = a.scale;
    p.ws = c.ws;  // and on into ws_rows
    p.counters = c.join_counters;
    p.times = c.join_counters + c.join_words / DECODE_COUNTERS;
    p.abort_word = c.abort_word;
    p.timeout_ns = c.timeout_ns;
    p.epoch = c.epoch;
    p.pdl = c.pdl;
    // As many CTAs as fit, and no more than there can be key tiles.
    int64_t grid = c.sms < TREE_MOST_CTAS ? c.sms : TREE_MOST_CTAS;
    const int64_t items = (T / (2 * p.tokens) + (a.n_seqs < T ? a.n_seqs : T)) * p.units;
    const int64_t tiles = (keys + TREE_KEYS - 1) / TREE_KEYS;
    const int64_t q_tiles = (T / p.tokens + (a.n_seqs < T ? a.n_seqs : T)) * p.units;
    if (q_tiles <= grid && q_tiles * tiles < grid) grid = q_tiles * tiles;
    p.many_units = items > INT32_MAX / TREE_MOST_UNITS / (tiles + 1) ? 1 : 0;
    const int64_t room = static_cast<int64_t>(c.ws_floats) + 512 * PROMPT_SLOTS;
    if (DECODE_COUNTERS * grid > c.join_words || TREE_SLOTS * grid * tree_slot_floats(a.head_dim) > room)
        return fail_call(UB_ERR_ARG, "%s: workspace too small for %lld CTAs", fn, (long long)grid);
    bool timed = false;
    if (int rc = handle_prof_start(h, UB_OP_ATTN_TREE, s, &timed)) return rc;
    const cudaError_t e = launch_attn_tree(p, static_cast<int>(grid), s);
    if (e != cudaSuccess) return cuda_failed(e, "tree attention kernel launch");
    return handle_prof_stop(h, UB_OP_ATTN_TREE, s, timed);
}

// The caches of ub_kv_copy and ub_kv_accept: the fields of ub_attn_t that describe them.
int check_cache_call(const char *fn, ub_handle_t h, const ub_attn_t *in, ub_attn_t *a)
{
    if (!h) return fail_call(UB_ERR_ARG, "null handle");
    if (!in) return fail_call(UB_ERR_ARG, "%s: null arguments", fn);
    if (in->size != sizeof(ub_attn_t))
        return fail_call(UB_ERR_ARG, "%s: argument struct of %u bytes, %zu expected", fn, in->size, sizeof(ub_attn_t));
    *a = *in;
    if (a->kv_heads <= 0) return fail_call(UB_ERR_ZERO, "%s: %d key/value heads", fn, a->kv_heads);
    if (a->kv_heads > 65536) return fail_call(UB_ERR_ARG, "%s: %d key/value heads", fn, a->kv_heads);
    if (a->head_dim != 64 && a->head_dim != 128)
        return fail_call(UB_ERR_ARG, "%s: head dimension %d is neither 64 nor 128", fn, a->head_dim);
    return UB_OK;
}

int log2_of(int x)
{
    int shift = 0;
    while ((1 << shift) < x) ++shift;
    return shift;
}

template <typename P>
void set_caches(P *p, const ub_attn_t &a)
{
    p->k_cache = a.k_cache.data;
    p->v_cache = a.v_cache.data;
    p->kc_page = a.k_cache.page;
    p->kc_head = a.k_cache.head;
    p->kc_row = a.k_cache.row;
    p->vc_page = a.v_cache.page;
    p->vc_head = a.v_cache.head;
    p->vc_row = a.v_cache.row;
    p->kv_heads = a.kv_heads;
    p->head_dim = a.head_dim;
}

}  // namespace

extern "C" {

int ub_kv_append(ub_handle_t h, const ub_attn_t *a, void *stream) { return append_call("ub_kv_append", h, a, nullptr, stream); }

int ub_kv_append_tree(ub_handle_t h, const ub_attn_t *a, const int32_t *parents, void *stream)
{
    if (h && a && !parents) return fail_call(UB_ERR_ARG, "ub_kv_append_tree: parents is null");
    return append_call("ub_kv_append_tree", h, a, parents, stream);
}

int ub_attn_prompt(ub_handle_t h, const ub_attn_t *a, void *stream) { return prompt_call("ub_attn_prompt", h, a, 0, 0, stream); }

int ub_attn_prompt_window(ub_handle_t h, const ub_attn_t *a, int32_t window, int32_t sinks, void *stream)
{
    return prompt_call("ub_attn_prompt_window", h, a, window, sinks, stream);
}

int ub_attn_decode(ub_handle_t h, const ub_attn_t *a, void *stream) { return decode_call("ub_attn_decode", h, a, 0, 0, stream); }

int ub_attn_decode_window(ub_handle_t h, const ub_attn_t *a, int32_t window, int32_t sinks, void *stream)
{
    return decode_call("ub_attn_decode_window", h, a, window, sinks, stream);
}

int ub_attn_tree(ub_handle_t h, const ub_attn_t *a, const int32_t *parents, int32_t window, int32_t sinks, void *stream)
{
    return tree_call("ub_attn_tree", h, a, parents, window, sinks, stream);
}

int ub_kv_copy(ub_handle_t h, const ub_attn_t *in, const int32_t *pairs, int64_t n_pairs, void *stream)
{
    static const char *fn = "ub_kv_copy";
    ub_attn_t a;
    if (int rc = check_cache_call(fn, h, in, &a)) return rc;
    a.table_width = 1;  // no table
    if (int rc = check_cache_sizes(fn, &a)) return rc;
    if (int rc = check_caches(fn, &a)) return rc;
    if (n_pairs < 0 || n_pairs > INT32_MAX) return fail_call(UB_ERR_ARG, "%s: %lld pairs", fn, (long long)n_pairs);
    if (n_pairs == 0) return UB_OK;
    if (!pairs) return fail_call(UB_ERR_ARG, "%s: pairs is null", fn);
    DeviceScope g(handle_device(h));
    if (!g.ok) return fail_call(UB_ERR_CUDA, "%s: cannot select the handle's device", fn);
    Range range(fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    HandleCall c;
    if (int rc = handle_call(h, s, &c)) return rc;
    PageCopyParams p;
    memset(&p, 0, sizeof p);
    set_caches(&p, a);
    p.pairs = pairs;
    p.n = n_pairs;
    p.pages = a.num_pages;
    p.page_shift = log2_of(a.page_size);
    p.status = c.status;
    p.pdl = c.pdl;
    bool timed = false;
    if (int rc = handle_prof_start(h, UB_OP_KV_COPY, s, &timed)) return rc;
    const cudaError_t e = launch_kv_copy(p, s);
    if (e != cudaSuccess) return cuda_failed(e, "page copy kernel launch");
    return handle_prof_stop(h, UB_OP_KV_COPY, s, timed);
}

int ub_kv_accept(ub_handle_t h, const ub_attn_t *in, const int32_t *parents, int64_t n_tokens, const int32_t *leaves,
                 int32_t *new_lens, void *stream)
{
    static const char *fn = "ub_kv_accept";
    ub_attn_t a;
    if (int rc = check_cache_call(fn, h, in, &a)) return rc;
    if (a.n_seqs <= 0) return fail_call(UB_ERR_ZERO, "%s: %d sequences", fn, a.n_seqs);
    if (!a.seq_starts || (!parents && n_tokens > 0) || !leaves || !new_lens)
        return fail_call(UB_ERR_ARG, "%s: a null array", fn);
    if (n_tokens < 0 || n_tokens > INT32_MAX) return fail_call(UB_ERR_ARG, "%s: %lld tokens", fn, (long long)n_tokens);
    if (int rc = check_cache_sizes(fn, &a)) return rc;
    if (int rc = check_table(fn, a)) return rc;
    if (int rc = check_caches(fn, &a)) return rc;
    const Words inputs[] = {words("kv_lens", a.kv_lens, a.n_seqs), words("leaves", leaves, a.n_seqs),
                            words("seq_starts", a.seq_starts, static_cast<int64_t>(a.n_seqs) + 1), words("parents", parents, n_tokens),
                            rows_of("page_table", a.page_table, a.n_seqs, a.table_row, a.table_width)};
    if (int rc = check_apart(fn, words("new_lens", new_lens, a.n_seqs), inputs, 5)) return rc;
    // One cache for keys and values moves once: twice, in CTAs of their own, the one's rows would be
    // loaded from where the other has stored.
    const bool one = a.k_cache.data == a.v_cache.data;
    if (one && (a.k_cache.page != a.v_cache.page || a.k_cache.head != a.v_cache.head || a.k_cache.row != a.v_cache.row))
        return fail_call(UB_ERR_ARG, "%s: k_cache and v_cache are two views of one array", fn);
    if (static_cast<int64_t>(a.n_seqs) * ((2 * static_cast<int64_t>(a.kv_heads) * a.head_dim / 8 + 127) / 128) > INT32_MAX)
        return fail_call(UB_ERR_ARG, "%s: %d sequences of %d heads are too many", fn, a.n_seqs, a.kv_heads);
    DeviceScope g(handle_device(h));
    if (!g.ok) return fail_call(UB_ERR_CUDA, "%s: cannot select the handle's device", fn);
    Range range(fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    HandleCall c;
    if (int rc = handle_call(h, s, &c)) return rc;
    AcceptParams p;
    memset(&p, 0, sizeof p);
    p.b = batch_of(a, c);
    set_caches(&p, a);
    p.parents = parents;
    p.leaves = leaves;
    p.new_lens = new_lens;
    p.tokens = static_cast<int>(n_tokens);
    p.caches = one ? 1 : 2;
    p.pdl = c.pdl;
    bool timed = false;
    if (int rc = handle_prof_start(h, UB_OP_KV_ACCEPT, s, &timed)) return rc;
    const cudaError_t e = launch_kv_accept(p, s);
    if (e != cudaSuccess) return cuda_failed(e, "accept kernel launch");
    return handle_prof_stop(h, UB_OP_KV_ACCEPT, s, timed);
}

}  // extern "C"
