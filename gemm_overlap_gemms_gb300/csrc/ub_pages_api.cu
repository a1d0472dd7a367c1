// Host side of the page operators declared in include/ub.h (ub_kv_take, ub_kv_free, ub_kv_fork,
// ub_kv_compact): argument checks and launches. Tables and counts are read on the device only.
#include <string.h>

#include "ub_attn.h"
#include "ub_attn_host.h"
#include "ub_internal.h"

using namespace ubk;

namespace {

int check_rows(const char *fn, const char *what, int64_t rows, int64_t row, int64_t width)
{
    if (rows > 1 && (row < width || row > INT32_MAX))
        return fail_call(UB_ERR_ARG, "%s: %s rows of %lld entries, %lld apart", fn, what, (long long)width, (long long)row);
    if (rows > INT32_MAX || rows * width > INT32_MAX)
        return fail_call(UB_ERR_ARG, "%s: %s of %lld rows of %lld entries is too large", fn, what, (long long)rows, (long long)width);
    return UB_OK;
}

Words refs_of(const ub_pool_t &in) { return words("refs", in.refs, in.num_pages); }
Words table_of(const ub_pool_t &in)
{
    return rows_of("page_table", in.page_table, in.n_seqs, in.table_row, in.table_width);
}

int check_pool(const char *fn, ub_handle_t h, const ub_pool_t *in)
{
    if (!h) return fail_call(UB_ERR_ARG, "null handle");
    if (!in) return fail_call(UB_ERR_ARG, "%s: null arguments", fn);
    if (in->size != sizeof(ub_pool_t))
        return fail_call(UB_ERR_ARG, "%s: argument struct of %u bytes, %zu expected", fn, in->size, sizeof(ub_pool_t));
    if (in->n_seqs <= 0 || in->num_pages <= 0 || in->table_width <= 0)
        return fail_call(UB_ERR_ZERO, "%s: %d sequences, %lld pages, %lld table entries per sequence", fn, in->n_seqs,
                         (long long)in->num_pages, (long long)in->table_width);
    if (in->page_size < 8 || in->page_size > 256 || (in->page_size & (in->page_size - 1)) != 0)
        return fail_call(UB_ERR_ARG, "%s: page size %d is not a power of two from 8 to 256", fn, in->page_size);
    if (!in->refs || !in->page_table) return fail_call(UB_ERR_ARG, "%s: refs or page_table is null", fn);
    if (in->num_pages > INT32_MAX || in->table_width > INT32_MAX || in->table_width * in->page_size > INT32_MAX - 256)
        return fail_call(UB_ERR_ARG, "%s: pool of %lld pages, table of %lld entries: too large", fn, (long long)in->num_pages,
                         (long long)in->table_width);
    if (int rc = check_rows(fn, "page_table", in->n_seqs, in->table_row, in->table_width)) return rc;
    const Words table = table_of(*in);
    return check_apart(fn, refs_of(*in), &table, 1);
}

// The device and the handle's state, the launch, and its timing.
int run(const char *fn, ub_handle_t h, PoolOp op, const ub_pool_t &in, PoolParams *p, int64_t list_words, void *stream)
{
    DeviceScope g(handle_device(h));
    if (!g.ok) return fail_call(UB_ERR_CUDA, "%s: cannot select the handle's device", fn);
    Range range(fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    HandleCall c;
    if (int rc = handle_call(h, s, &c)) return rc;
    if (list_words > static_cast<int64_t>(c.ws_floats))
        return fail_call(UB_ERR_ARG, "%s: pool of %lld pages: the workspace holds %zu words", fn, (long long)in.num_pages, c.ws_floats);
    p->refs = in.refs;
    p->table = in.page_table;
    p->table_row = in.table_row;
    p->width = in.table_width;
    p->pages = in.num_pages;
    p->rows = in.n_seqs;
    while ((1 << p->page_shift) < in.page_size) ++p->page_shift;
    p->list = reinterpret_cast<int32_t *>(c.ws);
    p->status = c.status;
    p->pdl = c.pdl;
    bool timed = false;
    if (int rc = handle_prof_start(h, UB_OP_KV_PAGES, s, &timed)) return rc;
    const cudaError_t e = launch_pool(op, *p, c.sms, s);
    if (e != cudaSuccess) return cuda_failed(e, "page kernel launch");
    return handle_prof_stop(h, UB_OP_KV_PAGES, s, timed);
}

int rows_call(const char *fn, ub_handle_t h, PoolOp op, const ub_pool_t *in, const int32_t *begin, const int32_t *end, void *stream)
{
    if (int rc = check_pool(fn, h, in)) return rc;
    if (!begin || !end) return fail_call(UB_ERR_ARG, "%s: begin or end is null", fn);
    const Words inputs[] = {words("begin", begin, in->n_seqs), words("end", end, in->n_seqs)};
    if (int rc = check_apart(fn, refs_of(*in), inputs, 2)) return rc;
    if (int rc = check_apart(fn, table_of(*in), inputs, 2)) return rc;
    PoolParams p;
    memset(&p, 0, sizeof p);
    p.n = in->n_seqs;
    p.begin = begin;
    p.end = end;
    return run(fn, h, op, *in, &p, op == PoolOp::take ? in->num_pages : 0, stream);
}

}  // namespace

extern "C" {

int ub_kv_take(ub_handle_t h, const ub_pool_t *pool, const int32_t *begin, const int32_t *end, void *stream)
{
    return rows_call("ub_kv_take", h, PoolOp::take, pool, begin, end, stream);
}

int ub_kv_free(ub_handle_t h, const ub_pool_t *pool, const int32_t *begin, const int32_t *end, void *stream)
{
    return rows_call("ub_kv_free", h, PoolOp::free, pool, begin, end, stream);
}

int ub_kv_fork(ub_handle_t h, const ub_pool_t *pool, const int32_t *kv_lens, const int32_t *source, int64_t n_children,
               int32_t *new_table, int64_t new_row, int32_t *copies, void *stream)
{
    static const char *fn = "ub_kv_fork";
    if (int rc = check_pool(fn, h, pool)) return rc;
    if (n_children < 0) return fail_call(UB_ERR_ARG, "%s: %lld children", fn, (long long)n_children);
    if (n_children == 0) return UB_OK;
    if (!kv_lens || !source || !new_table || !copies) return fail_call(UB_ERR_ARG, "%s: a null array", fn);
    if (int rc = check_rows(fn, "new_table", n_children, new_row, pool->table_width)) return rc;
    const Words arrays[] = {table_of(*pool),
                            refs_of(*pool),
                            words("kv_lens", kv_lens, pool->n_seqs),
                            words("source", source, n_children),
                            rows_of("new_table", new_table, n_children, new_row, pool->table_width)};
    if (int rc = check_apart(fn, arrays[1], arrays + 2, 2)) return rc;  // (lengths and sources are read twice)
    if (int rc = check_apart(fn, arrays[4], arrays, 4)) return rc;
    if (int rc = check_apart(fn, words("copies", copies, 2 * n_children), arrays, 5)) return rc;
    PoolParams p;
    memset(&p, 0, sizeof p);
    p.n = n_children;
    p.begin = kv_lens;
    p.source = source;
    p.new_table = new_table;
    p.new_row = new_row;
    p.pairs = copies;
    return run(fn, h, PoolOp::fork, *pool, &p, pool->num_pages, stream);
}

int ub_kv_compact(ub_handle_t h, const ub_pool_t *pool, int32_t *refs_out, int32_t *table_out, int64_t out_row,
                  int32_t *moves, int64_t n_moves, int32_t *used, void *stream)
{
    static const char *fn = "ub_kv_compact";
    if (int rc = check_pool(fn, h, pool)) return rc;
    if (!refs_out || !table_out || !used || (!moves && n_moves > 0)) return fail_call(UB_ERR_ARG, "%s: a null array", fn);
    if (n_moves < pool->num_pages / 2 || n_moves > INT32_MAX)
        return fail_call(UB_ERR_ARG, "%s: room for %lld moves of %lld pages: half as many are needed", fn, (long long)n_moves,
                         (long long)pool->num_pages);
    if (int rc = check_rows(fn, "table_out", pool->n_seqs, out_row, pool->table_width)) return rc;
    // refs_out and table_out may be refs and page_table, whole.
    const bool same_table = table_out == pool->page_table && (pool->n_seqs == 1 || out_row == pool->table_row);
    const Words refs = refs_of(*pool), to_refs = words("refs_out", refs_out, pool->num_pages), table = table_of(*pool);
    const Words to_table = rows_of("table_out", table_out, pool->n_seqs, out_row, pool->table_width);
    const Words arrays[] = {refs, table, to_refs, to_table, words("moves", moves, 2 * n_moves)};
    if (refs_out != pool->refs)
        if (int rc = check_apart(fn, to_refs, &refs, 1)) return rc;
    if (!same_table)
        if (int rc = check_apart(fn, to_table, &table, 1)) return rc;
    if (int rc = check_apart(fn, to_refs, &table, 1)) return rc;
    if (int rc = check_apart(fn, to_table, &refs, 1)) return rc;
    if (int rc = check_apart(fn, to_table, &to_refs, 1)) return rc;
    if (int rc = check_apart(fn, arrays[4], arrays, 4)) return rc;
    if (int rc = check_apart(fn, words("used", used, 1), arrays, 5)) return rc;
    PoolParams p;
    memset(&p, 0, sizeof p);
    p.n = n_moves;
    p.refs_out = refs_out;
    p.new_table = table_out;
    p.new_row = out_row;
    p.pairs = moves;
    p.used = used;
    return run(fn, h, PoolOp::compact, *pool, &p, 2 * pool->num_pages, stream);
}

}  // extern "C"
