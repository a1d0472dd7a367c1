"""The attention operators against their 64-bit definitions: append to a paged cache,
prompt attention (packed and over the cache), decode attention."""
import math

import pytest
import torch

import attn_ref as ref
from gemm_overlap_gemms_gb300 import ub
from gpu_helpers import is_sentinel, sentinel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def buf():
    from gemm_overlap_gemms_gb300 import _build
    _build.build()
    with ub.UserBuffer([16384, 256], 1) as b:
        yield b


def ok(buf):
    torch.cuda.synchronize()
    assert buf.query_status() == ub.UB_OK


def slices(b, heads, kv_heads, dim, std=1.0):
    """q, k, v as views of one QKV output row per token."""
    y = b.randn(b.T, heads + 2 * kv_heads, dim, std=std)
    return y[:, :heads], y[:, heads:heads + kv_heads], y[:, heads + kv_heads:]


# ---------------------------------------------------------------- decode

def check_decode(buf, b, q, out, lse, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    for s, n in enumerate(b.kv):
        last = torch.tensor([n - 1], device=q.device)
        o, e, ll, le = ref.attend(q[s:s + 1], b.rows(b.k_cache, s), b.rows(b.v_cache, s), last, scale)
        ref.within(out[s:s + 1], o, e, "sequence %d of %d keys" % (s, n))
        if lse is not None:
            ref.within(lse[s:s + 1], ll, le, "lse of sequence %d" % s)
    assert is_sentinel(out[len(b.kv):])


def run_decode(buf, b, heads, dim, std=1.5, **kw):
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, heads, dim, std=std)
    out = sentinel((b.T, heads, dim))
    out, lse = buf.attn_decode(q, b.k_cache, b.v_cache, b.lens, b.table, out=out, lse=True, **kw)
    ok(buf)
    check_decode(buf, b, q, out, lse, kw.get("scale"))
    return q, out


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (8, 1), (12, 4), (16, 1), (40, 2), (5, 5), (9, 1)])
def test_decode_heads(buf, dim, heads, kv_heads):
    kv = [1, 31, 32, 33, 0, 500, 129, 64]
    b = ref.Batch([1] * len(kv), kv, page=16, kv_heads=kv_heads, dim=dim, pad=3, seed=heads, fill=float("nan"))
    run_decode(buf, b, heads, dim)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_decode_pages(buf, page):
    kv = [1, page - 1, page, page + 1, 3 * page + 5, 700]
    b = ref.Batch([1] * len(kv), kv, page=page, kv_heads=2, dim=128, seed=page, fill=float("inf"))
    run_decode(buf, b, 8, 128)


@pytest.mark.parametrize("kv", [[0], [0, 0, 0], [1], [40000], [70001, 3], [9000, 1, 0, 12000], list(range(0, 400, 3)),
                                [17] * 1000])
def test_decode_lengths(buf, kv):
    b = ref.Batch([1] * len(kv), kv, page=64, kv_heads=1, dim=128, seed=len(kv), fill=float("nan"))
    run_decode(buf, b, 8, 128)


@pytest.mark.parametrize("heads,kv_heads,kv", [(5, 5, [1 + 7 * i % 30 for i in range(71)]), (8, 8, [17 + 13 * i % 53 for i in range(49)]),
                                               (12, 4, [0, 5, 0, 300, 33, 0] * 13), (12, 1, [2900 - i for i in range(15)]),
                                               (4, 1, [1500 + i for i in range(140)]), (16, 2, [0] * 30 + [3000])])
def test_decode_items_and_ctas(buf, heads, kv_heads, kv):
    """A CTA for every item of about the same length or of a tile or two; equal shares of others."""
    b = ref.Batch([1] * len(kv), kv, page=64, kv_heads=kv_heads, dim=128, seed=heads, fill=float("nan"))
    run_decode(buf, b, heads, 128)


def test_decode_grids_of_different_sizes_share_the_counters(buf):
    """A call's grid follows the table's width; what one call leaves counted must not meet another's."""
    long = ref.Batch([1] * 20, [700 + 97 * i % 1900 for i in range(20)], page=64, kv_heads=2, dim=128, seed=1, fill=float("nan"))
    buf.set_active_shape([20, 256])
    ql = long.randn(20, 8, 128)
    before = buf.attn_decode(ql, long.k_cache, long.v_cache, long.lens, long.table)
    for pages in range(13, 76):
        b = ref.Batch([1], [64 * pages], page=64, kv_heads=1, dim=64, seed=pages, fill=float("nan"))
        buf.set_active_shape([1, 256])
        buf.attn_decode(b.randn(1, 4, 64), b.k_cache, b.v_cache, b.lens, b.table)
    buf.set_active_shape([20, 256])
    after = buf.attn_decode(ql, long.k_cache, long.v_cache, long.lens, long.table)
    ok(buf)
    assert torch.equal(before, after)


def test_a_page_table_as_wide_as_it_may_be(buf):
    """The work that such a table could hold passes 32 bits; what the lengths ask for is small."""
    b = ref.Batch([1] * 3, [5000, 0, 300], page=256, kv_heads=8, dim=64, seed=7, fill=float("nan"))
    wide = torch.full((3, 8388600), -1, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = b.table
    narrow, b.table = b.table, wide
    q, out = run_decode(buf, b, 16, 64)
    assert torch.equal(out, buf.attn_decode(q, b.k_cache, b.v_cache, b.lens, narrow))
    out = sentinel(q.shape)
    _, lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, wide, out=out, lse=True)
    ok(buf)
    check_prompt(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, lse)


def test_decode_is_deterministic_and_leaves_its_counters_clean(buf):
    b = ref.Batch([1] * 3, [30000, 5000, 11], page=32, kv_heads=2, dim=64, seed=5)
    q, first = run_decode(buf, b, 8, 64)
    for _ in range(3):
        again = buf.attn_decode(q, b.k_cache, b.v_cache, b.lens, b.table)
        assert torch.equal(again, first)


@pytest.mark.parametrize("kv_heads,page", [(2, 16), (1, 64)])
def test_decode_back_to_back(buf, kv_heads, page):
    """Many launches in flight over two batches, their loads landing in any order: every result the same."""
    gen = torch.Generator().manual_seed(kv_heads)
    kv = torch.randint(128, 4096, (64,), generator=gen).tolist()
    runs = []
    for seed in (1, 2):
        b = ref.Batch([1] * 64, kv, page=page, kv_heads=kv_heads, dim=128, seed=seed)
        runs.append((b,) + run_decode(buf, b, 8, 128))
    outs = [torch.empty_like(runs[0][2]) for _ in range(100)]
    for i, out in enumerate(outs):
        b, q, _ = runs[i % 2]
        buf.attn_decode(q, b.k_cache, b.v_cache, b.lens, b.table, out=out)
    ok(buf)
    for i, out in enumerate(outs):
        assert torch.equal(out, runs[i % 2][2]), i


def test_decode_large_scores_and_scale(buf):
    b = ref.Batch([1] * 2, [300, 77], page=16, kv_heads=1, dim=128, seed=6)
    b.k_cache.mul_(8)
    run_decode(buf, b, 8, 128, std=8.0, scale=0.3)


def test_decode_strided_views(buf):
    """Cache rows laid out token by token, keys and values interleaved; strided q and out; a wide table."""
    b = ref.Batch([1] * 3, [100, 37, 64], page=32, kv_heads=3, dim=64, seed=7)
    both = torch.zeros(b.pages, 32, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
    both[:, :, 0] = b.k_cache.transpose(1, 2)
    both[:, :, 1] = b.v_cache.transpose(1, 2)
    b.k_cache, b.v_cache = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    wide = torch.full((3, 40), -7, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide[:, :b.table.shape[1]]
    buf.set_active_shape([3, 256])
    q = b.randn(3, 20, 64)[:, 1:19:2]
    big = sentinel((3, 18, 128))
    out = big[:, ::2, 64:]
    buf.attn_decode(q, b.k_cache, b.v_cache, b.lens, b.table, out=out)
    ok(buf)
    check_decode(buf, b, q, out, None)
    assert is_sentinel(big[:, 1::2]) and is_sentinel(big[:, :, :64])


def test_decode_over_a_cache_past_32_bits(buf):
    """A cache of more than 2^32 bytes and 2^31 elements, its last pages in use."""
    pages = (1 << 31) // (64 * 128) + 100
    k = torch.zeros(pages, 1, 64, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    b = ref.Batch([1, 1], [150, 90], page=64, kv_heads=1, dim=128, free=0, seed=8)
    k[pages - b.pages:], v[pages - b.pages:] = b.k_cache, b.v_cache
    b.k_cache, b.v_cache = k, v
    b.table[b.table >= 0] += pages - b.pages
    b.pages = pages
    run_decode(buf, b, 8, 128)


# ---------------------------------------------------------------- append

def check_append(buf, b, heads, kv_heads, dim, rot, interleaved, caches=None, in_place=False):
    buf.set_active_shape([b.T, 256])
    q, k, v = slices(b, heads, kv_heads, dim)
    positions = max(max(b.kv), 1)
    angle = torch.arange(positions, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device="cuda") / max(rot, 1))
    cos, sin = angle.cos().float(), angle.sin().float()
    before = [b.k_cache.clone(), b.v_cache.clone()]
    q0 = q.clone()
    out = q if in_place else sentinel((b.T, heads, dim))
    got = buf.kv_append(q, k, v, cos if rot else None, sin if rot else None, b.starts, b.lens, b.table, b.k_cache,
                        b.v_cache, q_out=out, interleaved=interleaved)
    ok(buf)
    assert got is out
    t0 = 0
    for s, n in enumerate(b.new):
        pos = torch.arange(b.kv[s] - n, b.kv[s], device="cuda")
        c, sn = (cos[pos], sin[pos]) if rot else (cos[:n, :0], sin[:n, :0])
        want, e = ref.rotate(q0[t0:t0 + n], c, sn, interleaved)
        ref.within(out[t0:t0 + n], want, e, "queries of sequence %d" % s)
        page, row = b.table[s].long()[pos // b.page], pos % b.page
        want, e = ref.rotate(k[t0:t0 + n], c, sn, interleaved)
        ref.within(b.k_cache[page, :, row], want, e, "keys of sequence %d" % s)
        assert torch.equal(b.v_cache[page, :, row], v[t0:t0 + n])
        before[0][page, :, row] = b.k_cache[page, :, row]
        before[1][page, :, row] = b.v_cache[page, :, row]
        t0 += n
    assert torch.equal(before[0], b.k_cache) and torch.equal(before[1], b.v_cache)  # nothing else written
    assert torch.equal(out[t0:], q0[t0:]) if in_place else is_sentinel(out[t0:])


@pytest.mark.parametrize("new,kv", [([1], [1]), ([1, 1, 1], [5, 16, 17]), ([3, 0, 40, 1], [3, 9, 77, 128]),
                                    ([700, 1, 333], [700, 600, 999]), ([1] * 100, list(range(1, 101)))])
@pytest.mark.parametrize("heads,kv_heads,dim,rot,interleaved", [
    (8, 8, 128, 128, False), (8, 2, 64, 64, True), (5, 1, 128, 32, False), (6, 3, 64, 16, True), (2, 1, 64, 0, False)])
def test_append(buf, new, kv, heads, kv_heads, dim, rot, interleaved):
    b = ref.Batch(new, kv, page=16, kv_heads=kv_heads, dim=dim, pad=2, seed=len(new))
    check_append(buf, b, heads, kv_heads, dim, rot, interleaved)


@pytest.mark.parametrize("page", [8, 32, 256])
def test_append_in_place_and_pages(buf, page):
    b = ref.Batch([20, 100], [300, 100], page=page, kv_heads=2, dim=128, pad=1, seed=page)
    check_append(buf, b, 4, 2, 128, 64, False, in_place=True)


def test_append_strided_cache(buf):
    b = ref.Batch([20, 3], [50, 3], page=16, kv_heads=2, dim=64, seed=3)
    b.k_cache = b.k_cache.transpose(1, 2).contiguous().transpose(1, 2)
    b.v_cache = torch.cat([b.v_cache, b.v_cache], 3)[..., 64:]
    check_append(buf, b, 4, 2, 64, 64, True)


# ---------------------------------------------------------------- prompt

def check_prompt(b, q, keys, out, lse, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    for s, n in enumerate(b.new):
        t0 = b.starts_list[s]
        k, v = keys(s)
        last = torch.arange(k.shape[1] - n, k.shape[1], device=q.device)
        for a in range(0, n, 2048):
            z = min(n, a + 2048)
            o, e, ll, le = ref.attend(q[t0 + a:t0 + z], k, v, last[a:z], scale)
            ref.within(out[t0 + a:t0 + z], o, e, "sequence %d, rows from %d" % (s, a))
            if lse is not None:
                ref.within(lse[t0 + a:t0 + z], ll, le, "lse of sequence %d" % s)
    assert is_sentinel(out[b.starts_list[-1]:])


def run_packed(buf, b, heads, kv_heads, dim, std=1.5, scale=None, poison=True):
    buf.set_active_shape([b.T, 256])
    q, k, v = slices(b, heads, kv_heads, dim, std)
    if poison:  # the padding rows are nobody's
        for x in (q, k, v):
            x[b.starts_list[-1]:] = float("nan")
    out = sentinel((b.T, heads, dim))
    out, lse = buf.attn_prompt(q, k, v, b.starts, out=out, lse=True, scale=scale)
    ok(buf)
    check_prompt(b, q, lambda s: tuple(x[b.starts_list[s]:b.starts_list[s + 1]].transpose(0, 1) for x in (k, v)), out,
                 lse, scale)
    return q, k, v, out


LENGTHS = [[1], [2, 1, 3], [16], [127], [128], [129], [255, 256, 257], [15, 0, 17, 64, 0], [700, 33, 1, 1300]]


@pytest.mark.parametrize("new", LENGTHS)
@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 128), (8, 1, 128), (6, 2, 64), (12, 1, 64), (3, 1, 128)])
def test_prompt_packed(buf, new, heads, kv_heads, dim):
    b = ref.Batch(new, [0] * len(new), kv_heads=kv_heads, dim=dim, pad=5, seed=len(new))
    run_packed(buf, b, heads, kv_heads, dim)


@pytest.mark.parametrize("tiles", [30, 31, 32, 62, 63, 64])
def test_prompt_packed_longest_of_any_number_of_key_tiles(buf, tiles):
    """The schedule looks items up by their number of key tiles, 32 numbers at a time."""
    b = ref.Batch([128 * tiles - 5, 700, 300], [0] * 3, kv_heads=2, dim=64, seed=tiles)
    run_packed(buf, b, 4, 2, 64)


@pytest.mark.parametrize("tiles", [30, 31, 32, 62, 63, 961, 962, 991, 992, 993, 1023, 1024])
def test_prompt_chunks_of_any_number_of_key_tiles(buf, tiles):
    b = ref.Batch([3, 300, 9], [128 * tiles - 60, 128 * tiles - 128, 700], page=64, kv_heads=1, dim=64, seed=tiles, fill=float("nan"))
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, 2, 64, std=1.5)
    out = sentinel(q.shape)
    _, lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, out=out, lse=True)
    ok(buf)
    check_prompt(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, lse)


def test_prompt_packed_many_sequences(buf):
    new = [(7 * i) % 61 for i in range(300)]
    b = ref.Batch(new, [0] * len(new), kv_heads=2, dim=64, pad=3, seed=1)
    run_packed(buf, b, 4, 2, 64)


def test_prompt_packed_long(buf):
    b = ref.Batch([5000, 3001], [0, 0], kv_heads=2, dim=128, pad=0, seed=1)
    run_packed(buf, b, 8, 2, 128)


def test_prompt_back_to_back(buf):
    """Many launches in flight, items of every length: every result the same."""
    new = [1900, 3, 130, 700, 64, 2000, 17, 128, 950]
    b = ref.Batch(new, [0] * len(new), kv_heads=2, dim=128, pad=0, seed=1)
    q, k, v, first = run_packed(buf, b, 8, 2, 128)
    outs = [torch.empty_like(first) for _ in range(60)]
    for out in outs:
        buf.attn_prompt(q, k, v, b.starts, out=out)
    ok(buf)
    assert all(torch.equal(out, first) for out in outs)


def test_prompt_growing_scores(buf):
    """Scores that grow along the keys, so that the running maximum moves at every tile."""
    b = ref.Batch([900], [0], kv_heads=1, dim=128, seed=2)
    buf.set_active_shape([900, 256])
    q, k, v = slices(b, 2, 1, 128)
    k *= torch.linspace(0.1, 12, 900, device="cuda")[:, None, None].bfloat16()
    out, lse = buf.attn_prompt(q, k, v, b.starts, lse=True, scale=0.7)
    ok(buf)
    check_prompt(b, q, lambda s: (k.transpose(0, 1), v.transpose(0, 1)), out, lse, 0.7)


def test_prompt_neighbour_of_nan(buf):
    """A sequence of NaNs poisons no row of its neighbours."""
    b = ref.Batch([37, 70, 45], [0, 0, 0], kv_heads=1, dim=128, seed=3)
    buf.set_active_shape([b.T, 256])
    q, k, v = slices(b, 2, 1, 128)
    for x in (q, k, v):
        x[37:107] = float("nan")
    out = buf.attn_prompt(q, k, v, b.starts)
    ok(buf)
    for t0, t1 in ((0, 37), (107, 152)):
        o, e, _, _ = ref.attend(q[t0:t1], k[t0:t1].transpose(0, 1), v[t0:t1].transpose(0, 1),
                                torch.arange(t1 - t0, device="cuda"), 128 ** -0.5)
        ref.within(out[t0:t1], o, e, "rows %d to %d" % (t0, t1))
    assert out[37:107].isnan().all()


@pytest.mark.parametrize("page", [8, 16, 64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 4, 128), (8, 1, 64), (12, 4, 128)])
def test_prompt_paged(buf, page, heads, kv_heads, dim):
    new, kv = [1, 5, 130, 0, 300, 17], [1, 400, 130, 9, 1000, 16]  # the last: fewer keys than tokens
    b = ref.Batch(new, kv, page=page, kv_heads=kv_heads, dim=dim, pad=2, seed=page, fill=float("nan"))
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, heads, dim, std=1.5)
    out = sentinel((b.T, heads, dim))
    out, lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, out=out, lse=True)
    ok(buf)
    check_prompt(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, lse)


@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 128), (8, 1, 64), (6, 3, 128)])
@pytest.mark.parametrize("new,kv", [([40, 1, 300], [9000, 5001, 300]), ([1], [20000]), ([700, 3, 16], [2500, 1030, 16]),
                                    ([130, 0, 129], [6000, 50, 4097])])
def test_prompt_chunks_over_long_caches(buf, new, kv, heads, kv_heads, dim):
    """Few tokens over many cached keys: items split over their keys and joined."""
    b = ref.Batch(new, kv, page=32, kv_heads=kv_heads, dim=dim, pad=1, seed=heads, fill=float("nan"))
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, heads, dim, std=1.5)
    out = sentinel((b.T, heads, dim))
    out, lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, out=out, lse=True)
    ok(buf)
    check_prompt(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, lse)
    for _ in range(5):
        assert torch.equal(buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table)[:sum(new)], out[:sum(new)])


def test_prompt_split_plans_one_after_another(buf):
    """Calls that split differently, back to back, on the same workspace and counters."""
    calls = []
    for i, (new, kv) in enumerate([([64, 64], [2000, 1999]), ([5], [30000]), ([300, 1], [1409, 1500]), ([17] * 3, [6000, 0, 40])]):
        b = ref.Batch(new, kv, page=64, kv_heads=2, dim=(64, 128)[i % 2], seed=i, fill=float("nan"))
        q = b.randn(b.T, 4, b.k_cache.shape[3], std=1.5)
        out = sentinel(q.shape)
        calls.append((b, q, out))
    for _ in range(3):
        for b, q, out in calls:
            buf.set_active_shape([b.T, 256])
            buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, out=out)
    ok(buf)
    for b, q, out in calls:
        buf.set_active_shape([b.T, 256])
        _, lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, out=out, lse=True)
        check_prompt(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, lse)


def test_prompt_packed_split(buf):
    b = ref.Batch([3000, 129, 2500, 17], [0] * 4, kv_heads=1, dim=128, pad=2, seed=4)
    run_packed(buf, b, 1, 1, 128)


def test_prompt_paged_rows_without_keys(buf):
    b = ref.Batch([300, 200, 40], [0, 3, 150], page=16, kv_heads=1, dim=64, pad=1, seed=1, fill=float("nan"))
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, 4, 64)
    out = sentinel((b.T, 4, 64))
    out, lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, out=out, lse=True)
    ok(buf)
    check_prompt(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, lse)
    assert (out[:497] == 0).all() and torch.isneginf(lse[:497]).all()


# ---------------------------------------------------------------- streams, graphs, the device's own checks

def test_another_stream_and_a_graph_with_new_lengths(buf):
    """A captured decoding step (append, attention) on a side stream, replayed with new lengths and tokens."""
    b = ref.Batch([1] * 3, [40, 3, 100], page=16, kv_heads=2, dim=64, free=12, seed=4)
    b.table = torch.arange(b.pages, device="cuda", dtype=torch.int32)[:18].reshape(3, 6).contiguous()
    buf.set_active_shape([3, 256])
    y = b.randn(3, 8, 64)
    cos = torch.ones(200, 32, device="cuda")
    sin = torch.zeros(200, 32, device="cuda")
    b.kv = [40, 3, 96]
    b.lens.copy_(torch.tensor(b.kv, dtype=torch.int32))
    q_out, out = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda"), sentinel((3, 4, 64))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        buf.kv_append(y[:, :4], y[:, 4:6], y[:, 6:], cos, sin, b.starts, b.lens, b.table, b.k_cache, b.v_cache,
                      q_out=q_out, stream=side)
        buf.attn_decode(q_out, b.k_cache, b.v_cache, b.lens, b.table, out=out, stream=side)

    step()
    side.synchronize()
    ok(buf)
    check_decode(buf, b, y[:, :4], out, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for kv in ([41, 4, 33], [64, 1, 80]):
        b.kv = kv
        b.lens.copy_(torch.tensor(kv, dtype=torch.int32))
        y.copy_(b.randn(3, 8, 64))
        torch.cuda.synchronize()
        graph.replay()
        ok(buf)
        check_decode(buf, b, y[:, :4], out, None)


def test_new_outputs_belong_to_the_call_stream(buf):
    b = ref.Batch([70, 30], [0, 0], kv_heads=1, dim=64, seed=9)
    buf.set_active_shape([100, 256])
    q, k, v = slices(b, 2, 1, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = buf.attn_prompt(q, k, v, b.starts, lse=True, stream=side)
    side.synchronize()
    check_prompt(b, q, lambda s: tuple(x[b.starts_list[s]:b.starts_list[s + 1]].transpose(0, 1) for x in (k, v)), out, lse)


def recorded_argument_error(buf):
    torch.cuda.synchronize()
    code = buf.query_status()
    buf.clear_status()
    return code == ub.CODES["UB_ERR_ARG"]


@pytest.mark.parametrize("entry", [-1, -2 ** 31, 10 ** 6])
def test_a_page_outside_the_cache_is_recorded(buf, entry):
    """Its keys read as zeros and appends to it are dropped; the other sequences are as they were."""
    b = ref.Batch([3, 2], [40, 40], page=16, kv_heads=1, dim=128, seed=2)
    b.table[0, 2] = entry
    buf.set_active_shape([5, 256])
    q, k, v = slices(b, 2, 1, 128)
    before = b.k_cache.clone()
    buf.kv_append(q, k, v, None, None, b.starts, b.lens, b.table, b.k_cache, b.v_cache)
    assert recorded_argument_error(buf)
    changed = (before != b.k_cache).any(-1).sum().item()
    assert changed == 2
    out = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table)
    assert recorded_argument_error(buf)
    o, e, _, _ = ref.attend(q[3:], b.rows(b.k_cache, 1), b.rows(b.v_cache, 1), torch.tensor([38, 39], device="cuda"), 128 ** -0.5)
    ref.within(out[3:], o, e, "prompt, the other sequence")
    buf.set_active_shape([2, 256])
    out = buf.attn_decode(q[2:4], b.k_cache, b.v_cache, b.lens, b.table)
    assert recorded_argument_error(buf)
    o, e, _, _ = ref.attend(q[3:4], b.rows(b.k_cache, 1), b.rows(b.v_cache, 1), torch.tensor([39], device="cuda"), 128 ** -0.5)
    ref.within(out[1:], o, e, "decode, the other sequence")


def test_lengths_beyond_the_table_and_starts_out_of_order(buf):
    b = ref.Batch([4, 4], [32, 20], page=16, kv_heads=1, dim=64, seed=2)
    buf.set_active_shape([8, 256])
    q, k, v = slices(b, 2, 1, 64)
    lens = torch.tensor([10 ** 9, -5], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    out = buf.attn_decode(q, b.k_cache, b.v_cache, lens, b.table)
    o, e, _, _ = ref.attend(q[:1], b.rows(b.k_cache, 0), b.rows(b.v_cache, 0), torch.tensor([31], device="cuda"), 0.125)
    ref.within(out[:1], o, e, "cut to the table")
    assert (out[1] == 0).all()
    cos = torch.ones(64, 32, device="cuda")
    buf.kv_append(q, k, v, cos, cos, starts, lens, b.table, b.k_cache, b.v_cache)
    assert recorded_argument_error(buf)
    for bad in ([6, 2, 4], [-9, 5, 100], [0, 10 ** 9, 3], [8, 8, 8]):
        starts = torch.tensor(bad, dtype=torch.int32, device="cuda")
        buf.attn_prompt(q, k, v, starts)
        buf.attn_prompt_paged(q, b.k_cache, b.v_cache, starts, b.lens, b.table)
        buf.kv_append(q, k, v, cos, cos, starts, b.lens, b.table, b.k_cache, b.v_cache)
        torch.cuda.synchronize()
        buf.clear_status()


def test_everything_strided(buf):
    """Token-by-token caches, keys beside values; strided q, k, v and outputs; rows between stay as they are."""
    b = ref.Batch([70, 1, 200], [300, 90, 200], page=32, kv_heads=3, dim=64, seed=7)
    both = torch.zeros(b.pages, 32, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
    both[:, :, 0], both[:, :, 1] = b.k_cache.transpose(1, 2), b.v_cache.transpose(1, 2)
    b.k_cache, b.v_cache = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    buf.set_active_shape([b.T, 256])
    y = b.randn(b.T, 40, 80)[..., :64]
    q, k, v = y[:, 0:18:3], y[:, 20:32:4], y[:, 33:39:2]
    big = sentinel((2 * b.T, 12, 128))
    out = big[1::2, ::2, 64:]
    buf.kv_append(q, k, v, None, None, b.starts, b.lens, b.table, b.k_cache, b.v_cache, q_out=out)
    ok(buf)
    assert torch.equal(out, q)
    for s, n in enumerate(b.new):
        t0 = b.starts_list[s]
        assert torch.equal(b.rows(b.k_cache, s)[:, -n:].transpose(0, 1), k[t0:t0 + n])
        assert torch.equal(b.rows(b.v_cache, s)[:, -n:].transpose(0, 1), v[t0:t0 + n])
    buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, out=out)
    ok(buf)
    check_prompt(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, None)
    buf.attn_prompt(q, k, v, b.starts, out=out)
    ok(buf)
    check_prompt(b, q, lambda s: tuple(x[b.starts_list[s]:b.starts_list[s + 1]].transpose(0, 1) for x in (k, v)), out, None)
    assert is_sentinel(big[::2]) and is_sentinel(big[1::2, 1::2]) and is_sentinel(big[1::2, ::2, :64])


def test_append_and_prompt_over_a_cache_past_32_bits(buf):
    pages = (1 << 31) // (64 * 128) + 100
    k = torch.zeros(pages, 1, 64, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    b = ref.Batch([50, 3], [150, 90], page=64, kv_heads=1, dim=128, free=0, seed=8)
    k[pages - b.pages:], v[pages - b.pages:] = b.k_cache, b.v_cache
    b.k_cache, b.v_cache = k, v
    b.table[b.table >= 0] += pages - b.pages
    b.pages = pages
    buf.set_active_shape([53, 256])
    q, kk, vv = slices(b, 4, 1, 128)
    out = buf.kv_append(q, kk, vv, None, None, b.starts, b.lens, b.table, k, v)
    ok(buf)
    assert torch.equal(b.rows(k, 0)[0, -50:], kk[:50, 0]) and torch.equal(b.rows(v, 1)[0, -3:], vv[50:, 0])
    got = buf.attn_prompt_paged(out, k, v, b.starts, b.lens, b.table)
    ok(buf)
    check_prompt(b, q, lambda s: (b.rows(k, s), b.rows(v, s)), got, None)


def test_prompt_from_a_graph_with_new_lengths(buf):
    b = ref.Batch([60, 40], [300, 40], page=16, kv_heads=2, dim=128, free=40, seed=4)
    b.table = torch.arange(b.pages, device="cuda", dtype=torch.int32)[:60].reshape(2, 30).contiguous()
    buf.set_active_shape([100, 256])
    q = b.randn(100, 4, 128)
    out = sentinel((100, 4, 128))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, out=out, stream=side)
    for new, kv in (([60, 40], [300, 40]), ([1, 99], [480, 99]), ([100, 0], [100, 7])):
        b.new, b.kv, b.starts_list = new, kv, [0, new[0], 100]
        b.starts.copy_(torch.tensor(b.starts_list, dtype=torch.int32))
        b.lens.copy_(torch.tensor(kv, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        ok(buf)
        check_prompt(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, None)


@pytest.mark.parametrize("options", [{"pdl": 0}, {"sm_margin": 100}, {"sm_margin": 151, "pdl": 0}, {"profile": 1}])
def test_options(buf, options):
    """Plain launches, few SMs and launch timing give the same results."""
    b = ref.Batch([700, 3, 16], [2500, 1030, 16], page=32, kv_heads=2, dim=64, seed=3)
    d = ref.Batch([1] * 5, [9000, 17, 300, 1, 0], page=32, kv_heads=2, dim=64, seed=4)
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, 8, 64)
    before = {k: buf.get_option(k) for k in options}
    for k, v in options.items():
        buf.set_option(k, v)
    try:
        out = sentinel((b.T, 8, 64))
        buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, out=out)
        ok(buf)
        check_prompt(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, None)
        run_decode(buf, d, 8, 64)
        if "profile" in options:
            for op in ("attn_prompt", "attn_decode"):
                ms, launches = buf.kernel_time(op)
                assert launches == 1 and 0 < ms < 100
    finally:
        for k, v in before.items():
            buf.set_option(k, v)


# ---------------------------------------------------------------- refusals

def test_refusals(buf):
    b = ref.Batch([2, 2], [20, 20], page=16, kv_heads=2, dim=64, seed=2)
    buf.set_active_shape([4, 256])
    q, k, v = slices(b, 4, 2, 64)
    cos = torch.ones(64, 32, device="cuda")
    seqs, cache = (b.starts, b.lens, b.table), (b.k_cache, b.v_cache)

    def append(q=q, k=k, v=v, cos=cos, sin=cos, seqs=seqs, cache=cache, **kw):
        return buf.kv_append(q, k, v, cos, sin, *seqs, *cache, **kw)

    def decode(q=q, cache=cache, lens=b.lens, table=b.table, **kw):
        return buf.attn_decode(q, *cache, lens, table, **kw)

    def prompt(q=q, k=k, v=v, starts=b.starts, **kw):
        return buf.attn_prompt(q, k, v, starts, **kw)

    def code(name, fn, *a, **kw):
        with pytest.raises(ub.UbError) as e:
            fn(*a, **kw)
        assert e.value.name == name, e.value

    for fn in (append, decode, prompt):
        for bad in (q.float(), q.cpu(), "q"):
            with pytest.raises(TypeError):
                fn(q=bad)
        for bad in (q[:3], q[0], q.transpose(1, 2)):
            with pytest.raises(ValueError):
                fn(q=bad)
    shifted = torch.zeros(4 * 4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    code("UB_ERR_ALIGN", decode, q=shifted[4:4 + 1024].view(4, 4, 64))       # 8-byte aligned
    code("UB_ERR_ALIGN", decode, q=torch.zeros(4, 4, 68, dtype=torch.bfloat16, device="cuda")[..., :64])
    code("UB_ERR_ALIGN", decode, q=q[:, :1].expand(4, 4, 64))               # stride 0
    code("UB_ERR_ARG", decode, q=torch.zeros(4, 3, 64, dtype=torch.bfloat16, device="cuda"))  # 3 heads over 2
    odd = torch.zeros(4, 4, 96, dtype=torch.bfloat16, device="cuda")
    code("UB_ERR_ARG", prompt, q=odd, k=odd[:, :2], v=odd[:, :2])
    for page in (4, 24, 512):
        c = torch.zeros(3, 2, page, 64, dtype=torch.bfloat16, device="cuda")
        code("UB_ERR_ARG", decode, cache=(c, c))
    for scale in (0.0, -1.0, math.inf, math.nan):
        code("UB_ERR_ARG", decode, scale=scale)
        code("UB_ERR_ARG", prompt, scale=scale)
    code("UB_ERR_CAPACITY", decode, lens=torch.ones(5, dtype=torch.int32, device="cuda"),
         table=torch.zeros(5, 1, dtype=torch.int32, device="cuda"))
    code("UB_ERR_ZERO", decode, lens=b.lens[:0], table=b.table[:0])
    code("UB_ERR_ZERO", decode, table=b.table[:, :0])
    code("UB_ERR_ZERO", prompt, starts=b.starts[:1])
    code("UB_ERR_ZERO", decode, cache=(b.k_cache[:0], b.v_cache[:0]))
    code("UB_ERR_ARG", append, cos=torch.ones(64, 4, device="cuda"), sin=torch.ones(64, 4, device="cuda"))  # rot 8
    code("UB_ERR_ARG", append, cos=torch.ones(64, 40, device="cuda"), sin=torch.ones(64, 40, device="cuda"))
    for kw in ({"lens": b.lens.long()}, {"table": b.table.float()}, {"lens": b.lens.cpu()}):
        with pytest.raises(TypeError):
            decode(**kw)
    for kw in ({"table": b.table.t()}, {"table": b.table[:1]}, {"cache": (b.k_cache, b.v_cache[:, :1])},
               {"cache": (b.k_cache[..., :32], b.v_cache)}, {"out": q[:, :2]}, {"lse": torch.ones(3, 4, device="cuda")}):
        with pytest.raises(ValueError):
            decode(**kw)
    for kw in ({"k": k[:, :1]}, {"sin": cos[:3]}, {"seqs": (b.starts[:2], b.lens, b.table)}, {"q_out": q[:, :2]}):
        with pytest.raises(ValueError):
            append(**kw)
    with pytest.raises(TypeError):
        append(cos=cos.double(), sin=cos.double())
    assert ub.load().ub_attn_decode(buf._h, ub._ATTN.pack(8, *[0] * 7, 1.0, *[0] * 31), None) == ub.CODES["UB_ERR_ARG"]
    torch.cuda.synchronize()
    assert buf.query_status() == ub.UB_OK
