"""Attention with a sliding window and sinks against its 64-bit definition: packed prompts, chunks
over the cache, single tokens; pages out of sight that are no longer the sequence's."""
import pytest
import torch

import attn_ref as ref
import serve_ref as sr
from gemm_overlap_gemms_gb300 import ub
from gpu_helpers import is_sentinel, sentinel

pytestmark = pytest.mark.gpu

SIGHTS = [(1, 0), (1, 1), (5, 3), (64, 4), (127, 0), (128, 128), (129, 1), (300, 200), (1000, 4), (1 << 30, 7)]


@pytest.fixture(scope="module")
def buf():
    from gemm_overlap_gemms_gb300 import _build
    _build.build()
    with ub.UserBuffer([16384, 256], 1) as b:
        yield b


def ok(buf):
    torch.cuda.synchronize()
    assert buf.query_status() == ub.UB_OK


def drop_unseen(b, window, sinks, new):
    """Entries of pages that no row sees: -1, or a page of another's, full of NaN."""
    nan = b.pages
    b.k_cache = torch.cat((b.k_cache, torch.full_like(b.k_cache[:1], float("nan"))))
    b.v_cache = torch.cat((b.v_cache, torch.full_like(b.v_cache[:1], float("nan"))))
    table = b.table.clone()
    for s, (n, total) in enumerate(zip(new, b.kv)):
        low = max(0, total - n - window + 1)
        for j in range(-(-total // b.page)):
            if (j + 1) * b.page <= low and j * b.page >= sinks:
                table[s, j] = nan if j % 2 else -1
    return table


def check(b, q, k_v, out, lse, window, sinks, new):
    at = 0
    for s, (n, total) in enumerate(zip(new, b.kv)):
        pos = torch.arange(total - n, total, device=q.device)
        k, v = k_v(s)
        seen = sr.in_window(pos, torch.arange(k.shape[1], device=q.device), window, sinks)
        o, e, ll, le = sr.attend_seen(q[at:at + n], k, v, seen, q.shape[2] ** -0.5)
        ref.within(out[at:at + n], o, e, "sequence %d: %d of %d, window %d, sinks %d" % (s, n, total, window, sinks))
        if lse is not None:
            ref.within(lse[at:at + n], ll, le, "lse of sequence %d" % s)
        at += n
    assert is_sentinel(out[at:])


def run_decode(buf, b, heads, dim, window, sinks, table=None):
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, heads, dim, std=1.5)
    out = sentinel((b.T, heads, dim))
    table = drop_unseen(b, window, sinks, [1] * len(b.kv)) if table is None else table
    _, lse = buf.attn_decode(q, b.k_cache, b.v_cache, b.lens, table, out=out, lse=True, window=window, sinks=sinks)
    ok(buf)
    new = [1 if n > 0 else 0 for n in b.kv]
    for s, n in enumerate(b.kv):  # a row each, also of a sequence without keys
        if n == 0:
            assert (out[s] == 0).all() and torch.isneginf(lse[s]).all()
    keep = [s for s, n in enumerate(new) if n]
    check_rows(b, q, out, lse, window, sinks, keep)
    assert is_sentinel(out[len(b.kv):])
    return q, out


def check_rows(b, q, out, lse, window, sinks, rows):
    for s in rows:
        total = b.kv[s]
        seen = sr.in_window(torch.tensor([total - 1], device=q.device), torch.arange(total, device=q.device), window, sinks)
        o, e, ll, le = sr.attend_seen(q[s:s + 1], b.rows(b.k_cache, s), b.rows(b.v_cache, s), seen, q.shape[2] ** -0.5)
        ref.within(out[s:s + 1], o, e, "sequence %d of %d keys, window %d, sinks %d" % (s, total, window, sinks))
        ref.within(lse[s:s + 1], ll, le, "lse of sequence %d" % s)


@pytest.mark.parametrize("window,sinks", SIGHTS)
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 64), (128, 8), (64, 256)])
def test_decode(buf, window, sinks, dim, page):
    kv = [1, 31, 32, 33, 0, 500, 129, 64, 1000, 2049]
    b = ref.Batch([1] * len(kv), kv, page=page, kv_heads=2, dim=dim, pad=3, seed=window + dim, fill=float("nan"))
    run_decode(buf, b, 8, dim, window, sinks)


@pytest.mark.parametrize("heads,kv_heads,kv", [(40, 2, [3000, 7]), (8, 1, [40000]), (12, 1, [9000, 1, 0, 12000]), (5, 5, [700] * 70),
                                               (16, 1, list(range(0, 4000, 31))), (8, 8, [30000] * 40)])
@pytest.mark.parametrize("window,sinks", [(100, 4), (4000, 33), (20000, 0)])
def test_decode_splits(buf, heads, kv_heads, kv, window, sinks):
    b = ref.Batch([1] * len(kv), kv, page=64, kv_heads=kv_heads, dim=128, seed=heads, fill=float("nan"))
    q, out = run_decode(buf, b, heads, 128, window, sinks)
    again = buf.attn_decode(q, b.k_cache, b.v_cache, b.lens, b.table, window=window, sinks=sinks)
    assert torch.equal(again, out)


@pytest.mark.parametrize("window,sinks", SIGHTS)
@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 8, 8), (64, 8, 1), (128, 6, 2)])
def test_packed_prompts(buf, window, sinks, dim, heads, kv_heads):
    new = [1, 130, 17, 0, 128, 700, 1, 257]
    b = ref.Batch(new, new, kv_heads=kv_heads, dim=dim, pad=5, seed=window)
    buf.set_active_shape([b.T, 256])
    y = b.randn(b.T, heads + 2 * kv_heads, dim)
    q, k, v = y[:, :heads], y[:, heads:heads + kv_heads], y[:, heads + kv_heads:]
    k[sum(new):] = float("nan")
    v[sum(new):] = float("nan")
    out = sentinel((b.T, heads, dim))
    _, lse = buf.attn_prompt(q, k, v, b.starts, out=out, lse=True, window=window, sinks=sinks)
    ok(buf)
    s0 = b.starts_list
    check(b, q, lambda s: (k[s0[s]:s0[s + 1]].transpose(0, 1), v[s0[s]:s0[s + 1]].transpose(0, 1)), out, lse, window, sinks, new)


@pytest.mark.parametrize("window,sinks", SIGHTS)
@pytest.mark.parametrize("dim,page,heads,kv_heads", [(128, 16, 8, 2), (64, 8, 16, 4), (64, 128, 5, 5), (128, 256, 8, 8)])
def test_chunks_over_the_cache(buf, window, sinks, dim, page, heads, kv_heads):
    new = [1, 130, 17, 0, 128, 400, 3]
    kv = [n + past for n, past in zip(new, [900, 0, 2000, 50, 128, 1111, 0])]
    b = ref.Batch(new, kv, page=page, kv_heads=kv_heads, dim=dim, pad=5, seed=window, fill=float("nan"))
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, heads, dim, std=1.5)
    table = drop_unseen(b, window, sinks, new)
    out = sentinel((b.T, heads, dim))
    _, lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, table, out=out, lse=True, window=window, sinks=sinks)
    ok(buf)
    check(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, lse, window, sinks, new)


@pytest.mark.parametrize("window,sinks", [(3000, 4), (9000, 500), (1500, 0)])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 1, 128), (8, 8, 64), (12, 4, 128)])
def test_few_tokens_over_long_windows_are_split(buf, window, sinks, heads, kv_heads, dim):
    new = [16, 1, 300, 40]
    kv = [20000, 9000, 5000, 40]
    b = ref.Batch(new, kv, page=64, kv_heads=kv_heads, dim=dim, seed=window, fill=float("nan"))
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, heads, dim, std=1.5)
    table = drop_unseen(b, window, sinks, new)
    out = sentinel((b.T, heads, dim))
    _, lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, table, out=out, lse=True, window=window, sinks=sinks)
    ok(buf)
    check(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, lse, window, sinks, new)


@pytest.mark.parametrize("n,heads,kv_heads,dim,window", [(10, 8, 8, 128, 2500), (11, 8, 8, 64, 1700), (20, 8, 8, 64, 2500), (40, 8, 2, 128, 3300),
                                                         (13, 6, 6, 128, 2000), (39, 4, 4, 64, 1500)])
def test_incomplete_last_rounds_are_split(buf, n, heads, kv_heads, dim, window):
    """A few items more than one or two for each SM: those are cut along their keys, after the whole ones."""
    new = [300 - 7 * (i % 3) for i in range(n)]
    kv = [m + 4000 + 13 * i for i, m in enumerate(new)]
    b = ref.Batch(new, kv, page=32, kv_heads=kv_heads, dim=dim, pad=1, seed=n, fill=float("nan"))
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, heads, dim, std=1.5)
    table = drop_unseen(b, window, 4, new)
    out = sentinel((b.T, heads, dim))
    args = (q, b.k_cache, b.v_cache, b.starts, b.lens, table)
    _, lse = buf.attn_prompt_paged(*args, out=out, lse=True, window=window, sinks=4)
    ok(buf)
    check(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out, lse, window, 4, new)
    for _ in range(2):
        assert torch.equal(buf.attn_prompt_paged(*args, window=window, sinks=4)[:sum(new)], out[:sum(new)])
    ok(buf)


@pytest.mark.parametrize("window,sinks", [(70, 5), (600, 0)])
@pytest.mark.parametrize("dim", [64, 128])
def test_strided_views(buf, window, sinks, dim):
    """Queries inside a fused projection, outputs by heads, caches and table as views."""
    new, heads, kv_heads = [5, 300, 1, 40], 8, 2
    kv = [n + past for n, past in zip(new, [200, 0, 33, 900])]
    b = ref.Batch(new, kv, page=16, kv_heads=kv_heads, dim=dim, pad=2, seed=dim, fill=float("nan"))
    whole = torch.stack((b.k_cache, b.v_cache)).transpose(1, 2).contiguous()  # pages inside the heads
    b.k_cache, b.v_cache = whole[0].transpose(0, 1), whole[1].transpose(0, 1)
    wide = torch.full((len(new), b.table.shape[1] + 7), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :-7] = b.table
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, heads + 2 * kv_heads, dim, std=1.5)[:, :heads]
    out = sentinel((heads, b.T, dim)).transpose(0, 1)
    _, lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, wide[:, :-7], out=out, lse=True,
                                   window=window, sinks=sinks)
    ok(buf)
    check(b, q, lambda s: (b.rows(b.k_cache, s), b.rows(b.v_cache, s)), out.contiguous(), lse, window, sinks, new)
    out = sentinel((heads, b.T, dim)).transpose(0, 1)
    _, lse = buf.attn_decode(q, b.k_cache, b.v_cache, b.lens, wide[:, :-7], out=out, lse=True, window=window, sinks=sinks)
    ok(buf)
    check_rows(b, q, out.contiguous(), lse, window, sinks, range(len(kv)))
    assert is_sentinel(out[len(kv):].contiguous())


def test_rows_without_a_key(buf):
    """kv_lens below the new tokens: the first rows have no position in the cache."""
    b = ref.Batch([40, 200], [30, 140], page=16, kv_heads=2, dim=128, seed=3, fill=float("nan"))
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, 8, 128)
    out, lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, lse=True, window=9, sinks=2)
    ok(buf)
    for row in list(range(10)) + list(range(40, 100)):
        assert (out[row] == 0).all() and torch.isneginf(lse[row]).all()
    for s, (n, total) in enumerate(zip(b.new, b.kv)):
        at = b.starts_list[s] + n - total
        pos = torch.arange(total, device="cuda")
        o, e, _, _ = sr.attend_seen(q[at:at + total], b.rows(b.k_cache, s), b.rows(b.v_cache, s), sr.in_window(pos, pos, 9, 2), 128 ** -0.5)
        ref.within(out[at:at + total], o, e, "sequence %d" % s)


def test_a_window_of_everything_is_none(buf):
    """A window as long as the cache, and no window, are the same call."""
    b = ref.Batch([100, 3], [700, 300], page=16, kv_heads=2, dim=64, seed=4)
    buf.set_active_shape([b.T, 256])
    q = b.randn(b.T, 8, 64)
    args = (q, b.k_cache, b.v_cache, b.starts, b.lens, b.table)
    assert torch.equal(buf.attn_prompt_paged(*args), buf.attn_prompt_paged(*args, window=10 ** 6, sinks=5))
    assert torch.equal(buf.attn_prompt_paged(*args), buf.attn_prompt_paged(*args, window=0, sinks=5))
    ok(buf)


def test_a_page_in_sight_that_is_missing_is_recorded(buf):
    b = ref.Batch([1], [300], page=16, kv_heads=1, dim=64, seed=4)
    buf.set_active_shape([1, 256])
    table = b.table.clone()
    table[0, 17] = -1
    buf.attn_decode(b.randn(1, 4, 64), b.k_cache, b.v_cache, b.lens, table, window=40)
    torch.cuda.synchronize()
    assert buf.query_status() == ub.CODES["UB_ERR_ARG"]
    buf.clear_status()
    buf.attn_decode(b.randn(1, 4, 64), b.k_cache, b.v_cache, b.lens, table, window=10)
    ok(buf)


def test_windows_from_a_graph(buf):
    """A captured step sees new lengths and tables at every replay."""
    b = ref.Batch([1] * 5, [400, 33, 1, 900, 77], page=16, kv_heads=2, dim=128, seed=6, fill=float("nan"))
    buf.set_active_shape([b.T, 256])
    q, out = b.randn(b.T, 8, 128), torch.empty(b.T, 8, 128, dtype=torch.bfloat16, device="cuda")
    lens = b.lens.clone()
    buf.attn_decode(q, b.k_cache, b.v_cache, lens, b.table, out=out, window=50, sinks=3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        buf.attn_decode(q, b.k_cache, b.v_cache, lens, b.table, out=out, window=50, sinks=3)
    for cut in (0, 5, 31):
        lens.copy_((b.lens - cut).clamp_min(0))
        graph.replay()
        torch.cuda.synchronize()
        eager = buf.attn_decode(q, b.k_cache, b.v_cache, lens, b.table, window=50, sinks=3)
        assert torch.equal(out, eager)
    ok(buf)


@pytest.mark.parametrize("window,sinks", [(-1, 0), (5, -1), (1 << 31, 0), (None, 0)])
def test_refused_windows(buf, window, sinks):
    b = ref.Batch([1], [30], page=16, kv_heads=1, dim=64)
    buf.set_active_shape([1, 256])
    q = b.randn(1, 4, 64)
    with pytest.raises(ValueError):
        buf.attn_decode(q, b.k_cache, b.v_cache, b.lens, b.table, window=window, sinks=sinks)
