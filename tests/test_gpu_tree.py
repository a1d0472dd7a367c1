"""Drafted tokens against their 64-bit definitions: tree attention over a paged cache, the append
that rotates drafts by their position, and the rows of accepted drafts."""
import random

import pytest
import torch

import attn_ref as ref
import serve_ref as sr
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


def trees(b, kind="bushy", seed=0):
    rng = random.Random(seed)
    per = [sr.random_tree(n, rng, kind) for n in b.new]
    flat = [p for t in per for p in t]
    flat += [12345] * (b.T - len(flat))  # rows of no sequence: not looked at
    return per, torch.tensor(flat, dtype=torch.int32, device="cuda")


def check(b, q, per, out, lse, window=0, sinks=0):
    for s, (n, total) in enumerate(zip(b.new, b.kv)):
        a = b.starts_list[s]
        seen = sr.tree_seen(per[s], total, window, sinks).to(q.device)
        o, e, ll, le = sr.attend_seen(q[a:a + n], b.rows(b.k_cache, s), b.rows(b.v_cache, s), seen, q.shape[2] ** -0.5)
        ref.within(out[a:a + n], o, e, "sequence %d: %d drafts of %d keys" % (s, n, total))
        ref.within(lse[a:a + n], ll, le, "lse of sequence %d" % s)
    assert is_sentinel(out[sum(b.new):])


def run(buf, b, heads, dim, kind="bushy", window=0, sinks=0, table=None):
    buf.set_active_shape([b.T, 256])
    per, parents = trees(b, kind, seed=len(b.kv))
    q = b.randn(b.T, heads, dim, std=1.5)
    out = sentinel((b.T, heads, dim))
    _, lse = buf.attn_tree(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table if table is None else table, parents, out=out,
                           lse=True, window=window, sinks=sinks)
    ok(buf)
    check(b, q, per, out, lse, window, sinks)
    return q, parents, out


@pytest.mark.parametrize("kind", ["bushy", "chain", "flat"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (8, 1), (12, 4), (5, 5), (9, 1), (40, 2)])
def test_trees_and_heads(buf, kind, dim, heads, kv_heads):
    new = [1, 5, 0, 64, 17, 33, 2]
    kv = [n + past for n, past in zip(new, [0, 123, 40, 64, 700, 95, 254])]
    b = ref.Batch(new, kv, page=16, kv_heads=kv_heads, dim=dim, pad=3, seed=heads, fill=float("nan"))
    run(buf, b, heads, dim, kind)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_pages(buf, page):
    new = [7, 30, 1, 64]
    kv = [page + 3, 5 * page + 30, 1, 1000]
    b = ref.Batch(new, kv, page=page, kv_heads=2, dim=128, seed=page, fill=float("inf"))
    run(buf, b, 8, 128)


@pytest.mark.parametrize("heads,kv_heads", [(160, 1), (300, 2), (129, 1), (128, 1)])
def test_many_heads_on_one(buf, heads, kv_heads):
    """More query heads to a key/value head than a q tile has rows, and just as many."""
    b = ref.Batch([3, 20], [200, 333], page=16, kv_heads=kv_heads, dim=64, pad=1, seed=heads, fill=float("nan"))
    run(buf, b, heads, 64)


@pytest.mark.parametrize("new,kv", [([200], [900]), ([300, 1], [300, 1]), ([1000], [5000]), ([130, 129, 128, 127], [400, 129, 5000, 130])])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (1, 1)])
def test_large_trees(buf, new, kv, heads, kv_heads):
    b = ref.Batch(new, kv, page=32, kv_heads=kv_heads, dim=128, pad=2, seed=1, fill=float("nan"))
    run(buf, b, heads, 128)
    run(buf, b, heads, 128, "chain")


@pytest.mark.parametrize("new,past,heads,kv_heads,dim", [
    ([6], [40000], 8, 1, 128), ([60], [70001], 8, 1, 64), ([30] * 16, [700 + 500 * i for i in range(16)], 8, 2, 128),
    ([3 + i % 30 for i in range(70)], [17 + 131 * i % 3000 for i in range(70)], 8, 8, 128), ([1] * 200, [50 + i for i in range(200)], 4, 1, 64),
    ([12] * 150, [1000 + 11 * i for i in range(150)], 4, 1, 128), ([64] * 5, [20000, 0, 300, 9000, 1], 32, 4, 64),
    ([0, 0, 0, 9, 0], [100, 0, 5, 8000, 3], 8, 8, 128), ([1, 300], [30000, 30000], 16, 2, 128)])
def test_splits(buf, new, past, heads, kv_heads, dim):
    """Items whole, split over two CTAs, over all of them; deterministic, and the counters left clean."""
    b = ref.Batch(new, [n + k for n, k in zip(new, past)], page=64, kv_heads=kv_heads, dim=dim, seed=heads, fill=float("nan"))
    q, parents, out = run(buf, b, heads, dim)
    for _ in range(3):
        assert torch.equal(out, buf.attn_tree(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents))
    ok(buf)


@pytest.mark.parametrize("window,sinks", [(0, 0), (500, 3)])
@pytest.mark.parametrize("new,past,heads,kv_heads,dim", [
    ([40 + i % 25 for i in range(44)], [100 + 37 * i for i in range(44)], 8, 2, 128),
    ([33 + i % 32 for i in range(40)], [3000 + 50 * i for i in range(40)], 16, 4, 64),
    ([64, 50], [70000, 70100], 8, 2, 128), ([130, 64, 1], [66000, 67000, 68000], 16, 4, 64)])
def test_items_of_two_query_tiles(buf, new, past, heads, kv_heads, dim, window, sinks):
    """More query tiles than CTAs, and few over so many keys that each takes them for two."""
    b = ref.Batch(new, [n + k for n, k in zip(new, past)], page=64, kv_heads=kv_heads, dim=dim, seed=dim, fill=float("nan"))
    q, parents, out = run(buf, b, heads, dim, window=window, sinks=sinks)
    for _ in range(3):
        again = buf.attn_tree(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents, window=window, sinks=sinks)
        assert torch.equal(out, again)
    ok(buf)


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (5, 0), (40, 4), (128, 200), (300, 1), (2000, 0), (1 << 30, 0)])
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 128)])
def test_windows(buf, window, sinks, dim, page):
    """A window shorter than a path hides ancestors; pages out of sight are not looked at."""
    new = [1, 5, 0, 64, 17, 33, 200]
    kv = [n + past for n, past in zip(new, [0, 123, 40, 64, 1700, 95, 3000])]
    b = ref.Batch(new, kv, page=page, kv_heads=2, dim=dim, pad=3, seed=window, fill=float("nan"))
    table = b.table.clone()
    for s, (n, total) in enumerate(zip(new, kv)):
        low = max(0, total - n - window + 1)
        for j in range(-(-total // page)):
            if (j + 1) * page <= low and j * page >= sinks:
                table[s, j] = -1
    run(buf, b, 8, dim, window=window, sinks=sinks, table=table)
    run(buf, b, 8, dim, "chain", window=window, sinks=sinks, table=table)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_strided_views(buf, dim, window, sinks):
    """Queries inside a fused projection, outputs by heads, caches and table as views."""
    new, heads, kv_heads = [5, 64, 1, 40, 9], 8, 2
    kv = [n + past for n, past in zip(new, [200, 0, 33, 900, 4000])]
    b = ref.Batch(new, kv, page=16, kv_heads=kv_heads, dim=dim, pad=2, seed=dim, fill=float("nan"))
    whole = torch.stack((b.k_cache, b.v_cache)).transpose(1, 2).contiguous()  # pages inside the heads
    b.k_cache, b.v_cache = whole[0].transpose(0, 1), whole[1].transpose(0, 1)
    wide = torch.full((len(new), b.table.shape[1] + 7), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :-7] = b.table
    buf.set_active_shape([b.T, 256])
    per, parents = trees(b)
    q = b.randn(b.T, heads + 2 * kv_heads, dim, std=1.5)[:, :heads]
    out = sentinel((heads, b.T, dim)).transpose(0, 1)
    _, lse = buf.attn_tree(q, b.k_cache, b.v_cache, b.starts, b.lens, wide[:, :-7], parents, out=out, lse=True,
                           window=window, sinks=sinks)
    ok(buf)
    check(b, q, per, out.contiguous(), lse, window, sinks)


@pytest.mark.parametrize("most,window", [(1, 0), (3, 0), (3, 64), (40, 0)])
def test_many_sequences(buf, most, window):
    """More sequences than a warp looks at at once, and than there are CTAs; some without drafts."""
    rng = random.Random(most)
    new = [rng.randint(0, most) for _ in range(700)]
    kv = [n + rng.randint(0, 300) for n in new]
    b = ref.Batch(new, kv, page=32, kv_heads=2, dim=64, pad=1, seed=most, fill=float("nan"))
    run(buf, b, 4, 64, window=window, sinks=2)


def test_a_chain_is_a_prompt(buf):
    """A chain of drafts is what attn_prompt_paged computes, an only draft what attn_decode does."""
    b = ref.Batch([40, 9], [900, 9], page=16, kv_heads=2, dim=128, seed=2, fill=float("nan"))
    q, parents, out = run(buf, b, 8, 128, "chain")
    prompt = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table)
    assert ((out[:49].float() - prompt.float()).abs() <= 4 * ref.U * prompt.float().abs() + 2e-2).all()


def test_drafts_before_the_cache(buf):
    """kv_lens below the drafts: the places below zero are no keys."""
    b = ref.Batch([40, 3], [30, 0], page=16, kv_heads=2, dim=64, seed=3, fill=float("nan"))
    buf.set_active_shape([b.T, 256])
    per, parents = trees(b, "chain")
    q = b.randn(b.T, 8, 64)
    out, lse = buf.attn_tree(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents, lse=True)
    ok(buf)
    for row in list(range(10)) + [40, 41, 42]:
        assert (out[row] == 0).all() and torch.isneginf(lse[row]).all()
    pos = torch.arange(30, device="cuda")
    o, e, _, _ = sr.attend_seen(q[10:40], b.rows(b.k_cache, 0), b.rows(b.v_cache, 0), pos[:, None] >= pos[None, :], 64 ** -0.5)
    ref.within(out[10:40], o, e, "the rest of the chain")


def test_a_wrong_parent_is_recorded(buf):
    """A parent that does not come before its child counts as the text, and is reported."""
    b = ref.Batch([6], [50], page=16, kv_heads=1, dim=64, seed=3)
    buf.set_active_shape([6, 256])
    q = b.randn(6, 4, 64)
    args = (q, b.k_cache, b.v_cache, b.starts, b.lens, b.table)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    good = buf.attn_tree(*args, ints(-1, -1, -1, 2, -1, 4))
    ok(buf)
    bad = buf.attn_tree(*args, ints(-1, 1, 5, 2, -7, 4))
    torch.cuda.synchronize()
    assert buf.query_status() == ub.CODES["UB_ERR_ARG"]
    buf.clear_status()
    assert torch.equal(good, bad)


def test_trees_on_a_stream_and_from_a_graph(buf):
    b = ref.Batch([9, 30], [900, 5000], page=16, kv_heads=2, dim=128, seed=5)
    buf.set_active_shape([b.T, 256])
    per, parents = trees(b)
    _, other = trees(b, seed=9)
    q = b.randn(b.T, 8, 128)
    args = (q, b.k_cache, b.v_cache, b.starts, b.lens, b.table)
    first, second = buf.attn_tree(*args, parents), buf.attn_tree(*args, other)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = buf.attn_tree(*args, parents, stream=side)
    side.synchronize()
    assert torch.equal(out, first)
    up, graph = parents.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        buf.attn_tree(*args, up, out=out)
    for tree, want in ((parents, first), (other, second)):
        up.copy_(tree)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    ok(buf)


def test_trees_between_other_attention_calls(buf):
    """The joins of trees and of decoding share their counters."""
    b = ref.Batch([20] * 3, [30000, 5000, 700], page=32, kv_heads=2, dim=64, seed=5)
    d = ref.Batch([1] * 3, [30000, 5000, 11], page=32, kv_heads=2, dim=64, seed=6)
    per, parents = trees(b)
    q, qd = b.randn(60, 8, 64), d.randn(3, 8, 64)
    want = None
    for _ in range(4):
        buf.set_active_shape([60, 256])
        o = buf.attn_tree(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents)
        buf.set_active_shape([3, 256])
        e = buf.attn_decode(qd, d.k_cache, d.v_cache, d.lens, d.table)
        want = want or (o, e)
        assert torch.equal(o, want[0]) and torch.equal(e, want[1])
    ok(buf)


def test_refused_calls(buf):
    b = ref.Batch([6], [50], page=16, kv_heads=1, dim=64)
    buf.set_active_shape([6, 256])
    q = b.randn(6, 4, 64)
    per, parents = trees(b)
    args = (q, b.k_cache, b.v_cache, b.starts, b.lens, b.table)
    for bad in (parents[:5], parents.long(), parents.cpu(), None, parents.view(2, 3)):
        with pytest.raises((TypeError, ValueError)):
            buf.attn_tree(*args, bad)
    with pytest.raises(ValueError):
        buf.attn_tree(*args, parents, window=-3)
    with pytest.raises(ub.UbError):
        buf.attn_tree(*args, parents, scale=0.0)


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot,heads,kv_heads", [(128, 128, 8, 2), (64, 32, 4, 4), (128, 0, 8, 1)])
def test_append_of_drafts(buf, interleaved, dim, rot, heads, kv_heads):
    new = [5, 64, 0, 1, 20]
    kv = [n + past for n, past in zip(new, [33, 100, 7, 0, 0])]
    b = ref.Batch(new, kv, page=16, kv_heads=kv_heads, dim=dim, pad=2, seed=rot)
    buf.set_active_shape([b.T, 256])
    per, parents = trees(b)
    y = b.randn(b.T, heads + 2 * kv_heads, dim)
    q, k, v = y[:, :heads], y[:, heads:heads + kv_heads], y[:, heads + kv_heads:]
    cos = sin = None
    if rot:
        angle = torch.rand(200, rot // 2, generator=b.gen, device="cuda") * 6
        cos, sin = angle.cos(), angle.sin()
    out = sentinel((b.T, heads, dim))
    kc, vc = b.k_cache.clone(), b.v_cache.clone()
    buf.kv_append(q, k, v, cos, sin, b.starts, b.lens, b.table, b.k_cache, b.v_cache, q_out=out, interleaved=interleaved,
                  parents=parents)
    ok(buf)
    for s, (n, total) in enumerate(zip(new, kv)):
        if n == 0:
            continue
        a = b.starts_list[s]
        pos = torch.tensor([total - n + len(p) - 1 for p in sr.paths(per[s])], device="cuda")
        place = torch.arange(total - n, total, device="cuda")
        at = b.table[s].long()[place // 16], place % 16
        for x, got in ((q[a:a + n], out[a:a + n]), (k[a:a + n], b.k_cache[at[0], :, at[1]])):
            if rot:
                want, e = ref.rotate(x, cos[pos], sin[pos], interleaved)
                ref.within(got, want, e, "sequence %d" % s)
            else:
                assert torch.equal(got, x)
        assert torch.equal(b.v_cache[at[0], :, at[1]], v[a:a + n])
        kc[at[0], :, at[1]] = b.k_cache[at[0], :, at[1]]
        vc[at[0], :, at[1]] = v[a:a + n]
    assert torch.equal(kc, b.k_cache) and torch.equal(vc, b.v_cache)
    assert is_sentinel(out[sum(new):])


def test_append_of_a_chain_is_the_plain_one(buf):
    b = ref.Batch([30, 7], [90, 7], page=16, kv_heads=2, dim=128, seed=2)
    buf.set_active_shape([b.T, 256])
    _, parents = trees(b, "chain")
    q, k, v = b.randn(37, 8, 128), b.randn(37, 2, 128), b.randn(37, 2, 128)
    angle = torch.rand(100, 64, device="cuda")
    args = (q, k, v, angle.cos(), angle.sin(), b.starts, b.lens, b.table)
    caches = [(b.k_cache.clone(), b.v_cache.clone()) for _ in range(2)]
    one, two = buf.kv_append(*args, *caches[0]), buf.kv_append(*args, *caches[1], parents=parents)
    ok(buf)
    assert torch.equal(one, two) and all(torch.equal(x, y) for x, y in zip(*caches))


@pytest.mark.parametrize("new,past", [([300, 33, 64, 1, 32], [5, 0, 90, 3, 31]), ([1500], [100]), ([31, 32, 33, 65] * 9, [7] * 36)])
def test_append_and_attention_of_deep_chains(buf, new, past):
    """Chains past a word of 32 drafts: what the plain calls compute."""
    kv = [n + k for n, k in zip(new, past)]
    b = ref.Batch(new, kv, page=16, kv_heads=2, dim=128, pad=3, seed=2)
    buf.set_active_shape([b.T, 256])
    _, parents = trees(b, "chain")
    q, k, v = b.randn(b.T, 8, 128), b.randn(b.T, 2, 128), b.randn(b.T, 2, 128)
    angle = torch.rand(2000, 64, generator=b.gen, device="cuda") * 6
    args = (q, k, v, angle.cos(), angle.sin(), b.starts, b.lens, b.table)
    caches = [(b.k_cache.clone(), b.v_cache.clone()) for _ in range(2)]
    n = sum(new)
    one, two = buf.kv_append(*args, *caches[0])[:n], buf.kv_append(*args, *caches[1], parents=parents)[:n]
    ok(buf)
    assert torch.equal(one, two) and all(torch.equal(x, y) for x, y in zip(*caches))
    for window, sinks in ((0, 0), (50, 2), (200, 0)):
        run(buf, b, 8, 128, "chain", window=window, sinks=sinks)


# ---------------------------------------------------------------- accept

def check_accept(b, per, leaves, before, new_lens):
    want = [c.clone() for c in before]
    lens = []
    for s, (n, total) in enumerate(zip(b.new, b.kv)):
        path = sr.paths(per[s])[leaves[s]] if leaves[s] >= 0 else []
        lens.append(total - n + len(path))
        if path:
            a = torch.tensor(path, device="cuda") + total - n
            z = torch.arange(len(path), device="cuda") + total - n
            row = b.table[s].long()
            for c, old in zip(want, before):
                c[row[z // b.page], :, z % b.page] = old[row[a // b.page], :, a % b.page]
    assert new_lens.tolist() == lens
    assert torch.equal(b.k_cache, want[0]) and torch.equal(b.v_cache, want[1])


@pytest.mark.parametrize("kind", ["bushy", "chain", "flat"])
@pytest.mark.parametrize("dim,page,kv_heads", [(128, 16, 2), (64, 8, 5), (64, 64, 1), (128, 128, 32)])
def test_accept(buf, kind, dim, page, kv_heads):
    new = [1, 5, 0, 64, 17, 33, 200, 8, 9]
    kv = [n + past for n, past in zip(new, [0, 123, 40, 64, 700, 95, 254, 3, 7])]
    b = ref.Batch(new, kv, page=page, kv_heads=kv_heads, dim=dim, seed=dim)
    rng = random.Random(page)
    per, parents = trees(b, kind)
    leaves = [-1 if n == 0 or i == 7 else rng.randint(max(0, n - 4), n - 1) for i, n in enumerate(new)]
    before = b.k_cache.clone(), b.v_cache.clone()
    new_lens = buf.kv_accept(b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents,
                             torch.tensor(leaves, dtype=torch.int32, device="cuda"))
    ok(buf)
    check_accept(b, per, leaves, before, new_lens)


def test_accept_on_strided_caches(buf):
    """Caches that are views: keys and values of one tensor, pages inside the heads."""
    b = ref.Batch([30, 12], [100, 40], page=16, kv_heads=3, dim=64, seed=1)
    whole = torch.randn(2, 3, b.pages, 16, 64, device="cuda").bfloat16()
    b.k_cache, b.v_cache = whole[0].transpose(0, 1), whole[1].transpose(0, 1)
    per, parents = trees(b)
    before = b.k_cache.clone(), b.v_cache.clone()
    leaves = torch.tensor([29, 10], dtype=torch.int32, device="cuda")
    new_lens = buf.kv_accept(b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents, leaves)
    ok(buf)
    check_accept(b, per, [29, 10], before, new_lens)


def test_accept_of_the_longest_trees(buf):
    n = ub.ACCEPT_MOST
    b = ref.Batch([n, n + 1], [n + 5, n + 9], page=64, kv_heads=1, dim=64, seed=1)
    per, parents = trees(b)
    before = b.k_cache.clone(), b.v_cache.clone()
    leaves = torch.tensor([n - 1, n], dtype=torch.int32, device="cuda")
    new_lens = buf.kv_accept(b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents, leaves)
    torch.cuda.synchronize()
    assert buf.query_status() == ub.CODES["UB_ERR_ARG"]  # of the second one
    buf.clear_status()
    check_accept(b, per, [n - 1, -1], before, new_lens)


@pytest.mark.parametrize("leaf,parent,starts,length", [(6, None, None, 50), (-2, None, None, 50), (5, 5, None, 50), (5, 4, [0, 7], 50),
                                                       (5, 4, [-1, 5], 50), (5, 4, None, 3), (5, 4, None, 99)])
def test_accept_reports_what_is_wrong(buf, leaf, parent, starts, length):
    """Nothing outside the sequence's pages is touched, and the status says so."""
    b = ref.Batch([6], [50], page=16, kv_heads=1, dim=64, seed=3)
    per, parents = trees(b, "chain")
    if parent is not None:
        parents[5] = parent
    if starts is not None:
        b.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
    keep = torch.ones(b.pages, dtype=torch.bool, device="cuda")
    keep[b.table[0].long()] = False
    before = b.k_cache.clone()
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    buf.kv_accept(b.k_cache, b.v_cache, b.starts, lens, b.table, parents, torch.tensor([leaf], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert buf.query_status() == ub.CODES["UB_ERR_ARG"]
    buf.clear_status()
    assert torch.equal(b.k_cache[keep], before[keep])


def test_accept_refuses_lengths_in_place(buf):
    b = ref.Batch([6], [50], page=16, kv_heads=1, dim=64)
    _, parents = trees(b)
    leaves = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ub.UbError):
        buf.kv_accept(b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents, leaves, new_lens=b.lens)
    with pytest.raises((TypeError, ValueError)):
        buf.kv_accept(b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents.long(), leaves)


def test_accept_refuses_what_it_reads_as_new_lengths(buf):
    b = ref.Batch([6, 2], [50, 9], page=16, kv_heads=1, dim=64)
    _, parents = trees(b)
    leaves = torch.zeros(2, dtype=torch.int32, device="cuda")
    for new_lens in (leaves, b.starts[:2], b.starts[1:], parents[:2], parents[-2:], b.table.view(-1)[:2], b.lens):
        with pytest.raises(ub.UbError):
            buf.kv_accept(b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents, leaves, new_lens=new_lens)
    ok(buf)
    assert leaves.tolist() == [0, 0] and b.lens.tolist() == [50, 9]
