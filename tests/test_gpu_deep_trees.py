"""Drafts in deep trees that are no chains (deep_trees.py): attention with and without windows, the append,
accepted paths whose rows all move; and sequences of one draft, which decoding computes too."""
import random

import pytest
import torch

import attn_ref as ref
import serve_ref as sr
from deep_trees import KINDS, deep_tree
from gemm_overlap_gemms_gb300 import ub
from gpu_helpers import sentinel
from test_gpu_tree import check, check_accept

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


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def trees(b, kind, seed=0):
    per = [deep_tree(kind, n, seed) for n in b.new]
    return per, ints([p for t in per for p in t] + [12345] * (b.T - sum(b.new)))


def attend(buf, b, heads, dim, kind, window=0, sinks=0):
    buf.set_active_shape([b.T, 256])
    per, parents = trees(b, kind)
    q, out = b.randn(b.T, heads, dim, std=1.5), sentinel((b.T, heads, dim))
    _, lse = buf.attn_tree(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents, out=out, lse=True, window=window, sinks=sinks)
    ok(buf)
    check(b, q, per, out, lse, window, sinks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,page,heads,kv_heads", [(128, 16, 8, 2), (64, 128, 6, 6)])
def test_attention(buf, kind, dim, page, heads, kv_heads):
    """Paths through many words of 32 drafts and tiles of 128 keys, which begin anywhere in them."""
    new = [1, 64, 33, 200, 0, 97, 130, 500]
    kv = [n + past for n, past in zip(new, [0, 123, 40, 64, 9, 1700, 95, 3001])]
    b = ref.Batch(new, kv, page=page, kv_heads=kv_heads, dim=dim, pad=3, seed=dim, fill=float("nan"))
    attend(buf, b, heads, dim, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (33, 0), (64, 200), (100, 1), (300, 40), (2000, 0)])
def test_windows(buf, kind, window, sinks):
    """Windows that end on the path: in it, in the text right before it, and far from it."""
    new = [1, 64, 33, 200, 0, 97, 500]
    kv = [n + past for n, past in zip(new, [0, 123, 40, 64, 9, 1700, 95])]
    b = ref.Batch(new, kv, page=32, kv_heads=2, dim=64, pad=1, seed=window, fill=float("nan"))
    attend(buf, b, 4, 64, kind, window, sinks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 2)])
def test_large_trees(buf, kind, window, sinks):
    """Two query tiles to an item, and items split over CTAs: a path goes on where the CTA begins."""
    b = ref.Batch([700, 40], [1000, 30000], page=64, kv_heads=2, dim=128, pad=1, seed=3, fill=float("nan"))
    attend(buf, b, 8, 128, kind, window, sinks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(buf, kind, interleaved):
    """Every draft rotated by its own depth, wherever its path runs."""
    new, dim, heads, kv_heads = [5, 64, 0, 1, 33, 200, 1500], 64, 4, 2
    kv = [n + past for n, past in zip(new, [33, 100, 7, 0, 0, 31, 11])]
    b = ref.Batch(new, kv, page=16, kv_heads=kv_heads, dim=dim, pad=2, seed=1)
    buf.set_active_shape([b.T, 256])
    per, parents = trees(b, kind)
    q, k, v = b.randn(b.T, heads, dim), b.randn(b.T, kv_heads, dim), b.randn(b.T, kv_heads, dim)
    angle = torch.rand(1600, dim // 2, generator=b.gen, device="cuda") * 6
    cos, sin = angle.cos(), angle.sin()
    out = buf.kv_append(q, k, v, cos, sin, b.starts, b.lens, b.table, b.k_cache, b.v_cache, interleaved=interleaved, parents=parents)
    ok(buf)
    for s, (n, total) in enumerate(zip(new, kv)):
        if n == 0:
            continue
        a, place = b.starts_list[s], torch.arange(total - n, total, device="cuda")
        pos = torch.tensor([total - n + len(p) - 1 for p in sr.paths(per[s])], device="cuda")
        at = b.table[s].long()[place // 16], place % 16
        for x, got in ((q[a:a + n], out[a:a + n]), (k[a:a + n], b.k_cache[at[0], :, at[1]])):
            want, e = ref.rotate(x, cos[pos], sin[pos], interleaved)
            ref.within(got, want, e, "sequence %d" % s)
        assert torch.equal(b.v_cache[at[0], :, at[1]], v[a:a + n])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,page,kv_heads", [(128, 16, 2), (64, 8, 5), (64, 256, 1), (128, 64, 40)])
def test_accept(buf, kind, dim, page, kv_heads):
    """Paths of many more rows than are moved at once, almost all of them to another place and page."""
    new = [1, 64, 33, 200, 0, 500, 97, 3]
    kv = [n + past for n, past in zip(new, [0, 123, 40, 64, 9, 700, 250, 5])]
    b = ref.Batch(new, kv, page=page, kv_heads=kv_heads, dim=dim, seed=dim + page)
    per, parents = trees(b, kind, seed=page)
    deepest = [max(range(n), key=lambda i, up=sr.paths(t): len(up[i])) if n else -1 for n, t in zip(new, per)]
    moved = [sum(d != a for d, a in enumerate(sr.paths(t)[leaf])) if t else 0 for t, leaf in zip(per, deepest)]
    assert max(moved) >= 16
    rng = random.Random(page)
    for leaves in (deepest, [n - 1 for n in new], [rng.randint(-1, n - 1) for n in new]):
        before = b.k_cache.clone(), b.v_cache.clone()
        lens = buf.kv_accept(b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents, ints(leaves))
        ok(buf)
        check_accept(b, per, leaves, before, lens)


@pytest.mark.parametrize("kind", KINDS)
def test_accept_of_the_longest_trees(buf, kind):
    n = ub.ACCEPT_MOST
    b = ref.Batch([n, n - 1], [n + 5, n + 90], page=16, kv_heads=2, dim=64, seed=1)
    per, parents = trees(b, kind)
    leaves = [max(range(len(t)), key=lambda i, up=sr.paths(t): len(up[i])) for t in per]
    before = b.k_cache.clone(), b.v_cache.clone()
    lens = buf.kv_accept(b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents, ints(leaves))
    ok(buf)
    check_accept(b, per, leaves, before, lens)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 3), (700, 0)])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (5, 5, 64), (16, 1, 64)])
def test_one_draft_is_a_decoding_step(buf, window, sinks, heads, kv_heads, dim):
    """A draft of the text is the next token: decoding, a prompt's chunk of one token, a tree of one
    draft, each within its bound of the same definition."""
    kv = [1, 17, 128, 129, 900, 5000, 64, 30000]
    b = ref.Batch([1] * len(kv), kv, page=16, kv_heads=kv_heads, dim=dim, seed=dim, fill=float("nan"))
    buf.set_active_shape([b.T, 256])
    q, see = b.randn(b.T, heads, dim, std=1.5), {"window": window, "sinks": sinks}
    tree, tree_lse = buf.attn_tree(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, ints([-1] * b.T), lse=True, **see)
    step, step_lse = buf.attn_decode(q, b.k_cache, b.v_cache, b.lens, b.table, lse=True, **see)
    chunk, chunk_lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, lse=True, **see)
    ok(buf)
    for s, n in enumerate(kv):
        seen = sr.in_window(torch.tensor([n - 1], device="cuda"), torch.arange(n, device="cuda"), window, sinks)
        o, e, ll, le = sr.attend_seen(q[s:s + 1], b.rows(b.k_cache, s), b.rows(b.v_cache, s), seen, dim ** -0.5)
        for name, out, lse in (("tree", tree, tree_lse), ("decode", step, step_lse), ("prompt", chunk, chunk_lse)):
            ref.within(out[s:s + 1], o, e, "%s, %d keys" % (name, n))
            ref.within(lse[s:s + 1], ll, le, "lse of %s, %d keys" % (name, n))
