"""The pages of a cache against plain lists: taking, freeing, forking, moving together, copying; and
what they are for, a run of forked and drafted decoding."""
import random

import pytest
import torch

import serve_ref as sr
from gemm_overlap_gemms_gb300 import ub

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def buf():
    from gemm_overlap_gemms_gb300 import _build
    _build.build()
    with ub.UserBuffer([1024, 256], 1) as b:
        yield b


def status(buf, name="UB_OK"):
    torch.cuda.synchronize()
    got = buf.query_status()
    buf.clear_status()
    assert got == (0 if name == "UB_OK" else ub.CODES[name])


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pool:
    """Lists and device arrays of a pool with `n` rows of which some hold pages."""

    def __init__(self, n, width, pages, page=16, seed=0, fill=0.5, room=0):
        rng = random.Random(seed)
        order = list(range(pages))
        rng.shuffle(order)
        self.page, self.rng = page, rng
        self.refs, self.table, self.lens = [0] * pages, [], []
        for _ in range(n):
            length = rng.randint(0, int(width * page * fill))
            need = -(-length // page)
            if need > len(order) - room:
                length = need = 0
            row = [order.pop() for _ in range(need)]
            for p in row:
                self.refs[p] += 1
            self.table.append(row + [-1] * (width - need))
            self.lens.append(length)
        self.width = width

    def device(self, pitch=None):
        t = torch.full((len(self.table), pitch or self.width), -7, dtype=torch.int32, device="cuda")[:, :self.width]
        t.copy_(ints(self.table))
        return ints(self.refs), t


@pytest.mark.parametrize("n,width,pages,page,pitch", [(1, 1, 1, 16, None), (3, 9, 40, 16, 13), (40, 33, 900, 8, None), (200, 70, 9000, 256, 71),
                                                      (7, 2000, 70001, 64, None), (1500, 40, 40000, 32, None)])
def test_take_and_free(buf, n, width, pages, page, pitch):
    pool = Pool(n, width, pages, page, seed=n)
    refs, table = pool.device(pitch)
    cap = width * page
    for step in range(3):
        b = [pool.rng.randint(0, cap) for _ in range(n)]
        e = [min(cap, x + pool.rng.choice((0, 1, page, 3 * page + 1))) for x in b]
        b[0] = e[0] if step else b[0]
        want = sr.take(pool.refs, pool.table, b, e, page)
        buf.kv_take(refs, table, ints(b), ints(e), page)
        status(buf, "UB_ERR_CAPACITY" if want[2] else "UB_OK")
        pool.refs, pool.table = want[:2]
        assert refs.tolist() == pool.refs and table.tolist() == pool.table
        b = [pool.rng.randint(-5, cap) for _ in range(n)]
        e = [pool.rng.choice((x, x + 4 * page, 1 << 30)) for x in b]
        pool.refs, pool.table = sr.give_up(pool.refs, pool.table, b, e, page)
        buf.kv_free(refs, table, ints(b), ints(e), page)
        status(buf)
        assert refs.tolist() == pool.refs and table.tolist() == pool.table
    if pitch:  # what lies between the rows
        assert (table.as_strided((n, pitch - width), (pitch, 1), width) == -7).all()


def test_take_with_too_few_pages(buf):
    """The last entries stay missing; the rest have their pages."""
    refs, table = ints([1, 0, 5, 0, 0]), ints([[-1, -1, -1], [2, -1, -1]])
    buf.kv_take(refs, table, ints([0, 0]), ints([16, 48]), 16)
    status(buf)
    assert table.tolist() == [[1, -1, -1], [2, 3, 4]] and refs.tolist() == [1, 1, 5, 1, 1]
    buf.kv_take(refs, table, ints([0, 0]), ints([48, 48]), 16)
    status(buf, "UB_ERR_CAPACITY")
    assert table.tolist() == [[1, -1, -1], [2, 3, 4]] and refs.tolist() == [1, 1, 5, 1, 1]


def test_take_outside_the_table_is_cut_and_recorded(buf):
    refs, table = ints([0] * 5), ints([[-1, -1], [-1, -1]])
    buf.kv_take(refs, table, ints([-20, 40]), ints([1, 80]), 16)
    status(buf, "UB_ERR_ARG")
    assert table.tolist() == [[0, -1], [-1, -1]] and refs.tolist() == [1, 0, 0, 0, 0]


def test_freeing_what_is_free_is_recorded(buf):
    refs, table = ints([1, 0, 3]), ints([[0, 0, 1], [2, 9, -1]])
    buf.kv_free(refs, table, ints([0, 0]), ints([1000, 1000]), 16)
    status(buf, "UB_ERR_ARG")
    assert table.tolist() == [[-1] * 3] * 2 and refs.tolist() == [0, 0, 2]


@pytest.mark.parametrize("n,width,pages,children,page,pitch", [(1, 1, 4, 1, 16, None), (3, 9, 60, 20, 16, 12), (40, 33, 2000, 300, 8, None),
                                                               (64, 200, 20000, 512, 128, None), (5, 40, 140, 200, 16, None)])
def test_fork(buf, n, width, pages, children, page, pitch):
    pool = Pool(n, width, pages, page, seed=children)
    pool.table[0] = pool.table[0][:width - 1] + [-1]
    refs, table = pool.device(pitch)
    source = [pool.rng.randrange(n) for _ in range(children)]
    new = torch.full((children, pitch or width), -7, dtype=torch.int32, device="cuda")[:, :width]
    copies = buf.kv_fork(refs, table, ints(pool.lens), ints(source), new, page)
    want = sr.fork(pool.refs, pool.table, pool.lens, source, page)
    short = [c for c, s in zip(want[2], source) if c[1] < 0 and pool.lens[s] % page and pool.table[s][pool.lens[s] // page] >= 0]
    status(buf, "UB_ERR_CAPACITY" if short else "UB_OK")
    assert refs.tolist() == want[0] and new.tolist() == want[1] and copies.tolist() == want[2]
    assert table.tolist() == pool.table
    # and given up again, everything is as it was
    buf.kv_free(refs, new, ints([0] * children), ints([width * page] * children), page)
    status(buf)
    assert refs.tolist() == pool.refs and (new == -1).all()


def test_fork_of_what_is_not_there(buf):
    """A source out of range, a length past the table, an entry outside the pool, holes of a window."""
    refs, table = ints([1, 1, 1, 0, 0, 0]), ints([[0, -1, 1], [2, 77, -1]])
    new = torch.zeros(4, 3, dtype=torch.int32, device="cuda")
    copies = buf.kv_fork(refs, table, ints([40, 20]), ints([0, 5, 1, -1]), new, 16)
    status(buf, "UB_ERR_ARG")
    assert new.tolist() == [[0, -1, 3], [-1] * 3, [2, -1, -1], [-1] * 3]
    assert copies.tolist() == [[1, 3], [-1, -1], [-1, -1], [-1, -1]] and refs.tolist() == [2, 1, 2, 1, 0, 0]
    copies = buf.kv_fork(refs, table, ints([1000, 20]), ints([0]), new[:1], 16)
    status(buf, "UB_ERR_ARG")
    assert new[0].tolist() == [0, -1, 1] and copies.tolist() == [[-1, -1]]


@pytest.mark.parametrize("n,width,pages,fill", [(1, 1, 1, 1.0), (1, 1, 2, 1.0), (3, 9, 40, 0.5), (40, 33, 900, 0.5), (300, 100, 30000, 0.9),
                                                (5, 300, 100000, 0.2), (20, 30, 601, 1.0)])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(buf, n, width, pages, fill, in_place):
    pool = Pool(n, width, pages, seed=pages, fill=fill)
    if n > 2:
        pool.table[1] = list(pool.table[2])  # shared pages, and one that is kept without an entry
        for p in pool.table[2]:
            if p >= 0:
                pool.refs[p] += 1
        pool.refs[pages - 1] += 1
    refs, table = pool.device()
    want = sr.compact(pool.refs, pool.table)
    out = {} if in_place else {"refs_out": torch.full_like(refs, -9), "table_out": torch.full_like(table, -9)}
    moves, used = buf.kv_compact(refs, table, **out)
    status(buf)
    r, t = (refs, table) if in_place else (out["refs_out"], out["table_out"])
    assert r.tolist() == want[0] and t.tolist() == want[1] and used.tolist() == [want[3]]
    assert moves.tolist() == want[2] + [[-1, -1]] * (pages // 2 - len(want[2]))
    if not in_place:
        assert refs.tolist() == pool.refs and table.tolist() == pool.table
    again, _ = buf.kv_compact(r, t)
    status(buf)
    assert (again == -1).all() and t.tolist() == want[1]


@pytest.mark.parametrize("heads,page,dim,pages,count", [(1, 8, 64, 5, 2), (3, 16, 128, 40, 11), (8, 128, 128, 60, 20), (2, 256, 64, 9, 3),
                                                        (5, 32, 64, 3000, 1000)])
@pytest.mark.parametrize("view", [False, True])
def test_copy(buf, heads, page, dim, pages, count, view):
    if view:  # keys and values of one tensor, the heads outside the pages
        whole = torch.randn(2, heads, pages, page, dim, device="cuda").bfloat16()
        k, v = whole[0].transpose(0, 1), whole[1].transpose(0, 1)
    else:
        k, v = (torch.randn(pages, heads, page, dim, device="cuda").bfloat16() for _ in range(2))
    order = torch.randperm(pages, device="cuda").to(torch.int32)
    pairs = torch.stack((order[:count], order[count:2 * count]), 1).contiguous()
    pairs[count // 2] = -1
    want = [c.clone() for c in (k, v)]
    real = pairs[pairs[:, 0] >= 0].long()
    for c in want:
        c[real[:, 1]] = c[real[:, 0]]
    buf.kv_copy(k, v, pairs)
    status(buf)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_copy_of_pages_outside_the_cache_is_recorded(buf):
    k, v = (torch.randn(6, 2, 16, 64, device="cuda").bfloat16() for _ in range(2))
    want = k.clone()
    want[5] = want[0]
    buf.kv_copy(k, v, ints([[0, 5], [1, 6], [7, 2], [-1, 3], [4, -2], [-1, -1]]))
    status(buf, "UB_ERR_ARG")
    assert torch.equal(k, want)
    buf.kv_copy(k, v, torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    status(buf)


def test_a_cache_past_32_bits(buf):
    """Pages whose elements lie past 2^32."""
    k, v = (torch.zeros(40000, 8, 128, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[1], v[39998] = 3, 5
    buf.kv_copy(k, v, ints([[1, 39999], [39998, 2]]))
    status(buf)
    assert (k[39999] == 3).all() and (v[2] == 5).all() and (v[39999] == 0).all() and int((k != 0).any(-1).any(-1).any(-1).sum()) == 2


def test_pages_from_a_graph(buf):
    """A captured step of taking and freeing, replayed with new lengths."""
    pool = Pool(6, 20, 200, seed=1)
    refs, table = pool.device()
    lens, zero, cap = ints(pool.lens), ints([0] * 6), ints([320] * 6)
    graph, after = torch.cuda.CUDAGraph(), lens.clone()
    buf.kv_take(refs.clone(), table.clone(), lens, lens, 16)
    with torch.cuda.graph(graph):
        after.copy_(lens + 5)
        buf.kv_take(refs, table, lens, after, 16)
    for _ in range(3):
        graph.replay()
        pool.refs, pool.table, _ = sr.take(pool.refs, pool.table, pool.lens, [n + 5 for n in pool.lens], 16)
        pool.lens = [n + 5 for n in pool.lens]
        status(buf)
        assert refs.tolist() == pool.refs and table.tolist() == pool.table
        lens.copy_(after)
    buf.kv_free(refs, table, zero, cap, 16)
    status(buf)
    assert (refs == 0).all() and (table == -1).all()


def test_refused_calls(buf):
    pool = Pool(4, 10, 50)
    refs, table = pool.device()
    lens, source = ints(pool.lens), ints([0, 1])
    new = torch.zeros(2, 10, dtype=torch.int32, device="cuda")
    for bad in (lambda: buf.kv_take(refs.long(), table, lens, lens, 16), lambda: buf.kv_take(refs, table, lens[:3], lens, 16),
                lambda: buf.kv_take(refs, table.t(), lens, lens, 16), lambda: buf.kv_take(refs, None, lens, lens, 16),
                lambda: buf.kv_take(refs, table, lens, lens, 17), lambda: buf.kv_free(refs, table, lens, lens, 4),
                lambda: buf.kv_fork(refs, table, lens, source, new[:1], 16), lambda: buf.kv_fork(refs, table, lens, source, new[:, :9], 16),
                lambda: buf.kv_fork(refs, table, lens, source, table[1:3], 16),
                lambda: buf.kv_fork(refs, table, lens, source, new, 16, copies=new[:, :2]),
                lambda: buf.kv_compact(refs, table, moves=torch.zeros(24, 2, dtype=torch.int32, device="cuda")),
                lambda: buf.kv_compact(refs, table, refs_out=refs[:49]), lambda: buf.kv_compact(refs, table, table_out=new),
                lambda: buf.kv_compact(refs, table[1:], table_out=table[:-1]),
                lambda: buf.kv_copy(new, new, new), lambda: buf.kv_copy(torch.zeros(3, 2, 16, 96, device="cuda").bfloat16(), None, new)):
        with pytest.raises((TypeError, ValueError, ub.UbError)):
            bad()
    with pytest.raises(ub.UbError):
        k = torch.zeros(3, 2, 16, 96, device="cuda").bfloat16()
        buf.kv_copy(k, k, torch.zeros(1, 2, dtype=torch.int32, device="cuda"))
    status(buf)
    assert refs.tolist() == pool.refs and table.tolist() == pool.table


def test_overlapping_arrays_are_refused(buf):
    """What a call writes among what it reads, or among what else it writes."""
    pool = Pool(4, 10, 50)
    refs, table = pool.device()
    lens, source = ints(pool.lens), ints([0, 1])
    new = torch.zeros(2, 10, dtype=torch.int32, device="cuda")
    scratch = torch.zeros(200, dtype=torch.int32, device="cuda")
    moves = scratch[:50].view(25, 2)
    pairs = lambda t: t.reshape(-1)[:4].view(2, 2)
    for bad in (lambda: buf.kv_take(refs, table, refs[:4], lens, 16), lambda: buf.kv_free(refs, table, lens, table[1, :4], 16),
                lambda: buf.kv_free(refs, refs[:40].view(4, 10), lens, lens, 16),
                lambda: buf.kv_fork(refs, table, lens, source, new, 16, copies=pairs(new)),
                lambda: buf.kv_fork(refs, table, lens, source, new, 16, copies=pairs(refs)),
                lambda: buf.kv_fork(refs, table, lens, source, new, 16, copies=pairs(table)),
                lambda: buf.kv_fork(refs, table, lens, source, new, 16, copies=pairs(lens)),
                lambda: buf.kv_fork(refs, table, lens, source, refs[:20].view(2, 10), 16),
                lambda: buf.kv_fork(refs, table, lens, pairs(new)[0], new, 16),
                lambda: buf.kv_compact(refs, table, moves=moves, used=scratch[49:50]),
                lambda: buf.kv_compact(refs, table, refs_out=scratch[:50], moves=moves),
                lambda: buf.kv_compact(refs, table, table_out=scratch[10:50].view(4, 10), refs_out=scratch[:50]),
                lambda: buf.kv_compact(refs, table, moves=moves, used=refs[:1]),
                lambda: buf.kv_compact(refs, table, moves=moves, used=table[0, :1])):
        with pytest.raises(ub.UbError):
            bad()
    status(buf)
    assert refs.tolist() == pool.refs and table.tolist() == pool.table and not scratch.any() and not new.any()


def test_forked_drafted_decoding(buf):
    """The operators together, as a server uses them: a prompt forked into candidates, each with its
    own drafts, verified, the accepted ones kept, pages taken, given up and moved together; against
    attention over each candidate's own keys and values, kept as plain tensors."""
    import attn_ref as ref
    page, heads, G, D, window, sinks = 16, 8, 2, 64, 40, 2
    pages, width, cap = 120, 12, 12 * 16
    gen = torch.Generator(device="cuda").manual_seed(0)
    rng = random.Random(3)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()
    k_cache, v_cache = (torch.full((pages, G, page, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[:30:3] = 1  # pages of others, so that compaction has something to do
    table = torch.full((5, width), -1, dtype=torch.int32, device="cuda")

    def append(rows, k, v, starts, lens, parents=None):
        buf.set_active_shape([k.shape[0], 256])
        buf.kv_append(randn(k.shape[0], heads, D), k, v, None, None, starts, lens, rows, k_cache, v_cache, parents=parents)

    # a prompt of 37 tokens in row 0, forked into rows 1 .. 4
    own = randn(37, G, D), randn(37, G, D)
    buf.kv_take(refs, table[:1], ints([0]), ints([37]), page)
    append(table[:1], *own, ints([0, 37]), ints([37]))
    copies = buf.kv_fork(refs, table[:1], ints([37]), ints([0] * 4), table[1:], page)
    buf.kv_copy(k_cache, v_cache, copies)
    buf.kv_free(refs, table[:1], ints([0]), ints([cap]), page)
    seqs = [own] * 4
    rows = table[1:]
    for step in range(6):
        new = [rng.randint(1, 9) for _ in seqs]
        per = [sr.random_tree(n, rng) for n in new]
        text = [k.shape[0] for k, _ in seqs]
        starts = ints([0] + [sum(new[:i + 1]) for i in range(4)])
        total = ints([t + n for t, n in zip(text, new)])
        parents = ints([p for t in per for p in t])
        buf.kv_take(refs, rows, ints(text), total, page)
        drafts = [(randn(n, G, D), randn(n, G, D)) for n in new]
        append(rows, torch.cat([k for k, _ in drafts]), torch.cat([v for _, v in drafts]), starts, total, parents)
        q = randn(sum(new), heads, D)
        out = buf.attn_tree(q, k_cache, v_cache, starts, total, rows, parents, window=window, sinks=sinks)
        leaves = []
        at = 0
        for i, (n, tree) in enumerate(zip(new, per)):
            k, v = (torch.cat((a, b)).transpose(0, 1) for a, b in zip(seqs[i], drafts[i]))
            seen = sr.tree_seen(tree, text[i] + n, window, sinks).cuda()
            o, e, _, _ = sr.attend_seen(q[at:at + n], k, v, seen, D ** -0.5)
            ref.within(out[at:at + n], o, e, "step %d, candidate %d" % (step, i))
            at += n
            leaves.append(rng.randint(-1, n - 1))
            path = sr.paths(tree)[leaves[i]] if leaves[i] >= 0 else []
            seqs[i] = tuple(torch.cat((a, b[path])) for a, b in zip(seqs[i], drafts[i]))
        lens = buf.kv_accept(k_cache, v_cache, starts, total, rows, parents, ints(leaves))
        assert lens.tolist() == [k.shape[0] for k, _ in seqs]
        # the pages of rejected drafts, and those that the window has left
        end = -(-lens // page) * page
        buf.kv_free(refs, rows, end, ints([cap] * 4), page)
        buf.kv_free(refs, rows, ints([sinks] * 4), (lens - window).clamp_min(0).to(torch.int32), page)
        if step == 1:
            refs[:30:3] = 0  # the others go (none of those pages is ours yet)
        if step % 2:
            moves, used = buf.kv_compact(refs, table)
            buf.kv_copy(k_cache, v_cache, moves)
        q = randn(4, heads, D)
        buf.set_active_shape([4, 256])
        out = buf.attn_decode(q, k_cache, v_cache, lens, rows, window=window, sinks=sinks)
        for i, (k, v) in enumerate(seqs):
            n = k.shape[0]
            seen = sr.in_window(torch.tensor([n - 1], device="cuda"), torch.arange(n, device="cuda"), window, sinks)
            o, e, _, _ = sr.attend_seen(q[i:i + 1], k.transpose(0, 1), v.transpose(0, 1), seen, D ** -0.5)
            ref.within(out[i:i + 1], o, e, "decoding, step %d, candidate %d" % (step, i))
    status(buf)
    count = torch.zeros(pages, dtype=torch.int32, device="cuda")
    named = table[table >= 0].long()
    count.index_add_(0, named, torch.ones_like(named, dtype=torch.int32))
    assert torch.equal(count, refs)  # every page is counted, and none is lost
