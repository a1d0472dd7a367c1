"""The serving operators where a wait runs out, under launch options, back to back with the others on
the same counters and workspace, on caches past 32 bits, and captured."""
import random

import pytest
import torch

import attn_ref as ref
import serve_ref as sr
from gemm_overlap_gemms_gb300 import ub

pytestmark = pytest.mark.gpu

TIMEOUT = ub.CODES["UB_ERR_TIMEOUT"]


@pytest.fixture(scope="module")
def buf():
    from gemm_overlap_gemms_gb300 import _build
    _build.build()
    with ub.UserBuffer([4096, 256], 1) as b:
        yield b


def ok(buf):
    torch.cuda.synchronize()
    assert buf.query_status() == ub.UB_OK


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Call:
    """One attention call, its 64-bit definition, and what it gave first."""

    def __init__(self, buf, op, new, kv, heads=4, kv_heads=2, dim=64, window=0, sinks=0, seed=0):
        self.buf, self.op, self.see = buf, op, {"window": window, "sinks": sinks}
        self.b = b = ref.Batch(new, kv, page=32, kv_heads=kv_heads, dim=dim, seed=seed, fill=float("nan"))
        self.q = b.randn(b.T, heads, dim, std=1.5)
        rng = random.Random(seed)
        self.trees = [sr.random_tree(n, rng) for n in new]
        self.parents = ints([p for t in self.trees for p in t])

    def __call__(self):
        b, buf = self.b, self.buf
        buf.set_active_shape([b.T, 256])
        if self.op == "tree":
            return buf.attn_tree(self.q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, self.parents, **self.see)
        if self.op == "decode":
            return buf.attn_decode(self.q, b.k_cache, b.v_cache, b.lens, b.table, **self.see)
        return buf.attn_prompt_paged(self.q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, **self.see)

    def check(self, out):
        b = self.b
        for s, (n, total) in enumerate(zip(b.new, b.kv)):
            a = b.starts_list[s]
            if self.op == "tree":
                seen = sr.tree_seen(self.trees[s], total, *self.see.values()).cuda()
            else:
                seen = sr.in_window(torch.arange(total - n, total, device="cuda"), torch.arange(total, device="cuda"), *self.see.values())
            o, e, _, _ = sr.attend_seen(self.q[a:a + n], b.rows(b.k_cache, s), b.rows(b.v_cache, s), seen, self.q.shape[2] ** -0.5)
            ref.within(out[a:a + n], o, e, "%s, sequence %d" % (self.op, s))


@pytest.fixture(scope="module")
def calls(buf):
    """Trees in whole items, in several rounds of them, in shares; windows split and whole."""
    return [Call(buf, "tree", [5, 20, 1], [300, 90, 1], heads=8, kv_heads=8, dim=128, seed=1),
            Call(buf, "tree", [16], [30000], heads=8, kv_heads=1, seed=2), Call(buf, "tree", [64, 40], [9000, 2000], heads=16, dim=128, seed=3),
            Call(buf, "tree", [2 + i % 9 for i in range(90)], [30 + 11 * i for i in range(90)], heads=4, kv_heads=4, seed=4),
            Call(buf, "tree", [60] * 6, [5000, 900, 70, 12000, 3000, 61], heads=8, window=2500, sinks=4, seed=5),
            Call(buf, "decode", [1], [50000], window=30000, sinks=1, seed=6), Call(buf, "decode", [1] * 12, [3000 + 70 * i for i in range(12)], seed=7),
            Call(buf, "prompt", [16], [30000], window=9000, sinks=40, seed=8),
            Call(buf, "prompt", [300] * 10, [5000] * 10, heads=8, kv_heads=8, window=2000, seed=9), Call(buf, "prompt", [64, 64], [2000, 1999], dim=128, seed=10)]


@pytest.fixture(scope="module")
def first(buf, calls):
    outs = [c() for c in calls]
    ok(buf)
    for c, out in zip(calls, outs):
        c.check(out)
    return outs


def test_back_to_back(buf, calls, first):
    """Many launches in flight, of all kinds: every result the same."""
    got = [(i, calls[i]()) for _ in range(8) for i in range(len(calls))]
    ok(buf)
    for i, out in got:
        assert torch.equal(out, first[i]), (i, calls[i].op)


@pytest.mark.parametrize("option,value", [("pdl", 0), ("sm_margin", 20), ("sm_margin", 100), ("sm_margin", 151)])
def test_launch_options(buf, calls, first, option, value):
    before = buf.get_option(option)
    buf.set_option(option, value)
    try:
        outs = [c() for c in calls]
        ok(buf)
    finally:
        buf.set_option(option, before)
    for c, out in zip(calls, outs):
        c.check(out)
    assert torch.equal(calls[1](), first[1])


@pytest.mark.parametrize("drafts", [9, 60])
@pytest.mark.parametrize("in_flight", [False, True])
def test_a_wait_that_runs_out(buf, calls, first, drafts, in_flight):
    """A tree over all SMs, half of its keys from few pages: those SMs are done sooner, and wait, here for
    a microsecond at most. The status says so; after ub_clear_status all calls give what they gave, also
    where more were in flight when it was called."""
    pages = 1 << 15
    k = torch.randn(pages, 1, 64, 64, device="cuda", dtype=torch.bfloat16)
    table = torch.arange(2 * pages, device="cuda").to(torch.int32).view(1, -1)
    table[0, pages:] %= 8
    q = torch.randn(drafts, 4, 64, device="cuda").bfloat16()
    args = (q, k, k, ints([0, drafts]), ints([128 * pages]), table, ints([i - 1 for i in range(drafts)]))
    limit = buf.get_option("timeout_ns")
    buf.set_option("timeout_ns", 1000)
    try:
        for _ in range(20):
            buf.set_active_shape([drafts, 256])
            buf.attn_tree(*args)
            torch.cuda.synchronize()
            code = buf.query_status()
            if code != ub.UB_OK:
                break
    finally:
        buf.set_option("timeout_ns", limit)
    assert code == TIMEOUT
    if in_flight:
        for c in calls:
            c()
    buf.clear_status()
    ok(buf)
    for _ in range(2):
        for c, want in zip(calls, first):
            assert torch.equal(c(), want), c.op
    ok(buf)


def test_profiled_calls(buf, calls, first):
    """Events around the launches, by operation."""
    buf.set_option("profile", 1)
    try:
        assert torch.equal(calls[1](), first[1])
        refs, table = ints([0] * 9), ints([[-1] * 3])
        buf.kv_take(refs, table, ints([0]), ints([40]), 16)
        assert buf.kernel_time("attn_tree")[1] == 1 and buf.kernel_time("kv_pages")[1] == 1
    finally:
        buf.set_option("profile", 0)
    ok(buf)


def test_caches_past_32_bits(buf):
    """Pages whose elements lie past 2^32, read by a tree and a window, moved by accepted drafts."""
    pages, G, page, D = 40000, 8, 128, 128
    k, v = (torch.zeros(pages, G, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    b = ref.Batch([30, 9], [200, 300], page=page, kv_heads=G, dim=D, seed=1)
    far = b.table.clone()
    far[b.table >= 0] = pages - 1 - b.table[b.table >= 0]
    used = b.table[b.table >= 0].long()
    k[pages - 1 - used], v[pages - 1 - used] = b.k_cache[used], b.v_cache[used]
    q = b.randn(b.T, 8, D)
    rng = random.Random(1)
    parents = ints([p for n in b.new for p in sr.random_tree(n, rng)])
    buf.set_active_shape([b.T, 256])
    for see in ({}, {"window": 40, "sinks": 3}):
        near = buf.attn_tree(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents, **see)
        assert torch.equal(near, buf.attn_tree(q, k, v, b.starts, b.lens, far, parents, **see))
        near = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, **see)
        assert torch.equal(near, buf.attn_prompt_paged(q, k, v, b.starts, b.lens, far, **see))
        near = buf.attn_decode(q, b.k_cache, b.v_cache, b.lens, b.table, **see)
        assert torch.equal(near[:2], buf.attn_decode(q, k, v, b.lens, far, **see)[:2])
    leaves = ints([29, 8])
    lens = buf.kv_accept(b.k_cache, b.v_cache, b.starts, b.lens, b.table, parents, leaves)
    assert torch.equal(lens, buf.kv_accept(k, v, b.starts, b.lens, far, parents, leaves))
    assert torch.equal(k[pages - 1 - used], b.k_cache[used]) and torch.equal(v[pages - 1 - used], b.v_cache[used])
    ok(buf)


def test_nothing_drafted_nothing_forked(buf):
    """Sequences without drafts are accepted as they are; no children, no pages, no pairs."""
    b = ref.Batch([0, 0], [20, 33], page=16, kv_heads=1, dim=64, seed=1)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    before = b.k_cache.clone()
    lens = buf.kv_accept(b.k_cache, b.v_cache, b.starts, b.lens, b.table, none, ints([-1, -1]))
    assert lens.tolist() == [20, 33] and torch.equal(before, b.k_cache)
    refs = ints([1] * b.pages)
    copies = buf.kv_fork(refs, b.table, b.lens, none, torch.empty(0, b.table.shape[1], dtype=torch.int32, device="cuda"), 16)
    assert copies.shape == (0, 2)
    buf.kv_copy(b.k_cache, b.v_cache, copies)
    ok(buf)


def test_a_captured_step_of_pages_and_drafts(buf):
    """Pages forked, copied and given up, a tree, accepted rows and a compaction in one graph, replayed on
    new contents, against the same calls one by one."""
    G, page, D, n = 2, 16, 64, 3
    rng = random.Random(4)

    def fresh(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        lens = [rng.randint(20, 90) for _ in range(n)]
        refs, rows = sr.take([0] * 80, [[-1] * 8] * n, [0] * n, lens, page)[:2]
        return {"refs": ints(refs), "table": ints(rows + [[-1] * 8] * n), "lens": ints(lens),
                "k": torch.randn(80, G, page, D, generator=g, device="cuda").bfloat16(),
                "v": torch.randn(80, G, page, D, generator=g, device="cuda").bfloat16(),
                "q": torch.randn(12, 4, D, generator=g, device="cuda").bfloat16(),
                "parents": ints([p for _ in range(n) for p in sr.random_tree(4, rng)]), "leaves": ints([rng.randint(-1, 3) for _ in range(n)])}
    starts, zero, end, order = ints([0, 4, 8, 12]), ints([0] * n), ints([128] * n), ints([2, 0, 1])

    def step(s):
        old, new = s["table"][:n], s["table"][n:]
        copies = buf.kv_fork(s["refs"], old, s["lens"], order, new, page)
        buf.kv_copy(s["k"], s["v"], copies)
        buf.kv_free(s["refs"], old, zero, end, page)
        lens = s["lens"][order.long()]
        total = lens + 4
        buf.kv_take(s["refs"], new, lens, total, page)
        out = buf.attn_tree(s["q"], s["k"], s["v"], starts, total, new, s["parents"], window=30, sinks=2)
        kept = buf.kv_accept(s["k"], s["v"], starts, total, new, s["parents"], s["leaves"])
        moves, used = buf.kv_compact(s["refs"], s["table"])
        buf.kv_copy(s["k"], s["v"], moves)
        return out, kept, used
    buf.set_active_shape([12, 256])
    static = fresh(0)
    step({k: v.clone() for k, v in static.items()})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = step(static)
    for seed in (1, 2, 3):
        s = fresh(seed)
        for key, value in s.items():
            static[key].copy_(value)
        graph.replay()
        want = step(s)
        ok(buf)
        assert all(torch.equal(a, b) for a, b in zip(results, want))
        assert all(torch.equal(static[key], s[key]) for key in ("refs", "table", "k", "v"))
