"""The attention operators where a wait runs out, beside ub_clear_status, and back to back on the
same counters."""
import pytest
import torch

import attn_ref as ref
from gemm_overlap_gemms_gb300 import ub
from gpu_helpers import sentinel

pytestmark = pytest.mark.gpu

TIMEOUT = ub.CODES["UB_ERR_TIMEOUT"]


@pytest.fixture(scope="module")
def buf():
    from gemm_overlap_gemms_gb300 import _build
    _build.build()
    with ub.UserBuffer([4096, 256], 1) as b:
        yield b


class Call:
    """One attention call, its 64-bit definition, and what it gave first."""

    def __init__(self, buf, op, new, kv, heads=4, kv_heads=2, dim=64, seed=0):
        self.buf, self.op = buf, op
        self.b = b = ref.Batch(new, kv, page=32, kv_heads=kv_heads, dim=dim, seed=seed, fill=float("nan"))
        self.q = b.randn(b.T, heads, dim, std=1.5)
        self.k, self.v = (b.randn(b.T, kv_heads, dim) for _ in range(2))

    def __call__(self):
        b, buf = self.b, self.buf
        buf.set_active_shape([b.T, 256])
        out = sentinel(self.q.shape)
        if self.op == "decode":
            return buf.attn_decode(self.q, b.k_cache, b.v_cache, b.lens, b.table, out=out)
        if self.op == "paged":
            return buf.attn_prompt_paged(self.q, b.k_cache, b.v_cache, b.starts, b.lens, b.table, out=out)
        return buf.attn_prompt(self.q, self.k, self.v, b.starts, out=out)

    def check(self, out):
        b = self.b
        for s, n in enumerate(b.new):
            t0, t1 = b.starts_list[s], b.starts_list[s + 1]
            k, v = (b.rows(c, s) if self.op != "packed" else x[t0:t1].transpose(0, 1)
                    for c, x in ((b.k_cache, self.k), (b.v_cache, self.v)))
            last = torch.arange(k.shape[1] - n, k.shape[1], device="cuda")
            o, e, _, _ = ref.attend(self.q[t0:t1], k, v, last, self.q.shape[2] ** -0.5)
            ref.within(out[t0:t1], o, e, "%s, sequence %d" % (self.op, s))


@pytest.fixture(scope="module")
def calls(buf):
    """Items by tickets; prompts split over their keys, each in its own way; decoding with items
    split over more than 8 CTAs, over fewer, and whole."""
    return [Call(buf, "packed", [900, 1, 130, 300, 64, 700, 17], [0] * 7, heads=8, kv_heads=8, seed=1),
            Call(buf, "paged", [16], [30000], seed=2), Call(buf, "paged", [64, 64], [2000, 1999], dim=128, seed=3),
            Call(buf, "decode", [1], [50000], seed=4), Call(buf, "decode", [1] * 12, [3000 + 70 * i for i in range(12)], seed=5),
            Call(buf, "decode", [1] * 40, [7 * i for i in range(40)], dim=128, seed=6), Call(buf, "paged", [5, 300], [9000, 1500], seed=7)]


def ok(buf):
    torch.cuda.synchronize()
    assert buf.query_status() == ub.UB_OK


def rounds(calls, n):
    """n rounds of the calls, back to back, each with its own output."""
    return [(c, c()) for _ in range(n) for c in calls]


def same(got, calls, first):
    for i, (c, out) in enumerate(got):
        assert torch.equal(out, first[calls.index(c)]), (i, c.op)


@pytest.fixture(scope="module")
def first(buf, calls):
    outs = []
    for c in calls:
        outs.append(c())
        ok(buf)
        c.check(outs[-1])
    return outs


def test_calls_that_split_differently_back_to_back(buf, calls, first):
    """Every launch keeps its own output and nothing is waited for in between: calls that share
    workspace, tickets and counters are right although their launches overlap."""
    got = rounds(calls, 20)
    ok(buf)
    same(got, calls, first)


def test_clear_status_beside_calls_in_flight(buf, calls, first):
    """No call loses a count to it, whether it is before, in or behind the calls."""
    got = []
    for _ in range(15):
        got += rounds(calls, 2)
        buf.clear_status()
    ok(buf)
    same(got, calls, first)


def long_prompt(pages, width):
    """16 tokens over a table of `width` entries that names few pages: half a millisecond."""
    b = ref.Batch([16], [pages * 64], page=64, kv_heads=1, dim=64, free=0, seed=8)
    b.table = (torch.arange(width, device="cuda") % pages).to(torch.int32).view(1, width)
    b.lens.fill_(64 * width)
    return b


def run_out(buf, call, tries=20):
    """Calls with waits of at most a microsecond, until one has run out."""
    limit = buf.get_option("timeout_ns")
    buf.set_option("timeout_ns", 1000)
    try:
        for _ in range(tries):
            call()
            torch.cuda.synchronize()
            code = buf.query_status()
            if code != ub.UB_OK:
                return code
    finally:
        buf.set_option("timeout_ns", limit)
    return ub.UB_OK


@pytest.mark.parametrize("in_flight", [False, True])
def test_a_split_prompt_whose_wait_runs_out(buf, calls, first, in_flight):
    """The status says so; after ub_clear_status everything is as before, also where more calls were
    in flight when it was called."""
    b = long_prompt(64, 120000)
    q = b.randn(16, 4, 64)

    def call():
        buf.set_active_shape([16, 256])
        buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table)
    assert run_out(buf, call) == TIMEOUT
    if in_flight:
        rounds(calls, 3)
    buf.clear_status()
    ok(buf)
    got = rounds(calls, 2)
    ok(buf)
    same(got, calls, first)


@pytest.mark.parametrize("in_flight", [False, True])
def test_a_join_of_many_parts_whose_wait_runs_out(buf, calls, first, in_flight):
    """One sequence over all SMs, half of it from few pages: those SMs are done sooner, and wait."""
    pages = 1 << 15
    k = torch.randn(pages, 1, 64, 64, device="cuda", dtype=torch.bfloat16)
    table = torch.arange(2 * pages, device="cuda").to(torch.int32).view(1, -1)
    table[0, pages:] %= 8
    lens = torch.full((1,), 128 * pages, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 8, 64, device="cuda").bfloat16()

    def call():
        buf.set_active_shape([1, 256])
        buf.attn_decode(q, k, k, lens, table)
    assert run_out(buf, call) == TIMEOUT
    if in_flight:
        rounds(calls, 3)
    buf.clear_status()
    ok(buf)
    got = rounds(calls, 2)
    ok(buf)
    same(got, calls, first)


def test_a_wait_that_runs_out_after_another_error(buf, calls, first):
    """The first error is the one that is kept; what the later call left counted is reset all the same."""
    b = long_prompt(64, 120000)
    q = b.randn(16, 4, 64)
    bad = b.table[:, :4].clone()
    bad[0, 1] = -1
    buf.set_active_shape([16, 256])
    buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, bad)
    torch.cuda.synchronize()
    assert buf.query_status() == ub.CODES["UB_ERR_ARG"]
    limit = buf.get_option("timeout_ns")
    buf.set_option("timeout_ns", 1000)
    for _ in range(5):
        buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, b.lens, b.table)
    buf.set_option("timeout_ns", limit)
    torch.cuda.synchronize()
    assert buf.query_status() == ub.CODES["UB_ERR_ARG"]
    buf.clear_status()
    ok(buf)
    got = rounds(calls, 2)
    ok(buf)
    same(got, calls, first)


def test_a_sequence_as_long_as_a_table_may_hold(buf):
    """Almost 2^31 keys: seven pages, named over and over by a table of 8388600 entries. Each distinct
    key then counts as often as it is seen.

    Bounds: those of attn_ref.attend, and the rounding of the fp32 sums over the key tiles of one SM's
    part: a step of the sum of weights per tile, 2^-24, and eight of the weighted sum, 2^-23 (the
    tensor core need not round to nearest)."""
    page, pages, width, n, heads, dim = 256, 7, 8388600, 3, 2, 64
    keys = page * width - 5
    b = ref.Batch([n], [page * pages], page=page, kv_heads=1, dim=dim, free=0, seed=9)
    table = (torch.arange(width, device="cuda") % pages).to(torch.int32).view(1, width)
    lens = torch.tensor([keys], dtype=torch.int32, device="cuda")
    q = b.randn(n, heads, dim, std=1.5)
    k, v = (c.transpose(0, 1).flatten(1, 2)[0].double() for c in (b.k_cache, b.v_cache))  # in page order
    s = torch.einsum("nhd,jd->nhj", q.double(), k) * dim ** -0.5
    seen = torch.arange(keys - n + 1, keys + 1, device="cuda")[:, None]
    times = seen // (page * pages) + (torch.arange(page * pages, device="cuda") < seen % (page * pages))
    w = torch.exp(s - s.amax(-1, keepdim=True)) * times[:, None]
    total = w.sum(-1)
    want, mag = ((w @ x) / total[..., None] for x in (v, v.abs()))
    want_lse = s.amax(-1) + total.log()
    tiles = keys / 128 / torch.cuda.get_device_properties(0).multi_processor_count + 1
    shift = 2.0 ** -19 * (1 + dim ** -0.5 * torch.einsum("nhd,jd->nhj", q.double().abs(), k.abs()).amax(-1))
    bound = mag * (2.1 * ref.U + 2 * shift[..., None] + tiles * 9 * 2.0 ** -23)
    for name in ("prompt", "decode"):
        rows = n if name == "prompt" else 1
        out = sentinel((rows, heads, dim))
        buf.set_active_shape([rows, 256])
        if name == "prompt":
            _, lse = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, b.starts, lens, table, out=out, lse=True)
            rows = slice(0, n)
        else:
            _, lse = buf.attn_decode(q[n - 1:], b.k_cache, b.v_cache, lens, table, out=out, lse=True)
            rows = slice(n - 1, n)
        ok(buf)
        ref.within(out, want[rows], bound[rows], name)
        ref.within(lse, want_lse[rows], shift[rows] + tiles * 2.0 ** -23, name + ", lse")


@pytest.mark.parametrize("starts", [[0, 5, 12], [-3, 5, 8], [0, 5, 2 ** 31 - 1], [-2 ** 31, 5, 9]])
def test_starts_past_the_active_tokens_are_cut_in_every_operator(buf, starts):
    """The tokens' positions follow the cut starts: append stores where the attention looks."""
    b = ref.Batch([5, 3], [25, 37], page=16, kv_heads=1, dim=64, seed=10)
    buf.set_active_shape([8, 256])
    q, k, v = b.randn(8, 2, 64), b.randn(8, 1, 64), b.randn(8, 1, 64)
    given = torch.tensor(starts, dtype=torch.int32, device="cuda")
    buf.kv_append(q, k, v, None, None, given, b.lens, b.table, b.k_cache, b.v_cache)
    got = buf.attn_prompt_paged(q, b.k_cache, b.v_cache, given, b.lens, b.table)
    ok(buf)
    for s, (t0, t1) in enumerate(((0, 5), (5, 8))):
        n = t1 - t0
        assert torch.equal(b.rows(b.k_cache, s)[0, -n:], k[t0:t1, 0]) and torch.equal(b.rows(b.v_cache, s)[0, -n:], v[t0:t1, 0])
        o, e, _, _ = ref.attend(q[t0:t1], b.rows(b.k_cache, s), b.rows(b.v_cache, s),
                                torch.arange(b.kv[s] - n, b.kv[s], device="cuda"), 0.125)
        ref.within(got[t0:t1], o, e, "sequence %d" % s)
