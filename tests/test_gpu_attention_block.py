"""The attention half of a layer: projections, append and attention together, against 64-bit
dense arithmetic, and decoding against the prompt of one token more."""
import pytest
import torch

from gemm_overlap_gemms_gb300 import attention_block as ab
from gemm_overlap_gemms_gb300 import synth, ub

pytestmark = pytest.mark.gpu

TP, HIDDEN, HEADS, KV_HEADS, D, PAGE = 2, 256, 4, 2, 64, 16


@pytest.fixture(scope="module")
def block():
    from gemm_overlap_gemms_gb300 import _build
    _build.build()
    dev = torch.device("cuda")
    gen = synth.generator(dev)
    caches = [tuple(torch.full((40, KV_HEADS, PAGE, D), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2))
              for _ in range(TP)]
    Wqkv = [synth.normal_bf16(((HEADS + 2 * KV_HEADS) * D, HIDDEN), HIDDEN ** -0.5, gen, dev) for _ in range(TP)]
    Wo = [synth.normal_bf16((HIDDEN, HEADS * D), (TP * HEADS * D) ** -0.5, gen, dev) for _ in range(TP)]
    cos, sin = ab.rotation_tables(256, D)
    with ub.UserBuffer([256, HIDDEN], TP) as buf:
        yield ab.AttentionBlock(buf, Wqkv, Wo, HEADS, KV_HEADS, caches, cos, sin)


def dense(block, x):
    """One sequence [n, hidden] through the layer in 64 bits, nothing rounded."""
    n = x.shape[0]
    out = torch.zeros(n, HIDDEN, dtype=torch.float64, device=x.device)
    c, s = block.cos[:n].double()[:, None], block.sin[:n].double()[:, None]

    def turn(t):
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)
    for Wqkv, Wo in zip(block.Wqkv, block.Wo):
        y = (x.double() @ Wqkv.double().T).view(n, HEADS + 2 * KV_HEADS, D)
        q, k, v = turn(y[:, :HEADS]), turn(y[:, HEADS:HEADS + KV_HEADS]), y[:, HEADS + KV_HEADS:]
        k, v = (t.repeat_interleave(HEADS // KV_HEADS, 1) for t in (k, v))
        z = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
        z = z.masked_fill(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), -torch.inf)
        a = torch.einsum("hij,jhd->ihd", z.softmax(-1), v)
        out += a.reshape(n, HEADS * D) @ Wo.double().T
    return out


def close(got, want):
    """Five BF16 roundings on the way (QKV, rotation, weights, attention, output), each 2^-8 of
    values of about 1, spread over sums whose weights' squares add up to 1: the difference's
    root mean square stays under 5 roundings of the output's."""
    d = (got.double() - want).square().mean().sqrt()
    assert d <= 5 * 2.0 ** -8 * want.square().mean().sqrt(), d


def test_prompts_then_steps(block):
    buf = block.buf
    dev = torch.device("cuda")
    gen = synth.generator(dev, seed=3)
    lengths, steps = [37, 1, 90], 5
    x = [synth.normal_bf16((n + steps, HIDDEN), 1.0, gen, dev) for n in lengths]
    table = torch.randperm(40, device=dev)[:21].to(torch.int32).view(3, 7)
    want = [dense(block, t) for t in x]

    # Prompts in one packed microbatch.
    T = sum(lengths)
    buf.set_active_shape([T, HIDDEN])
    packed = torch.cat([t[:n] for t, n in zip(x, lengths)])
    starts = torch.tensor([0, 37, 38, 128], dtype=torch.int32, device=dev)
    lens = torch.tensor(lengths, dtype=torch.int32, device=dev)
    got = torch.cat(block.prompt(list(packed.view(TP, T // TP, HIDDEN)), starts, lens, table))
    torch.cuda.synchronize()
    assert buf.query_status() == ub.UB_OK
    for i, n in enumerate(lengths):
        close(got[starts[i]:starts[i] + n], want[i][:n])

    # Steps of the three sequences, in an active shape of four rows (the last is none's).
    buf.set_active_shape([4, HIDDEN])
    one = torch.arange(4, dtype=torch.int32, device=dev)
    for step in range(steps):
        lens += 1
        rows = torch.stack([t[n + step] for t, n in zip(x, lengths)] + [torch.zeros_like(x[0][0])])
        got = torch.cat(block.step([rows[:2].contiguous(), rows[2:].contiguous()], one, lens, table))
        torch.cuda.synchronize()
        assert buf.query_status() == ub.UB_OK
        close(got[:3], torch.stack([w[n + step] for w, n in zip(want, lengths)]))
        assert (got[3] == 0).all()


def test_chunks_match_the_whole_prompt(block):
    """A prompt in chunks gives what it gives in one piece: the cache holds the same keys, and
    each row attends to the same ones."""
    buf = block.buf
    dev = torch.device("cuda")
    gen = synth.generator(dev, seed=4)
    n = 100
    x = synth.normal_bf16((n, HIDDEN), 1.0, gen, dev)
    table = torch.arange(7, dtype=torch.int32, device=dev).view(1, 7) + 30
    want = dense(block, x)
    done = 0
    for chunk in (40, 2, 58):
        buf.set_active_shape([chunk, HIDDEN])
        rows = x[done:done + chunk]
        done += chunk
        got = torch.cat(block.prompt(list(rows.view(TP, chunk // TP, HIDDEN)), torch.tensor([0, chunk], dtype=torch.int32, device=dev),
                                     torch.tensor([done], dtype=torch.int32, device=dev), table))
        torch.cuda.synchronize()
        assert buf.query_status() == ub.UB_OK
        close(got, want[done - chunk:done])


def _busy(ms=30):
    """Keep the current stream busy for some milliseconds."""
    torch.cuda._sleep(int(ms * 1.5e6))


def test_another_stream_beside_a_busy_current_one(block):
    """prompt and step on a stream of their own, while the current stream is behind and allocates:
    what they give on the current stream, bit for bit."""
    buf = block.buf
    dev = torch.device("cuda")
    gen = synth.generator(dev, seed=5)
    table = torch.randperm(40, device=dev)[:21].to(torch.int32).view(3, 7)
    starts = torch.tensor([0, 37, 38, 128], dtype=torch.int32, device=dev)
    lens = torch.tensor([37, 1, 90], dtype=torch.int32, device=dev)
    one, longer = torch.arange(4, dtype=torch.int32, device=dev), lens + 1
    x = [list(synth.normal_bf16((TP, n // TP, HIDDEN), 1.0, gen, dev)) for n in (128, 4)]

    def both(stream=None):
        buf.set_active_shape([128, HIDDEN])
        first = block.prompt(x[0], starts, lens, table, stream=stream)
        buf.set_active_shape([4, HIDDEN])
        return first + block.step(x[1], one, longer, table, stream=stream)
    want = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        _busy()
        got = both(side)
        for _ in range(8):     # the current stream's own allocations, behind its work
            torch.full((128, HEADS, D), float("nan"), dtype=torch.bfloat16, device=dev)
        torch.cuda.synchronize()
        assert buf.query_status() == ub.UB_OK
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_captured_step_with_new_lengths(block):
    """A step captured into a graph and replayed with new tokens and lengths: what the same steps
    give outside it."""
    buf = block.buf
    dev = torch.device("cuda")
    gen = synth.generator(dev, seed=6)
    table = torch.arange(21, dtype=torch.int32, device=dev).view(3, 7)
    one = torch.arange(4, dtype=torch.int32, device=dev)
    lens = torch.zeros(3, dtype=torch.int32, device=dev)
    x = [torch.zeros(2, HIDDEN, dtype=torch.bfloat16, device=dev) for _ in range(TP)]
    tokens = [synth.normal_bf16((TP, 2, HIDDEN), 1.0, gen, dev) for _ in range(6)]
    counts = [torch.tensor(n, dtype=torch.int32, device=dev) for n in ([1, 1, 1], [2, 2, 2], [3, 2, 3], [4, 3, 4], [5, 4, 4], [6, 5, 5])]
    buf.set_active_shape([4, HIDDEN])

    def put(i):
        for s, t in zip(x, tokens[i]):
            s.copy_(t)
        lens.copy_(counts[i])
    want = []
    for i in range(6):
        put(i)
        want.append([y.clone() for y in block.step(x, one, lens, table)])
    torch.cuda.synchronize()
    for c in block.caches:
        for t in c:
            t[:21] = float("nan")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = block.step(x, one, lens, table, stream=side)
    for i in range(6):
        put(i)
        graph.replay()
        torch.cuda.synchronize()
        assert buf.query_status() == ub.UB_OK
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
