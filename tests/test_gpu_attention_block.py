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
