"""Windows, drafts and forked sequences through the attention block, against 64-bit dense
arithmetic of every path, and its example."""
import random

import pytest
import torch

import serve_ref as sr
from gemm_overlap_gemms_gb300 import attention_block as ab
from gemm_overlap_gemms_gb300 import synth, ub
from test_gpu_attention_block import D, HEADS, HIDDEN, KV_HEADS, PAGE, TP, close

pytestmark = pytest.mark.gpu

PAGES, WIDTH = 60, 8


@pytest.fixture(scope="module", params=[(0, 0), (20, 3)])
def block(request):
    from gemm_overlap_gemms_gb300 import _build
    _build.build()
    dev = torch.device("cuda")
    gen = synth.generator(dev)
    caches = [tuple(torch.full((PAGES, KV_HEADS, PAGE, D), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2))
              for _ in range(TP)]
    Wqkv = [synth.normal_bf16(((HEADS + 2 * KV_HEADS) * D, HIDDEN), HIDDEN ** -0.5, gen, dev) for _ in range(TP)]
    Wo = [synth.normal_bf16((HIDDEN, HEADS * D), (TP * HEADS * D) ** -0.5, gen, dev) for _ in range(TP)]
    cos, sin = ab.rotation_tables(256, D)
    window, sinks = request.param
    with ub.UserBuffer([256, HIDDEN], TP) as buf:
        yield ab.AttentionBlock(buf, Wqkv, Wo, HEADS, KV_HEADS, caches, cos, sin, window=window, sinks=sinks)


def dense(block, x):
    """One path [n, hidden] through the layer in 64 bits, nothing rounded."""
    n = x.shape[0]
    out = torch.zeros(n, HIDDEN, dtype=torch.float64, device=x.device)
    c, s = block.cos[:n].double()[:, None], block.sin[:n].double()[:, None]

    def turn(t):
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)
    pos = torch.arange(n, device=x.device)
    seen = sr.in_window(pos, pos, block.sight.get("window", 0), block.sight.get("sinks", 0))
    for Wqkv, Wo in zip(block.Wqkv, block.Wo):
        y = (x.double() @ Wqkv.double().T).view(n, HEADS + 2 * KV_HEADS, D)
        q, k, v = turn(y[:, :HEADS]), turn(y[:, HEADS:HEADS + KV_HEADS]), y[:, HEADS + KV_HEADS:]
        k, v = (t.repeat_interleave(HEADS // KV_HEADS, 1) for t in (k, v))
        z = (torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5).masked_fill(~seen, -torch.inf)
        out += torch.einsum("hij,jhd->ihd", z.softmax(-1), v).reshape(n, HEADS * D) @ Wo.double().T
    return out


def split(rows):
    return [t.contiguous() for t in rows.view(TP, rows.shape[0] // TP, HIDDEN)]


def test_prompts_drafts_and_forks(block):
    buf, dev = block.buf, torch.device("cuda")
    gen, rng = synth.generator(dev, seed=5), random.Random(1)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    table, refs = torch.full((6, WIDTH), -1, dtype=torch.int32, device=dev), torch.zeros(PAGES, dtype=torch.int32, device=dev)
    seqs = [synth.normal_bf16((n, HIDDEN), 1.0, gen, dev) for n in (37, 50)]
    buf.kv_take(refs, table[:2], ints([0, 0]), ints([37, 50]), PAGE)
    buf.set_active_shape([88, HIDDEN])  # a row of none's
    got = torch.cat(block.prompt(split(torch.cat(seqs + [torch.zeros_like(seqs[0][:1])])), ints([0, 37, 87]), ints([37, 50]), table[:2]))
    for a, x in ((0, seqs[0]), (37, seqs[1])):
        close(got[a:a + x.shape[0]], dense(block, x))
    # two candidates of the first, one of the second, in place of them
    source = [0, 1, 0]
    block.copy_pages(buf.kv_fork(refs, table[:2], ints([37, 50]), ints(source), table[2:5], PAGE))
    buf.kv_free(refs, table[:2], ints([0, 0]), ints([999, 999]), PAGE)
    seqs, rows = [seqs[i] for i in source], table[2:5]
    for step in range(4):
        new = [rng.randint(1, 9) for _ in seqs]
        pad = sum(new) % TP
        per = [sr.random_tree(n, rng) for n in new]
        text = [x.shape[0] for x in seqs]
        total, starts = ints([a + b for a, b in zip(text, new)]), ints([0, new[0], new[0] + new[1], sum(new)])
        parents = ints([p for t in per for p in t] + [0] * pad)
        buf.kv_take(refs, rows, ints(text), total, PAGE)
        drafts = [synth.normal_bf16((n, HIDDEN), 1.0, gen, dev) for n in new]
        buf.set_active_shape([sum(new) + pad, HIDDEN])
        got = torch.cat(block.draft(split(torch.cat(drafts + [torch.zeros(pad, HIDDEN, dtype=torch.bfloat16, device=dev)])), starts, total,
                                    rows, parents))
        at, leaves = 0, []
        for i, (tree, n) in enumerate(zip(per, new)):
            want = [dense(block, torch.cat((seqs[i], drafts[i][path])))[-1] for path in sr.paths(tree)]
            close(got[at:at + n], torch.stack(want))
            at += n
            leaves.append(rng.randint(-1, n - 1))
            if leaves[i] >= 0:
                seqs[i] = torch.cat((seqs[i], drafts[i][sr.paths(tree)[leaves[i]]]))
        lens = block.accept(starts, total, rows, parents, ints(leaves))
        assert lens.tolist() == [x.shape[0] for x in seqs]
        buf.kv_free(refs, rows, -(-lens // PAGE) * PAGE, ints([999] * 3), PAGE)
        moves, _ = buf.kv_compact(refs, table)
        block.copy_pages(moves)
        # a decoding step of all candidates
        x = synth.normal_bf16((4, HIDDEN), 1.0, gen, dev)
        buf.set_active_shape([4, HIDDEN])
        buf.kv_take(refs, rows, lens, lens + 1, PAGE)
        got = torch.cat(block.step(split(x), ints([0, 1, 2, 3]), lens + 1, rows))
        seqs = [torch.cat((s, x[i:i + 1])) for i, s in enumerate(seqs)]
        close(got[:3], torch.stack([dense(block, s)[-1] for s in seqs]))
        assert (got[3] == 0).all()
    torch.cuda.synchronize()
    assert buf.query_status() == ub.UB_OK


def test_drafts_on_another_stream(block):
    """draft and accept on a stream of their own give what they give on the current one."""
    buf, dev = block.buf, torch.device("cuda")
    gen = synth.generator(dev, seed=6)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    table = torch.arange(4, dtype=torch.int32, device=dev).view(1, 4)
    buf.set_active_shape([8, HIDDEN])
    shards = split(synth.normal_bf16((8, HIDDEN), 1.0, gen, dev))
    args = (ints([0, 8]), ints([8]), table, ints([-1, 0, 0, 1, 1, 2, 2, -1]))
    want = block.draft(shards, *args)
    lens = block.accept(*args, ints([6]))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = block.draft(shards, *args, stream=side)
    lens2 = block.accept(*args, ints([6]), stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and lens.tolist() == lens2.tolist() == [3]
    assert buf.query_status() == ub.UB_OK


def test_the_example_runs(capsys):
    ab.main()
    said = capsys.readouterr().out
    for what in ("prompts", "decoding step", "drafts", "accepted", "forks", "moved"):
        assert what in said
