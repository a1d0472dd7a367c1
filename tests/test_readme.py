"""The serving recipe of the readme, run as it is written on two layers: every layer's cache has to
hold the accepted path, the tables and counts what they should."""
import os
import random
import re

import pytest
import torch

import attn_ref as ref
import serve_ref as sr

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def recipe():
    return [b for b in re.findall(r"```python\n(.*?)```", open(README).read(), flags=re.S) if "kv_accept" in b][0]


class Recorder:
    """Stands for the user buffer: keeps what each call was given."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args, **kw):
            self.calls.append((name, args))
            return ("pairs", "used") if name == "kv_compact" else name + " result"
        return call


def test_every_layer_accepts_from_the_same_lengths():
    """As many layers as there are caches: each accepts the lengths that the attention had, the pages are
    given up and forked by the accepted ones."""
    buf = Recorder()
    names = ("refs table zero lens page_size q k v cos sin starts parents leaves capacity source new_table rows k_cache v_cache").split()
    exec(recipe(), {**{n: n for n in names}, "buf": buf, "caches": [("k0", "v0"), ("k1", "v1")]})
    accepted = [args for name, args in buf.calls if name == "kv_accept"]
    assert [args[:2] for args in accepted] == [("k0", "v0"), ("k1", "v1")]
    assert all(args[2:] == ("starts", "lens", "table", "parents", "leaves") for args in accepted)
    later = {name: args for name, args in buf.calls if name in ("kv_free", "kv_fork")}
    assert later["kv_free"][2] == later["kv_fork"][2] == "kv_accept result"


@pytest.mark.gpu
def test_the_recipe():
    from gemm_overlap_gemms_gb300 import _build, ub
    _build.build()
    rng, gen = random.Random(2), torch.Generator(device="cuda").manual_seed(2)
    page, width, heads, G, D, text, new = 16, 12, 4, 2, 64, [70, 33, 5], [9, 4, 14]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()
    per = [[max(-1, i - 1 - rng.randint(0, 2)) for i in range(n)] for n in new]
    leaves = [8, -1, 12]
    paths = [sr.paths(t)[leaf] if leaf >= 0 else [] for t, leaf in zip(per, leaves)]
    starts, total = [0, 9, 13, 27], [a + b for a, b in zip(text, new)]
    angle = torch.rand(120, D // 2, generator=gen, device="cuda") * 6
    refs, rows = torch.zeros(60, dtype=torch.int32, device="cuda"), torch.full((7, width), -1, dtype=torch.int32, device="cuda")
    caches = [(randn(60, G, page, D), randn(60, G, page, D)) for _ in range(2)]
    with ub.UserBuffer([1024, 256], 1) as buf:
        buf.set_active_shape([27, 256])
        own = {"buf": buf, "refs": refs, "table": rows[:3], "rows": rows, "new_table": rows[3:], "zero": ints([0] * 3), "lens": ints(total),
               "page_size": page, "caches": caches, "q": randn(27, heads, D), "k": randn(27, G, D), "v": randn(27, G, D),
               "cos": angle.cos(), "sin": angle.sin(), "starts": ints(starts), "parents": ints([p for t in per for p in t]),
               "leaves": ints(leaves), "capacity": ints([width * page] * 3), "source": ints([0, 2, 2, 1])}
        # the text of each layer, on the pages that the recipe's first call goes on with
        buf.kv_take(refs, own["table"], own["zero"], ints(text), page)
        place = rows[:3].long()
        kept_text = [[tuple(c[place[s][torch.arange(text[s], device="cuda") // page], :, torch.arange(text[s], device="cuda") % page].clone()
                            for c in pair) for s in range(3)] for pair in caches]
        exec(recipe(), own)
        torch.cuda.synchronize()
        assert buf.query_status() == ub.UB_OK
    assert own["kept"].tolist() == [t + len(p) for t, p in zip(text, paths)]
    table = rows.tolist()
    for layer, (k_cache, v_cache) in enumerate(caches):
        for row, s in [(0, 0), (1, 1), (2, 2), (3, 0), (4, 2), (5, 2), (6, 1)]:  # the sequences and their children
            n = text[s] + len(paths[s])
            assert all(p >= 0 for p in table[row][:-(-n // page)]) and all(p < 0 for p in table[row][-(-n // page):])
            at, pos = rows[row].long(), torch.arange(n, device="cuda")
            k, v = (c[at[pos // page], :, pos % page] for c in (k_cache, v_cache))
            drafts = torch.tensor(paths[s], dtype=torch.long, device="cuda") + starts[s]
            assert torch.equal(k[:text[s]], kept_text[layer][s][0]) and torch.equal(v[:text[s]], kept_text[layer][s][1])
            assert torch.equal(v[text[s]:], own["v"][drafts])
            turn = text[s] + torch.arange(len(paths[s]), device="cuda")
            want, e = ref.rotate(own["k"][drafts], own["cos"][turn], own["sin"][turn], False)
            ref.within(k[text[s]:], want, e, "layer %d, row %d" % (layer, row))
    named = rows[rows >= 0].long()
    count = torch.zeros_like(refs).index_add_(0, named, torch.ones_like(named, dtype=torch.int32))
    assert torch.equal(count, refs) and own["used"].item() == int((refs > 0).sum())
    assert (refs[own["used"].item():] == 0).all()
