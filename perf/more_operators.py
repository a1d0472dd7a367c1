"""Serving operators over the paged cache, as measured cases: windows, drafted tokens, pages.

Five operators next to the append and the attention of a layer:

* prompt, decode: attention with a sliding window and a few first tokens that stay visible (sinks),
  of packed prompts or chunks over the cache, and of one new token per sequence;
* tree: attention of drafted tokens, a tree of them for each sequence, over the cache that holds
  its text and the drafts;
* accept: the drafts of an accepted path move together behind the text, in place;
* pages: the cache's pages are shared out: rows of the table forked (whole pages shared by
  reference counts, the last one copied), dropped, and the pages in use moved together.

``run`` computes them with elementary torch operations, or, where ``own`` is true, through
``ub.UserBuffer``. Head counts are those of one tensor-parallel shard of the workloads in
``synth.py`` (eight query heads of 128), or of an unsharded layer.
"""
import math
import random

import torch

own = False

MAX_TOKENS = 16384  # capacity of the registered user buffer (synth.WORKLOADS["stress"])
_buffer = None      # the one user buffer of this program
_tokens = None      # ... and its active tokens


def listed():
    return [
        # The QKV workload's microbatch in a layer that sees 1024 tokens and the first four.
        {"name": "prompt_window_8192", "op": "prompt", "n": 16, "lo": 128, "hi": 4096, "cap": 8192, "log": False,
         "past": 0, "heads": 8, "kv_heads": 8, "dim": 128, "page": 0, "window": 1024, "sinks": 4, "mix": 118},
        # Chunks of prompts whose beginnings are cached already, heads of 64, odd window, no sinks.
        {"name": "prompt_window_chunks_64", "op": "prompt", "n": 9, "lo": 33, "hi": 1000, "cap": 4096, "log": True,
         "past": 8000, "heads": 16, "kv_heads": 4, "dim": 64, "page": 16, "window": 2000, "sinks": 0, "mix": 8},
        # A decoding step of four sequences, most of them longer than their window.
        {"name": "decode_window_4", "op": "decode", "n": 4, "lo": 90, "hi": 2000,
         "heads": 8, "kv_heads": 8, "dim": 128, "page": 16, "window": 512, "sinks": 1, "mix": 9},
        # The largest decoding step: 128 long sequences, unsharded heads.
        {"name": "decode_window_128", "op": "decode", "n": 128, "lo": 1024, "hi": 8192,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 32, "window": 2048, "sinks": 64, "mix": 12},
        # A few drafts for each of four short sequences.
        {"name": "tree_4_few", "op": "tree", "n": 4, "lo": 1, "hi": 12, "past_lo": 90, "past": 600, "bushy": True,
         "heads": 8, "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "sinks": 0, "mix": 21},
        # Ordinary verification of 16 sequences with up to 64 drafts, four query heads to a key head.
        {"name": "tree_16_ragged", "op": "tree", "n": 16, "lo": 24, "hi": 64, "past_lo": 500, "past": 8192, "bushy": True,
         "heads": 8, "kv_heads": 2, "dim": 128, "page": 32, "window": 0, "sinks": 0, "mix": 22},
        # The largest: 64 sequences, unsharded heads of 64.
        {"name": "tree_64_wide", "op": "tree", "n": 64, "lo": 5, "hi": 60, "past_lo": 1024, "past": 8192, "bushy": True,
         "heads": 32, "kv_heads": 8, "dim": 64, "page": 64, "window": 0, "sinks": 0, "mix": 23},
        # The accepted drafts of four sequences.
        {"name": "accept_4", "op": "accept", "n": 4, "lo": 1, "hi": 12, "past_lo": 90, "past": 600, "bushy": False,
         "kv_heads": 8, "dim": 128, "page": 16, "mix": 31},
        # The accepted drafts of a large batch, unsharded heads, long accepted paths.
        {"name": "accept_256_wide", "op": "accept", "n": 256, "lo": 16, "hi": 63, "past_lo": 1, "past": 500, "bushy": False,
         "kv_heads": 32, "dim": 128, "page": 64, "mix": 32},
        # Two prompts, eight candidates each.
        {"name": "pages_fork_2x8", "op": "pages", "what": "fork", "n": 2, "children": 16, "lo": 100, "hi": 700,
         "kv_heads": 8, "dim": 128, "page": 16, "spare": 40, "mix": 41},
        # The beams of a large batch, 128 rows of keys to a page.
        {"name": "pages_fork_64x8", "op": "pages", "what": "fork", "n": 64, "children": 512, "lo": 128, "hi": 4096,
         "kv_heads": 8, "dim": 128, "page": 128, "spare": 900, "mix": 42},
        # A pool that a load peak has left half empty is moved together.
        {"name": "pages_compact_24000", "op": "pages", "what": "compact", "n": 400, "lo": 64, "hi": 1000,
         "kv_heads": 2, "dim": 128, "page": 16, "spare": 12000, "mix": 43},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "decode", "decode", "tree", "tree", "tree", "accept", "pages", "pages"))
    kv_heads, group = rng.choice(((8, 1), (2, 4), (1, 8), (4, 2), (8, 4), (2, 3), (1, 12), (4, 4), (1, 1), (5, 1), (1, 7)))
    case = {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": rng.choice((64, 128, 128)),
            "page": rng.choice((16, 32, 64, 128)), "mix": rng.randrange(1 << 20)}
    window = {"window": _log_int(rng, 1, 6000), "sinks": rng.choice((0, 0, 1, 4, 4, 16, 100, 300))}
    if op == "prompt":
        case["heads"], case["kv_heads"] = rng.choice(((8, 8), (8, 2), (8, 1), (6, 2), (12, 4), (5, 1), (16, 4)))
        cap, n = _log_int(rng, 30, 8192), rng.randint(1, 12)
        paged = rng.random() < 0.5
        case.update(window, n=n, lo=1, hi=max(1, min(cap, 2 * cap // n)), cap=cap, log=rng.random() < 0.5,
                    past=_log_int(rng, 1, 4096) if paged else 0, page=case["page"] if paged else 0)
        if paged:  # the padded scores of the plain form stay within those of the listed cases
            case["cap"] = min(cap, 2048)
            case["hi"] = min(case["hi"], 1024)
    elif op == "decode":
        n = _log_int(rng, 1, 128)
        hi = _log_int(rng, 16, max(16, min(131072, (1 << 22) // (n * kv_heads))))
        case.update(window, n=n, lo=rng.randint(1, hi), hi=hi)
    elif op == "tree":
        n, hi = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        past = _log_int(rng, 16, max(16, min(131072, (1 << 22) // (n * kv_heads), (1 << 24) // (n * hi * kv_heads * group) * 8)))
        case.update(n=n, lo=rng.randint(1, hi), hi=hi, past_lo=rng.randint(0, past), past=past, bushy=rng.random() < 0.7,
                    window=0, sinks=0)
        if rng.random() < 0.25:
            case.update(window)
    elif op == "accept":
        n, hi = _log_int(rng, 1, 256), _log_int(rng, 1, 63)
        del case["heads"]
        case.update(n=n, lo=rng.randint(1, hi), hi=hi, past_lo=0, past=_log_int(rng, 1, 500), bushy=rng.random() < 0.5)
    else:
        what = rng.choice(("fork", "compact"))
        n = _log_int(rng, 1, 64 if what == "fork" else 400)
        hi = _log_int(rng, 1, 4096 if what == "fork" else 1000)
        del case["heads"]
        case.update(what=what, n=n, lo=rng.randint(1, hi), hi=hi, spare=_log_int(rng, 1, 4000))
        if what == "fork":
            case["children"] = n * rng.randint(1, 8)
            case["spare"] += case["children"]  # room for every copied page
    return case


def _lengths(case):
    """(new tokens, tokens in the cache after them) of each sequence."""
    rng = random.Random(case["mix"])
    if case["op"] in ("decode", "pages"):
        kv = [rng.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
        return [1] * case["n"], kv
    if case["op"] in ("tree", "accept"):
        new = [rng.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
        return new, [length + rng.randint(case["past_lo"], case["past"]) for length in new]
    new, total = [], 0
    for _ in range(case["n"]):
        length = (_log_int if case["log"] else random.Random.randint)(rng, case["lo"], case["hi"])
        if total + length > case["cap"]:
            break
        new.append(length)
        total += length
    new = new or [case["cap"]]
    return new, [length + (rng.randint(0, case["past"]) if case["past"] else 0) for length in new]


def _trees(case, new, seed):
    """Parent of each draft of each sequence (-1: the text itself), and an accepted draft (-1: none)."""
    rng = random.Random(case["mix"] * 7919 + seed)
    parents, leaves = [], []
    for n in new:
        if case["bushy"]:
            tree = [rng.randint(-1, i - 1) for i in range(n)]
        else:  # a few long branches
            tree = [i - 1 if rng.random() < 0.7 else rng.randint(-1, i - 1) for i in range(n)]
        parents.append(tree)
        leaves.append(rng.randint(-1, n - 1) if rng.random() < 0.3 else n - 1 - rng.randint(0, min(2, n - 1)))
    return parents, leaves


def _paths(tree):
    """The drafts of the path from the text to each draft."""
    paths = []
    for i, p in enumerate(tree):
        paths.append((paths[p] if p >= 0 else []) + [i])
    return paths


def _seen_keys(n, total, window, sinks):
    """Keys that the last n of `total` positions see: (of all rows together, rows counted one by one)."""
    if not window:
        return total, n * (total - n) + n * (n + 1) // 2
    pairs = 0
    for pos in range(total - n, total):
        near = min(window, pos + 1)
        pairs += near + min(sinks, pos + 1 - near)
    low = max(0, total - n - window + 1)
    return total - low + min(sinks, low), pairs


def work(case):
    new, kv = _lengths(case)
    kv_heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "accept":
        rows = 0
        for tree, leaf in zip(*_trees(case, new, 0)):
            path = _paths(tree)[leaf] if leaf >= 0 else []
            rows += sum(at != i for i, at in enumerate(path))
        return {"bytes": 2 * rows * 2 * kv_heads * dim * 2 + 4 * (sum(new) + 4 * len(new)), "flops": rows}
    if case["op"] == "pages":
        page_bytes = 2 * kv_heads * page * dim * 2
        need = [-(-length // page) for length in kv]
        pages = sum(need) + case["spare"]
        if case["what"] == "fork":
            source = _sources(case)
            copied = sum(kv[s] % page != 0 for s in source)
            entries = sum(need[s] for s in source)
            return {"bytes": 2 * copied * page_bytes + 4 * (2 * pages + 4 * entries), "flops": entries}
        moved = _moved(case)
        return {"bytes": 2 * moved * page_bytes + 4 * (2 * pages + 2 * sum(need)), "flops": pages}
    tokens, heads = sum(new), case["heads"]
    keys = pairs = 0
    if case["op"] == "tree":
        trees, _ = _trees(case, new, 0)
        for tree, n, total in zip(trees, new, kv):
            depth = [len(path) for path in _paths(tree)]
            keys += _seen_keys(n, total, case["window"], case["sinks"])[0]
            for d in depth:  # the text and the path
                pos = total - n + d - 1
                near = min(case["window"], pos + 1) if case["window"] else pos + 1
                pairs += near + min(case["sinks"], pos + 1 - near)
    else:
        for n, total in zip(new, kv):
            a, b = _seen_keys(n, total, case["window"], case["sinks"])
            keys, pairs = keys + a, pairs + b
    return {"bytes": 2 * tokens * heads * dim * 2 + 2 * keys * kv_heads * dim * 2, "flops": 4 * dim * heads * pairs}


def _sources(case):
    """The row of the table that each child comes from."""
    rng = random.Random(case["mix"] + 5)
    return [rng.randrange(case["n"]) for _ in range(case["children"])]


def _order(case, pages):
    """The pages in the order in which sequences got them; the rest are free."""
    order = list(range(pages))
    random.Random(case["mix"] + 6).shuffle(order)
    return order


def _moved(case):
    kv = _lengths(case)[1]
    used = sum(-(-length // case["page"]) for length in kv)
    return sum(p >= used for p in _order(case, used + case["spare"])[:used])


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    new, kv = _lengths(case)
    n, tokens = len(new), sum(new)
    kv_heads, dim, page = case["kv_heads"], case["dim"], case["page"]

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(0.0, std, generator=gen)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    s = {"case": case, "tokens": tokens, "longest": (max(new), max(kv))}
    starts = [0]
    for length in new:
        starts.append(starts[-1] + length)
    s["starts"], s["kv_lens"] = ints(starts), ints(kv)
    if case["op"] not in ("accept", "pages"):
        # One row of the QKV projection's output per token: the three parts are views of it.
        heads = case["heads"]
        qkv = normal(tokens, heads + 2 * kv_heads, dim)
        qkv[:, :heads] *= 2  # scores of some spread
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
        s["out"] = torch.zeros(tokens, heads, dim, dtype=torch.bfloat16, device=dev)
    if page:
        # Pages are handed out in no order; some stay free, and a row's unused entries are -1.
        need = [-(-length // page) for length in kv]
        pages = sum(need) + case.get("spare", 3)
        if case["op"] == "pages":  # the same ones for every seed, so that the work is
            order = ints(_order(case, pages))
        else:
            order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        rows = n + case.get("children", 0)
        table = torch.full((rows, max(need) + 1), -1, dtype=torch.int32, device=dev)
        used = torch.zeros_like(table, dtype=torch.bool)
        used[:n] = torch.arange(max(need) + 1, device=dev)[None, :] < torch.tensor(need, device=dev)[:, None]
        table[used] = order[: sum(need)]
        s["table"] = table
        s["k_cache"] = normal(pages, kv_heads, page, dim)
        s["v_cache"] = normal(pages, kv_heads, page, dim)
    if case["op"] in ("tree", "accept"):
        trees, leaves = _trees(case, new, seed if case["op"] == "tree" else 0)
        s["parents"] = ints([p for tree in trees for p in tree])
        s["leaves"] = ints(leaves)
        s["new_lens"] = torch.zeros_like(s["kv_lens"])
        # What a program without these operators keeps of a tree: which drafts are on whose path.
        widest = max(new)
        seen = torch.zeros(n, widest, widest, dtype=torch.bool)
        for i, tree in enumerate(trees):
            for j, path in enumerate(_paths(tree)):
                seen[i, j, path] = True
        s["seen"] = seen.to(dev)
    if case["op"] == "pages":
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device=dev)
        s["refs"][order[: sum(need)].long()] = 1
        if case["what"] == "fork":
            s["source"] = ints(_sources(case))
            s["zero"], s["end"] = ints([0] * case["children"]), ints([(max(need) + 1) * page] * case["children"])
            s["copies"] = torch.full((case["children"], 2), -1, dtype=torch.int32, device=dev)
        else:
            s["new_refs"], s["new_table"] = torch.zeros_like(s["refs"]), torch.zeros_like(table)
            s["moves"] = torch.full((pages // 2, 2), -1, dtype=torch.int32, device=dev)
            s["used"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------- plain forms

def _token_places(s):
    """(sequence, position in the cache) of each packed token."""
    starts = s["starts"].long()
    t = torch.arange(s["tokens"], device=starts.device)
    seq = torch.searchsorted(starts[1:], t, right=True)
    return seq, s["kv_lens"].long()[seq] - starts[seq + 1] + t


def _gathered(s, cache):
    """The cached rows of each sequence, [sequences, kv heads, longest, dim], in 32 bits."""
    rows = cache[s["table"].long().clamp_min(0)]
    return rows.permute(0, 2, 1, 3, 4).flatten(2, 3).float()


def _in_sight(c, pos, key):
    """Whether a row at `pos` looks as far as `key`, or at the first tokens."""
    if not c["window"]:
        return key <= pos
    return (key <= pos) & ((key > pos - c["window"]) | (key < c["sinks"]))


def _attend(scores, seen, v):
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(-3e38)
    weights = torch.exp(scores - top)
    return (weights @ v) / weights.sum(-1, keepdim=True).clamp_min(1e-38)


def _plain_prompt_packed(s):
    c = s["case"]
    seq, pos = _token_places(s)
    group = c["heads"] // c["kv_heads"]
    q = s["q"].float().unflatten(1, (c["kv_heads"], group)).permute(1, 2, 0, 3)  # [kv heads, group, T, dim]
    k = s["k"].float().permute(1, 0, 2)[:, None]
    v = s["v"].float().permute(1, 0, 2)[:, None]
    seen = (seq[:, None] == seq[None, :]) & _in_sight(c, pos[:, None], pos[None, :])
    o = _attend(q @ k.transpose(-1, -2) * c["dim"] ** -0.5, seen, v)
    return o.permute(2, 0, 1, 3).flatten(1, 2).bfloat16()


def _plain_over_cache(s, seen):
    """Rows of every sequence over its cache; seen [sequences, rows, keys]."""
    c = s["case"]
    seq, _ = _token_places(s)
    starts = s["starts"].long()
    at = torch.arange(s["longest"][0], device=starts.device)
    take = (starts[:-1, None] + at).clamp_max(s["tokens"] - 1)
    group = c["heads"] // c["kv_heads"]
    q = s["q"].float()[take].unflatten(2, (c["kv_heads"], group)).permute(0, 2, 3, 1, 4)
    k, v = _gathered(s, s["k_cache"]), _gathered(s, s["v_cache"])
    o = _attend(q @ k[:, :, None].transpose(-1, -2) * c["dim"] ** -0.5, seen[:, None, None], v[:, :, None])
    t = torch.arange(s["tokens"], device=starts.device)
    return o.permute(0, 3, 1, 2, 4)[seq, t - starts[seq]].flatten(1, 2).bfloat16()


def _plain_prompt_paged(s):
    starts, lens = s["starts"].long(), s["kv_lens"].long()
    at = torch.arange(s["longest"][0], device=starts.device)
    key = torch.arange(s["table"].shape[1] * s["case"]["page"], device=starts.device)
    pos = (lens - (starts[1:] - starts[:-1]))[:, None] + at  # position of each row
    return _plain_over_cache(s, _in_sight(s["case"], pos[:, :, None], key) & (key < lens[:, None, None]))


def _plain_tree(s):
    starts, lens = s["starts"].long(), s["kv_lens"].long()
    text = (lens - (starts[1:] - starts[:-1]))[:, None, None]  # keys of the text, of each sequence
    key = torch.arange(s["table"].shape[1] * s["case"]["page"], device=starts.device)[None, None, :]
    depth = s["seen"].sum(-1)
    pos = text + depth[:, :, None] - 1
    draft = (key - text).clamp(0, s["seen"].shape[2] - 1).expand(len(lens), s["seen"].shape[1], -1)
    is_draft = (key >= text) & (key < lens[:, None, None])
    key_depth = depth.gather(1, (key - text)[:, 0].clamp(0, depth.shape[1] - 1))[:, None, :]
    key_pos = torch.where(is_draft, text + key_depth - 1, key)
    on_path = (key < text) | (is_draft & s["seen"].gather(2, draft))
    return _plain_over_cache(s, on_path & _in_sight(s["case"], pos, key_pos))


def _plain_decode(s):
    c = s["case"]
    k, v = _gathered(s, s["k_cache"]), _gathered(s, s["v_cache"])
    q = s["q"].float().unflatten(1, (c["kv_heads"], c["heads"] // c["kv_heads"]))
    seen = _in_sight(c, s["kv_lens"][:, None] - 1, torch.arange(k.shape[2], device=k.device))
    o = _attend(q @ k.transpose(-1, -2) * c["dim"] ** -0.5, seen[:, None, None], v)
    return o.flatten(1, 2).bfloat16()


def _plain_accept(s):
    page = s["case"]["page"]
    starts, lens, leaves = s["starts"].long(), s["kv_lens"].long(), s["leaves"].long()
    text = lens - (starts[1:] - starts[:-1])
    rows = torch.arange(len(lens), device=starts.device)
    path = s["seen"][rows, leaves.clamp_min(0)] & (leaves >= 0)[:, None]  # [sequences, drafts]
    seq, draft = path.nonzero(as_tuple=True)
    source = text[seq] + draft
    target = text[seq] + path.cumsum(1)[seq, draft] - 1
    table = s["table"].long()
    for cache in (s["k_cache"], s["v_cache"]):
        cache[table[seq, target // page], :, target % page] = cache[table[seq, source // page], :, source % page]
    s["new_lens"].copy_(text + path.sum(1))
    return {"new_lens": s["new_lens"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_copy(s, pairs):
    pairs = pairs[pairs[:, 0] >= 0].long()
    for cache in (s["k_cache"], s["v_cache"]):
        cache[pairs[:, 1]] = cache[pairs[:, 0]]


def _plain_fork(s):
    page, n = s["case"]["page"], s["case"]["n"]
    refs, table = s["refs"], s["table"]
    dropped = table[n:][table[n:] >= 0].long()
    refs.index_add_(0, dropped, torch.full_like(dropped, -1, dtype=torch.int32))
    source = s["source"].long()
    lens = s["kv_lens"].long()[source]
    at = torch.arange(table.shape[1], device=table.device)
    child = torch.where(at < (lens // page)[:, None], table[source], -1)  # the whole pages, shared
    shared = child[child >= 0].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    part = lens % page != 0
    free = torch.argsort((refs > 0).to(torch.uint8), stable=True).to(torch.int32)  # free pages first, lowest first
    target = free[(part.cumsum(0) - 1).clamp_min(0)]
    copies = torch.where(part[:, None], torch.stack((table[source, lens // page], target), 1), -1)
    child = torch.where(part[:, None] & (at == (lens // page)[:, None]), target[:, None], child)
    refs[target[part].long()] = 1
    table[n:] = child
    _plain_copy(s, copies)
    return {"table": table, "refs": refs, "copies": copies, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    used = refs > 0
    count = used.sum()
    at = torch.arange(len(refs), device=refs.device)
    holes, movers = (~used) & (at < count), used & (at >= count)
    source, target = movers.nonzero()[:, 0], holes.nonzero()[:, 0]
    moves = torch.full_like(s["moves"], -1)
    moves[: len(source)] = torch.stack((source, target), 1).to(torch.int32)
    place = at.clone()
    place[source] = target
    new_table = torch.where(table >= 0, place[table.long().clamp_min(0)].to(torch.int32), -1)
    new_refs = torch.where(at < count, refs, 0)
    new_refs[target] = refs[source]
    _plain_copy(s, moves)
    return {"table": new_table, "refs": new_refs, "moves": moves, "used": count.to(torch.int32)[None],
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain(s):
    c = s["case"]
    if c["op"] == "prompt":
        return _plain_prompt_paged(s) if c["page"] else _plain_prompt_packed(s)
    if c["op"] == "pages":
        return _plain_fork(s) if c["what"] == "fork" else _plain_compact(s)
    return {"decode": _plain_decode, "tree": _plain_tree, "accept": _plain_accept}[c["op"]](s)


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    global _buffer, _tokens
    c = s["case"]
    if _buffer is None:
        from gemm_overlap_gemms_gb300 import ub
        _buffer = ub.UserBuffer([MAX_TOKENS, 4096], 1)
    buf = _buffer
    if c["op"] == "pages":
        if c["what"] == "fork":
            children = s["table"][c["n"]:]
            buf.kv_free(s["refs"], children, s["zero"], s["end"], c["page"])
            buf.kv_fork(s["refs"], s["table"][:c["n"]], s["kv_lens"], s["source"], children, c["page"], copies=s["copies"])
            buf.kv_copy(s["k_cache"], s["v_cache"], s["copies"])
            return {"table": s["table"], "refs": s["refs"], "copies": s["copies"], "k_cache": s["k_cache"],
                    "v_cache": s["v_cache"]}
        buf.kv_compact(s["refs"], s["table"], refs_out=s["new_refs"], table_out=s["new_table"], moves=s["moves"],
                       used=s["used"])
        buf.kv_copy(s["k_cache"], s["v_cache"], s["moves"])
        return {"table": s["new_table"], "refs": s["new_refs"], "moves": s["moves"], "used": s["used"],
                "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["op"] == "accept":
        buf.kv_accept(s["k_cache"], s["v_cache"], s["starts"], s["kv_lens"], s["table"], s["parents"], s["leaves"],
                      new_lens=s["new_lens"])
        return {"new_lens": s["new_lens"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if _tokens != s["tokens"]:
        _tokens = s["tokens"]
        buf.set_active_shape([_tokens, 4096])
    see = {"window": c["window"], "sinks": c["sinks"]}
    if c["op"] == "decode":
        return buf.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["kv_lens"], s["table"], out=s["out"], **see)
    if c["op"] == "tree":
        return buf.attn_tree(s["q"], s["k_cache"], s["v_cache"], s["starts"], s["kv_lens"], s["table"], s["parents"],
                             out=s["out"], **see)
    if c["page"]:
        return buf.attn_prompt_paged(s["q"], s["k_cache"], s["v_cache"], s["starts"], s["kv_lens"], s["table"],
                                     out=s["out"], **see)
    return buf.attn_prompt(s["q"], s["k"], s["v"], s["starts"], out=s["out"], **see)


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------- definitions in 64 bits

def _exact_pages(case, s):
    """Page by page, on the host."""
    n, page = case["n"], case["page"]
    table, refs, lens = s["table"].tolist(), s["refs"].tolist(), s["kv_lens"].tolist()
    pairs, out = [], {}
    if case["what"] == "fork":
        free = iter([p for p, r in enumerate(refs) if r == 0])
        for i, parent in enumerate(s["source"].tolist()):
            whole = lens[parent] // page
            row = table[parent][:whole]
            for p in row:
                refs[p] += 1
            pair = (-1, -1)
            if lens[parent] % page:
                pair = (table[parent][whole], next(free))
                refs[pair[1]] = 1
                row.append(pair[1])
            pairs.append(pair)
            table[n + i] = row + [-1] * (len(table[0]) - len(row))
        out["copies"] = torch.tensor(pairs, dtype=torch.int32)
    else:
        count = sum(r > 0 for r in refs)
        pairs = list(zip([p for p, r in enumerate(refs) if r > 0 and p >= count],
                         [p for p, r in enumerate(refs) if r == 0 and p < count]))
        where = dict(pairs)
        table = [[where.get(p, p) for p in row] for row in table]
        for a, b in pairs:
            refs[b], refs[a] = refs[a], 0
        out["moves"] = torch.tensor(pairs + [(-1, -1)] * (len(refs) // 2 - len(pairs)), dtype=torch.int32).view(-1, 2)
        out["used"] = torch.tensor([count], dtype=torch.int32)
    out["table"], out["refs"] = torch.tensor(table, dtype=torch.int32), torch.tensor(refs, dtype=torch.int32)
    pairs = torch.tensor([p for p in pairs if p[0] >= 0], device=s["k_cache"].device).view(-1, 2).long()
    for name in ("k_cache", "v_cache"):
        cache = s[name].clone()
        cache[pairs[:, 1]] = s[name][pairs[:, 0]]
        out[name] = cache.double()
    return out


def _exact_accept(s, new, kv, trees, leaves, page):
    out = {name: s[name].double() for name in ("k_cache", "v_cache")}
    lens = []
    for i, (tree, leaf, n, total) in enumerate(zip(trees, leaves, new, kv)):
        path = _paths(tree)[leaf] if leaf >= 0 else []
        lens.append(total - n + len(path))
        if not path:
            continue
        a = torch.tensor(path, device=s["table"].device) + total - n
        b = torch.arange(len(path), device=a.device) + total - n
        row = s["table"][i].long()
        for name in out:
            out[name][row[b // page], :, b % page] = s[name][row[a // page], :, a % page].double()
    return {"new_lens": torch.tensor(lens, dtype=torch.int32), **out}


def exact(case, seed):
    """The operators' definitions in 64 bits, sequence by sequence and head by head."""
    new, kv = _lengths(case)
    if case["op"] in ("accept", "pages"):
        s = prepare(case, seed)
        return _exact_pages(case, s) if case["op"] == "pages" else _exact_accept(s, new, kv, *_trees(case, new, 0), case["page"])
    if 4 * case["dim"] * case["heads"] * sum(n * k for n, k in zip(new, kv)) > 4e12:
        return None
    s = prepare(case, seed)
    heads, kv_heads, page = case["heads"], case["kv_heads"], case["page"]
    window = case["window"] or 1 << 40
    dev = s["q"].device
    trees = _trees(case, new, seed)[0] if case["op"] == "tree" else None
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    t = 0
    for i, (n, total) in enumerate(zip(new, kv)):
        if page:
            at = s["table"][i, :-(-total // page)].long()
            k, v = (c[at].permute(1, 0, 2, 3).flatten(1, 2)[:, :total].double() for c in (s["k_cache"], s["v_cache"]))
        else:
            k, v = (x[t:t + n].permute(1, 0, 2).double() for x in (s["k"], s["v"]))
        key = torch.arange(total, device=dev)
        pos, hidden = key[total - n:], torch.zeros(n, total, dtype=torch.bool, device=dev)
        if trees is not None:
            paths = _paths(trees[i])
            pos = torch.tensor([total - n + len(path) - 1 for path in paths], device=dev)
            key = torch.cat((key[:total - n], pos))
            hidden[:, total - n:] = True
            for j, path in enumerate(paths):
                hidden[j, torch.tensor(path, device=dev) + total - n] = False
        hidden |= key[None, :] > pos[:, None]
        hidden |= (key[None, :] <= pos[:, None] - window) & (key[None, :] >= case["sinks"])
        for h in range(heads):
            kh, vh = k[h // (heads // kv_heads)], v[h // (heads // kv_heads)]
            z = s["q"][t:t + n, h].double() @ kh.T / math.sqrt(case["dim"])
            out[t:t + n, h] = torch.softmax(z.masked_fill_(hidden, -math.inf), -1) @ vh
        t += n
    return out
