"""The attention operators between the QKV and the attention-out projections, as measured cases.

Three operators on packed tokens ``[T, heads, dim]`` of several sequences:

* append: rotate queries and keys by their positions, and write keys and values to a paged cache;
* prompt: causal attention of whole packed prompts, or of prompt chunks over a paged cache;
* decode: attention of one new token per sequence over a paged cache.

``run`` computes them with elementary torch operations, or, where ``own`` is true, through
``ub.UserBuffer``. Head counts are those of one tensor-parallel shard of the workloads in
``synth.py`` (hidden 4096 over 4 shards, 8192 over 8: eight query heads of 128), with all, a
quarter or one of them as key/value heads, or of an unsharded layer.
"""
import math
import random

import torch

own = False

MAX_TOKENS = 16384  # capacity of the registered user buffer (synth.WORKLOADS["stress"])
_buffer = None      # the one user buffer of this program


def listed():
    return [
        # The append of a decoding step: one token for each of four sequences.
        {"name": "append_step_4", "op": "append", "n": 4, "lo": 1, "hi": 1, "cap": 4, "log": False, "past": 900,
         "heads": 8, "kv_heads": 8, "dim": 128, "page": 16, "rot": 128, "pairs": False, "mix": 1},
        # The append of a packed microbatch of new prompts, lengths as in the QKV workload.
        {"name": "append_packed_8192", "op": "append", "n": 16, "lo": 128, "hi": 4096, "cap": 8192, "log": False, "past": 0,
         "heads": 8, "kv_heads": 8, "dim": 128, "page": 16, "rot": 128, "pairs": False, "mix": 67},
        # The largest microbatch, unsharded heads, half of each head rotated, in neighbouring pairs.
        {"name": "append_wide_16384", "op": "append", "n": 40, "lo": 200, "hi": 1000, "cap": 16384, "log": False, "past": 3000,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "rot": 64, "pairs": True, "mix": 3},
        # A few short prompts, one of a single token.
        {"name": "prompt_few_odd", "op": "prompt", "n": 3, "lo": 1, "hi": 150, "cap": 300, "log": True, "past": 0,
         "heads": 8, "kv_heads": 8, "dim": 128, "page": 0, "mix": 52},
        # The QKV workload's microbatch: packed sequences of 128 to 4096 tokens.
        {"name": "prompt_packed_8192", "op": "prompt", "n": 16, "lo": 128, "hi": 4096, "cap": 8192, "log": False, "past": 0,
         "heads": 8, "kv_heads": 8, "dim": 128, "page": 0, "mix": 118},
        # Many lengths, few long ones, one key/value head for eight query heads.
        {"name": "prompt_ragged_16384", "op": "prompt", "n": 60, "lo": 20, "hi": 8192, "cap": 16384, "log": True, "past": 0,
         "heads": 8, "kv_heads": 1, "dim": 128, "page": 0, "mix": 31},
        # One sequence that fills the buffer.
        {"name": "prompt_long_16384", "op": "prompt", "n": 1, "lo": 16384, "hi": 16384, "cap": 16384, "log": False, "past": 0,
         "heads": 8, "kv_heads": 2, "dim": 128, "page": 0, "mix": 7},
        # Chunks of prompts whose beginnings are cached already, heads of 64.
        {"name": "prompt_chunks_paged_64", "op": "prompt", "n": 9, "lo": 33, "hi": 1000, "cap": 4096, "log": True, "past": 8000,
         "heads": 16, "kv_heads": 4, "dim": 64, "page": 16, "mix": 8},
        # A decoding step of four short sequences.
        {"name": "decode_4_short", "op": "decode", "n": 4, "lo": 90, "hi": 600,
         "heads": 8, "kv_heads": 8, "dim": 128, "page": 16, "mix": 9},
        # A decoding step of an ordinary batch, lengths as in the QKV workload.
        {"name": "decode_64_ragged", "op": "decode", "n": 64, "lo": 128, "hi": 4096,
         "heads": 8, "kv_heads": 2, "dim": 128, "page": 16, "mix": 10},
        # One very long sequence with a single key/value head: only a split over its length fills the GPU.
        {"name": "decode_1_long", "op": "decode", "n": 1, "lo": 131071, "hi": 131071,
         "heads": 8, "kv_heads": 1, "dim": 128, "page": 64, "mix": 11},
        # The largest: 128 long sequences, unsharded heads.
        {"name": "decode_128_wide", "op": "decode", "n": 128, "lo": 1024, "hi": 8192,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 32, "mix": 12},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "prompt", "prompt", "decode", "decode"))
    kv_heads, group = rng.choice(((8, 1), (2, 4), (1, 8), (4, 2), (8, 4), (2, 3), (1, 12), (4, 4), (1, 1), (5, 1)))
    case = {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": rng.choice((64, 128, 128)),
            "mix": rng.randrange(1 << 20)}
    if op == "append":
        case["dim"] = rng.choice((64, 128))
        step = rng.random() < 0.4
        cap = _log_int(rng, 1, 256 if step else MAX_TOKENS)
        case.update(n=cap if step else rng.randint(1, 32), lo=1, hi=1 if step else max(1, cap // 2), cap=cap,
                    log=rng.random() < 0.5, past=_log_int(rng, 1, 4000), page=rng.choice((16, 32, 64, 128)),
                    rot=rng.choice((32, 64, case["dim"])), pairs=rng.random() < 0.5)
    elif op == "prompt":
        case["heads"], case["kv_heads"] = rng.choice(((8, 8), (8, 2), (8, 1), (6, 2), (12, 4), (5, 1), (16, 4)))
        cap = _log_int(rng, 30, 8192)
        n = rng.randint(1, 12)
        paged = rng.random() < 0.5
        case.update(n=n, lo=1, hi=max(1, min(cap, 2 * cap // n)), cap=cap, log=rng.random() < 0.5,
                    past=_log_int(rng, 1, 4096) if paged else 0, page=rng.choice((16, 32, 64, 128)) if paged else 0)
        if paged:  # the padded scores of the plain form stay within those of the listed cases
            case["cap"] = min(cap, 2048)
            case["hi"] = min(case["hi"], 1024)
    else:
        n = _log_int(rng, 1, 128)
        hi = _log_int(rng, 16, max(16, min(131072, (1 << 22) // (n * case["kv_heads"]))))
        case.update(n=n, lo=rng.randint(1, hi), hi=hi, page=rng.choice((16, 32, 64, 128)))
    return case


def _lengths(case):
    """(new tokens, tokens in the cache after them) of each sequence."""
    rng = random.Random(case["mix"])
    if case["op"] == "decode":
        kv = [rng.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
        return [1] * case["n"], kv
    new, total = [], 0
    for _ in range(case["n"]):
        length = (_log_int if case["log"] else random.Random.randint)(rng, case["lo"], case["hi"])
        if total + length > case["cap"]:
            break
        new.append(length)
        total += length
    new = new or [case["cap"]]
    return new, [length + (rng.randint(0, case["past"]) if case["past"] else 0) for length in new]


def work(case):
    new, kv = _lengths(case)
    tokens, heads, kv_heads, dim = sum(new), case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        rows = tokens * (heads + 2 * kv_heads) * dim * 2
        return {"bytes": 2 * rows + tokens * case["rot"] * 4, "flops": 3 * tokens * (heads + kv_heads) * case["rot"]}
    pairs = sum(n * (k - n) + n * (n + 1) // 2 for n, k in zip(new, kv))
    keys = sum(kv)
    return {"bytes": 2 * tokens * heads * dim * 2 + 2 * keys * kv_heads * dim * 2, "flops": 4 * dim * heads * pairs}


def prepare(case, seed):
    global _buffer
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    new, kv = _lengths(case)
    n, tokens = len(new), sum(new)
    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(0.0, std, generator=gen)

    # One row of the QKV projection's output per token: the three parts are views of it.
    qkv = normal(tokens, heads + 2 * kv_heads, dim)
    qkv[:, :heads] *= 2  # scores of some spread
    s = {"case": case, "tokens": tokens, "longest": (max(new), max(kv)),
         "q": qkv[:, :heads], "k": qkv[:, heads:heads + kv_heads], "v": qkv[:, heads + kv_heads:]}
    starts = [0]
    for length in new:
        starts.append(starts[-1] + length)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    if page:
        # Pages are handed out in no order; some stay free, and a row's unused entries are -1.
        need = [-(-length // page) for length in kv]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        table = torch.full((n, max(need)), -1, dtype=torch.int32, device=dev)
        at = torch.arange(max(need), device=dev)
        need = torch.tensor(need, device=dev)
        used = at[None, :] < need[:, None]
        table[used] = order[: int(used.sum())]
        s["table"] = table
        s["k_cache"] = normal(pages, kv_heads, page, dim)
        s["v_cache"] = normal(pages, kv_heads, page, dim)
    if case["op"] == "append":
        rot = case["rot"]
        angle = torch.arange(max(kv), device=dev, dtype=torch.float32)[:, None] * torch.exp(
            torch.arange(0, rot, 2, device=dev, dtype=torch.float32) * (-math.log(10000.0) / rot))[None, :]
        s["cos"], s["sin"] = angle.cos(), angle.sin()
    s["out"] = torch.zeros(tokens, heads, dim, dtype=torch.bfloat16, device=dev)
    if own:
        from gemm_overlap_gemms_gb300 import ub
        if _buffer is None:
            _buffer = ub.UserBuffer([MAX_TOKENS, 4096], 1)
        _buffer.set_active_shape([tokens, 4096])
    return s


def _token_places(s):
    """(sequence, position in the cache) of each packed token."""
    starts = s["starts"].long()
    t = torch.arange(s["tokens"], device=starts.device)
    seq = torch.searchsorted(starts[1:], t, right=True)
    return seq, s["kv_lens"].long()[seq] - starts[seq + 1] + t


def _rotate(x, cos, sin, pairs):
    rot = 2 * cos.shape[-1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_append(s):
    seq, pos = _token_places(s)
    page = s["case"]["page"]
    cos, sin = s["cos"][pos], s["sin"][pos]
    place, row = s["table"].long()[seq, pos // page], pos % page
    s["k_cache"][place, :, row] = _rotate(s["k"].float(), cos, sin, s["case"]["pairs"]).bfloat16()
    s["v_cache"][place, :, row] = s["v"]
    return {"q": _rotate(s["q"].float(), cos, sin, s["case"]["pairs"]).bfloat16(),
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(s, cache):
    """The cached rows of each sequence, [sequences, kv heads, longest, dim], in 32 bits."""
    rows = cache[s["table"].long().clamp_min(0)]
    return rows.permute(0, 2, 1, 3, 4).flatten(2, 3).float()


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
    seen = (seq[:, None] == seq[None, :]) & (pos[:, None] >= pos[None, :])
    o = _attend(q @ k.transpose(-1, -2) * c["dim"] ** -0.5, seen, v)
    return o.permute(2, 0, 1, 3).flatten(1, 2).bfloat16()


def _plain_prompt_paged(s):
    c = s["case"]
    seq, pos = _token_places(s)
    starts, lens = s["starts"].long(), s["kv_lens"].long()
    at = torch.arange(s["longest"][0], device=starts.device)
    take = (starts[:-1, None] + at).clamp_max(s["tokens"] - 1)
    group = c["heads"] // c["kv_heads"]
    q = s["q"].float()[take].unflatten(2, (c["kv_heads"], group)).permute(0, 2, 3, 1, 4)
    k, v = _gathered(s, s["k_cache"]), _gathered(s, s["v_cache"])
    key = torch.arange(k.shape[2], device=starts.device)
    last = (lens - (starts[1:] - starts[:-1]))[:, None] + at  # last position that a query sees
    seen = (key <= last[:, :, None]) & (key < lens[:, None, None])
    o = _attend(q @ k[:, :, None].transpose(-1, -2) * c["dim"] ** -0.5, seen[:, None, None], v[:, :, None])
    t = torch.arange(s["tokens"], device=starts.device)
    return o.permute(0, 3, 1, 2, 4)[seq, t - starts[seq]].flatten(1, 2).bfloat16()


def _plain_decode(s):
    c = s["case"]
    k, v = _gathered(s, s["k_cache"]), _gathered(s, s["v_cache"])
    q = s["q"].float().unflatten(1, (c["kv_heads"], c["heads"] // c["kv_heads"]))
    seen = torch.arange(k.shape[2], device=k.device) < s["kv_lens"][:, None]
    o = _attend(q @ k.transpose(-1, -2) * c["dim"] ** -0.5, seen[:, None, None], v)
    return o.flatten(1, 2).bfloat16()


def run(s):
    c = s["case"]
    if c["op"] == "append":
        if not own:
            return _plain_append(s)
        q = _buffer.kv_append(s["q"], s["k"], s["v"], s["cos"], s["sin"], s["starts"], s["kv_lens"], s["table"],
                              s["k_cache"], s["v_cache"], q_out=s["out"], interleaved=c["pairs"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["op"] == "prompt" and not c["page"]:
        return _buffer.attn_prompt(s["q"], s["k"], s["v"], s["starts"], out=s["out"]) if own else _plain_prompt_packed(s)
    if c["op"] == "prompt":
        if not own:
            return _plain_prompt_paged(s)
        return _buffer.attn_prompt_paged(s["q"], s["k_cache"], s["v_cache"], s["starts"], s["kv_lens"], s["table"],
                                         out=s["out"])
    if not own:
        return _plain_decode(s)
    return _buffer.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["kv_lens"], s["table"], out=s["out"])


def exact(case, seed):
    """The operators' definitions in 64 bits, sequence by sequence and head by head."""
    new, kv = _lengths(case)
    if 4 * case["dim"] * case["heads"] * sum(n * k for n, k in zip(new, kv)) > 4e12:
        return None
    s = prepare(case, seed)
    heads, kv_heads, page = case["heads"], case["kv_heads"], case["page"]
    if case["op"] == "append":
        half = case["rot"] // 2
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        flat = [c.double().transpose(1, 2).flatten(0, 1).clone() for c in (s["k_cache"], s["v_cache"])]
        cos, sin = s["cos"].double(), s["sin"].double()
        first = torch.arange(half, device=q.device) * (2 if case["pairs"] else 1)
        second = first + (1 if case["pairs"] else half)
        t = 0
        for i, (n, total) in enumerate(zip(new, kv)):
            at = torch.arange(total - n, total, device=q.device)
            z = torch.complex(cos[at], sin[at])[:, None, :]
            for x in (q, k):
                turned = torch.complex(x[t:t + n][..., first], x[t:t + n][..., second]) * z
                x[t:t + n, :, first], x[t:t + n, :, second] = turned.real, turned.imag
            where = s["table"][i].long()[at // page] * page + at % page
            flat[0][where], flat[1][where] = k[t:t + n], v[t:t + n]
            t += n
        caches = [f.unflatten(0, (-1, page)).transpose(1, 2) for f in flat]
        return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    t = 0
    for i, (n, total) in enumerate(zip(new, kv)):
        if page:
            at = s["table"][i, :-(-total // page)].long()
            k, v = (c[at].permute(1, 0, 2, 3).flatten(1, 2)[:, :total].double() for c in (s["k_cache"], s["v_cache"]))
        else:
            k, v = (x[t:t + n].permute(1, 0, 2).double() for x in (s["k"], s["v"]))
        for h in range(heads):
            kh, vh = k[h // (heads // kv_heads)], v[h // (heads // kv_heads)]
            for a in range(0, n, 4096):
                b = min(n, a + 4096)
                reach = total - n + b  # keys that the last of these queries sees
                z = s["q"][t + a:t + b, h].double() @ kh[:reach].T / math.sqrt(case["dim"])
                p = torch.softmax(z.masked_fill_(torch.ones_like(z, dtype=torch.bool).triu_(reach - (b - a) + 1), -math.inf), -1)
                out[t + a:t + b, h] = p @ vh[:reach]
        t += n
    return out
