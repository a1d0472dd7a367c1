"""Plain 64-bit definitions of the serving operators next to the attention: windows with sinks,
drafted trees, accepted drafts, and the sharing of pages. Shares no code with the library."""
import torch

import attn_ref as ref


def attend_seen(q, k, v, seen, scale):
    """q [n, heads, D] over k, v [kv heads, keys, D]: query i sees the keys of seen[i]. Returns
    (out, bound, lse, its bound) as attn_ref.attend, whose derivation of the bounds holds here too:
    the masked keys have the weight zero on both sides."""
    n, heads, dim = q.shape
    group = heads // k.shape[0]
    q, k, v = q.double(), k.double().repeat_interleave(group, 0), v.double().repeat_interleave(group, 0)
    if k.shape[1] == 0:
        z = torch.zeros(n, heads, dim, dtype=torch.float64, device=q.device)
        return z, z, torch.full((n, heads), -torch.inf, device=q.device, dtype=torch.float64), z[..., 0]
    s = (torch.einsum("nhd,hjd->hnj", q, k) * scale).masked_fill(~seen, -torch.inf)
    top = s.amax(-1, keepdim=True).clamp_min(-1e300)
    p = torch.exp(s - top)
    total = p.sum(-1)
    w = p / total.clamp_min(1e-300)[..., None]
    out = torch.einsum("hnj,hjd->nhd", w, v)
    mag = torch.einsum("hnj,hjd->nhd", w, v.abs())
    b = scale * torch.where(seen, torch.einsum("nhd,hjd->hnj", q.abs(), k.abs()), 0.0).amax(-1)
    shift = 2.0 ** -19 * (1 + b)
    lse = torch.where(total > 0, top[..., 0] + torch.log(total.clamp_min(1e-300)), -torch.inf)
    return out, mag * (2.1 * ref.U + 2 * shift.T[..., None]) + 1e-30, lse.T, shift.T


def in_window(pos, key, window, sinks):
    """[rows, keys]: which keys (their positions) rows at pos see of a causal window with sinks."""
    pos, key = pos[:, None], key[None, :]
    if window == 0:
        return key <= pos
    return (key <= pos) & ((key > pos - window) | (key < sinks))


def paths(parents):
    """The drafts from the text to each draft, itself included."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if p >= 0 else []) + [i])
    return out


def tree_seen(parents, total, window, sinks):
    """[drafts, total]: which cached places each draft sees; the last len(parents) are the drafts."""
    n = len(parents)
    text = total - n
    seen = torch.zeros(n, max(total, 0), dtype=torch.bool)
    up = paths(parents)
    pos = torch.tensor([text + len(path) - 1 for path in up])
    if text > 0:
        seen[:, :text] = in_window(pos, torch.arange(text), window, sinks)
    for i, path in enumerate(up):
        for d, a in enumerate(path):
            at = text + d  # position of ancestor a
            if text + a >= 0 and (window == 0 or at > pos[i] - window or at < sinks):
                seen[i, text + a] = True
    return seen


def random_tree(n, rng, kind="bushy"):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "flat":
        return [-1] * n
    return [rng.randint(-1, i - 1) for i in range(n)]


# ---------------------------------------------------------------- pages, on lists

def take(refs, table, begin, end, page):
    refs, table = list(refs), [list(r) for r in table]
    free = [p for p, r in enumerate(refs) if r <= 0]
    short = False
    for row, b, e in zip(table, begin, end):
        if e <= b:
            continue
        for j in range(max(b, 0) // page, min(-(-e // page), len(row))):
            if row[j] < 0:
                if free:
                    row[j] = free.pop(0)
                    refs[row[j]] = 1
                else:
                    short = True
    return refs, table, short


def give_up(refs, table, begin, end, page):
    refs, table = list(refs), [list(r) for r in table]
    for row, b, e in zip(table, begin, end):
        for j in range(len(row)):
            if row[j] >= 0 and j * page >= b and (j + 1) * page <= e:
                refs[row[j]] -= 1
                row[j] = -1
    return refs, table


def fork(refs, table, lens, source, page):
    refs = list(refs)
    free = [p for p, r in enumerate(refs) if r <= 0]
    rows, copies = [], []
    for s in source:
        whole = lens[s] // page
        row = [-1 if p < 0 else p for p in table[s][:whole]]
        for p in row:
            if p >= 0:
                refs[p] += 1
        pair = [-1, -1]
        if lens[s] % page and table[s][whole] >= 0:
            if free:
                pair = [table[s][whole], free.pop(0)]
                refs[pair[1]] = 1
            row.append(pair[1])
        rows.append(row + [-1] * (len(table[s]) - len(row)))
        copies.append(pair)
    return refs, rows, copies


def compact(refs, table):
    used = sum(r > 0 for r in refs)
    moves = list(zip([p for p, r in enumerate(refs) if r > 0 and p >= used],
                     [p for p, r in enumerate(refs) if r <= 0 and p < used]))
    refs, to = list(refs), dict(moves)
    for a, b in moves:
        refs[b], refs[a] = refs[a], 0
    return refs, [[to.get(p, p) for p in row] for row in table], [list(m) for m in moves], used
