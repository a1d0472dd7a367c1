"""Trees of drafts whose paths are long and skip drafts on their way: what neither chains (a path is every
draft) nor random trees (a path is short) have."""
import random

KINDS = ("two", "three", "late", "half", "comb", "near", "far")


def deep_tree(kind, n, seed=0):
    rng = random.Random(seed * 7919 + n)
    if kind == "two":    # two chains, draft by draft in turn
        return [max(-1, i - 2) for i in range(n)]
    if kind == "three":
        return [max(-1, i - 3) for i in range(n)]
    if kind == "late":   # some drafts of the text, then a chain
        return [i - 1 if i > 5 else -1 for i in range(n)]
    if kind == "half":   # the same, half of them: whole words and tiles of drafts are skipped
        return [i - 1 if i > n // 2 else -1 for i in range(n)]
    if kind == "comb":   # a chain with a leaf on each of its drafts
        return [i - 1 if i % 2 else i - 2 + (i == 0) for i in range(n)]
    if kind == "near":   # a draft follows one of the last few
        return [max(-1, i - rng.randint(1, 5)) for i in range(n)]
    # a word or a tile back at a time, from a chain
    return [i - 1 if i < 8 or rng.random() < 0.5 else max(-1, i - rng.choice((31, 32, 33, 127, 128, 129))) for i in range(n)]
