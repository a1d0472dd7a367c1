"""Accepted drafts that test_gpu_tree.py does not draw: paths of many rows that all move, and one cache
for keys and values."""
import random

import pytest
import torch

import attn_ref as ref
import serve_ref as sr
from gemm_overlap_gemms_gb300 import ub

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def buf():
    from gemm_overlap_gemms_gb300 import _build
    _build.build()
    with ub.UserBuffer([16384, 256], 1) as b:
        yield b


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def moved(b, per, leaves, cache):
    """A cache with the rows of the accepted paths behind the text, and the new lengths."""
    want, lens = cache.clone(), []
    for s, (n, total) in enumerate(zip(b.new, b.kv)):
        path = sr.paths(per[s])[leaves[s]] if leaves[s] >= 0 else []
        lens.append(total - n + len(path))
        row = b.table[s].long()
        for d, a in enumerate(path):
            place, at = total - n + d, total - n + a
            want[row[place // b.page], :, place % b.page] = cache[row[at // b.page], :, at % b.page]
    return want, lens


@pytest.mark.parametrize("heads,dim,page", [(1, 64, 16), (2, 128, 8), (40, 128, 64)])
def test_one_cache_for_keys_and_values(buf, heads, dim, page):
    """Moved once, however many CTAs there are for a sequence's rows."""
    rng = random.Random(heads)
    b = ref.Batch([90, 33, 1, 300], [400, 33, 70, 1000], page=page, kv_heads=heads, dim=dim, seed=page)
    per = [[max(-1, i - 1 - rng.randint(0, 2)) for i in range(n)] for n in b.new]
    parents, leaves = ints([p for t in per for p in t]), [n - 1 for n in b.new]
    want, lens = moved(b, per, leaves, b.k_cache)
    got = buf.kv_accept(b.k_cache, b.k_cache, b.starts, b.lens, b.table, parents, ints(leaves))
    torch.cuda.synchronize()
    assert buf.query_status() == ub.UB_OK
    assert got.tolist() == lens and torch.equal(b.k_cache, want)


def test_two_views_of_one_cache_are_refused(buf):
    b = ref.Batch([5], [40], page=16, kv_heads=16, dim=64)
    before = b.k_cache.clone()
    with pytest.raises(ub.UbError, match="two views of one"):
        buf.kv_accept(b.k_cache, b.k_cache.transpose(1, 2), b.starts, b.lens, b.table, ints([-1, 0, 0, 1, 1]), ints([4]))
    torch.cuda.synchronize()
    assert buf.query_status() == ub.UB_OK and torch.equal(b.k_cache, before)
