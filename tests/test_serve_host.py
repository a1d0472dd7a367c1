"""Host side of the serving operators that needs no GPU: argument structs, refusals of nulls, and
the tests' own definitions on small cases."""
import ctypes
import os
import random
import re

import pytest
import torch

import serve_ref as sr
from gemm_overlap_gemms_gb300 import _build, ub

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ub.h")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ub.load()


def test_packed_pool_matches_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = [b for b in re.findall(r"typedef struct \{([^}]*)\} (\w+);", text) if b[1] == "ub_pool_t"][0][0]
    sizes = {"uint32_t": "I", "int32_t": "i", "int64_t": "q"}
    fmt = "".join("Q" if "*" in line else sizes[line.split()[0]] for line in body.split(";") if line.strip())
    spelled = "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([a-zA-Z])", ub._POOL.format.lstrip("=")))
    assert fmt == spelled and ctypes.sizeof(ctypes.c_void_p) == 8
    assert int(re.search(r"#define UB_ACCEPT_MOST (\d+)", open(HEADER).read()).group(1)) == ub.ACCEPT_MOST


NONE = {"ub_attn_prompt_window": [1, 0], "ub_attn_decode_window": [1, 0], "ub_kv_append_tree": [None], "ub_attn_tree": [None, 0, 0],
        "ub_kv_accept": [None, 0, None, None], "ub_kv_copy": [None, 0], "ub_kv_take": [None, None], "ub_kv_free": [None, None],
        "ub_kv_fork": [None, None, 0, None, 0, None], "ub_kv_compact": [None, None, 0, None, 0, None]}


@pytest.mark.parametrize("name", sorted(NONE))
def test_null_handles_are_refused(lib, name):
    size = ub._POOL.size if name in ("ub_kv_take", "ub_kv_free", "ub_kv_fork", "ub_kv_compact") else ub._ATTN.size
    for args in (None, bytes(size)):
        assert getattr(lib, name)(None, args, *NONE[name], None) == ub.CODES["UB_ERR_ARG"]


@pytest.mark.parametrize("window,sinks", [(-1, 0), (3, -1), (None, 0), (1 << 31, 0), (4, 1 << 31)])
def test_refused_windows(window, sinks):
    with pytest.raises(ValueError):
        ub._sight(window, sinks)
    assert not ub._sight(0, 5) and ub._sight(1, 0)


def test_definition_of_windows():
    key = torch.arange(8)
    seen = sr.in_window(torch.tensor([0, 2, 7]), key, 3, 2)
    assert seen.int().tolist() == [[1, 0, 0, 0, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 1, 1, 1]]
    assert sr.in_window(torch.tensor([4]), key, 0, 0).int().tolist() == [[1, 1, 1, 1, 1, 0, 0, 0]]


def test_definition_of_trees():
    parents = [-1, 0, 0, 2, -1]
    assert sr.paths(parents) == [[0], [0, 1], [0, 2], [0, 2, 3], [4]]
    seen = sr.tree_seen(parents, 7, 0, 0).int().tolist()
    assert seen == [[1, 1, 1, 0, 0, 0, 0], [1, 1, 1, 1, 0, 0, 0], [1, 1, 1, 0, 1, 0, 0], [1, 1, 1, 0, 1, 1, 0], [1, 1, 0, 0, 0, 0, 1]]
    assert sr.tree_seen(parents, 7, 2, 1).int().tolist() == [[1, 1, 1, 0, 0, 0, 0], [1, 0, 1, 1, 0, 0, 0], [1, 0, 1, 0, 1, 0, 0],
                                                               [1, 0, 0, 0, 1, 1, 0], [1, 1, 0, 0, 0, 0, 1]]
    chain = sr.random_tree(6, random.Random(0), "chain")
    pos = torch.arange(4, 10)
    assert torch.equal(sr.tree_seen(chain, 10, 3, 1), sr.in_window(pos, torch.arange(10), 3, 1))


def test_definition_of_pages():
    refs, table, short = sr.take([1, 0, 0, 1], [[0, -1, -1], [3, -1, -1]], [0, 16], [20, 17], 16)
    assert (refs, table, short) == ([1, 1, 1, 1], [[0, 1, -1], [3, 2, -1]], False)
    new, rows, copies = sr.fork([1, 1, 0, 0, 0], [[0, 1]], [20], [0, 0], 16)
    assert (new, rows, copies) == ([3, 1, 1, 1, 0], [[0, 2], [0, 3]], [[1, 2], [1, 3]])
    assert sr.give_up(new, rows, [0, 0], [32, 31], 16) == ([1, 1, 0, 1, 0], [[-1, -1], [-1, 3]])
    assert sr.compact([0, 2, 0, 1, 1], [[1, 4], [1, 3]]) == ([1, 2, 1, 0, 0], [[1, 2], [1, 0]], [[3, 0], [4, 2]], 3)
