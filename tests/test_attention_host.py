"""Host side of the attention operators that needs no GPU: the packed argument struct is
the header's, null handles and arguments are refused, and the test's own definitions hold
on small cases."""
import ctypes
import os
import re

import pytest
import torch

import attn_ref as ref
from gemm_overlap_gemms_gb300 import _build, ub

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ub.h")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ub.load()


def test_packed_arguments_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} ub_attn_t;", text).group(1)
    sizes = {"uint32_t": "I", "int32_t": "i", "float": "f", "int64_t": "q", "ub_heads_t": "Q2q", "ub_pages_t": "Q3q"}
    fmt = ""
    for line in body.split(";"):
        words = line.replace("const", "").split(None, 1)
        if len(words) != 2:
            continue
        for field in words[1].split(","):
            fmt += "Q" if "*" in field else sizes[words[0]]
    assert ctypes.sizeof(ctypes.c_void_p) == 8

    def spelled(f):
        return "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([a-zA-Z])", f))
    assert spelled(fmt) == spelled(ub._ATTN.format.lstrip("="))


@pytest.mark.parametrize("name", ["ub_kv_append", "ub_attn_prompt", "ub_attn_decode"])
def test_null_handle_is_rejected(lib, name):
    assert getattr(lib, name)(None, None, None) == ub.CODES["UB_ERR_ARG"]
    assert getattr(lib, name)(None, bytes(ub._ATTN.size), None) == ub.CODES["UB_ERR_ARG"]


def test_definition_of_attention():
    """One key: its value; equal scores: the mean; the causal limit; no key: zero."""
    q = torch.zeros(3, 2, 4)
    k, v = torch.randn(1, 3, 4), torch.randn(1, 3, 4)
    out, bound, lse, _ = ref.attend(q, k, v, torch.tensor([0, 1, -1]), 0.5)
    v = v.double()
    assert torch.allclose(out[0], v[0, :1].expand(2, 4))
    assert torch.allclose(out[1], v[0, :2].mean(0).expand(2, 4))
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()
    assert torch.allclose(lse[1].exp(), torch.full((2,), 2.0).double())
    assert (bound >= 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_definition_of_rotation(interleaved):
    """A rotation keeps pair lengths, rotates (1, 0) to (cos, sin), and leaves the rest."""
    a = torch.tensor([[0.3, 1.1]])
    x = torch.zeros(1, 1, 6)
    ia, ib = ([0, 2], [1, 3]) if interleaved else ([0, 1], [2, 3])
    x[0, 0, ia] = 1.0
    x[0, 0, 4:] = 7.0
    y, _ = ref.rotate(x, a.cos(), a.sin(), interleaved)
    assert torch.allclose(y[0, 0, ia].float(), a.cos()[0]) and torch.allclose(y[0, 0, ib].float(), a.sin()[0])
    assert (y[0, 0, 4:] == 7).all()


def test_bounds_catch_a_planted_mistake():
    q, k, v = torch.randn(4, 2, 64), torch.randn(1, 50, 64), torch.randn(1, 50, 64)
    last = torch.tensor([46, 47, 48, 49])
    out, bound, _, _ = ref.attend(q, k, v, last, 0.125)
    ref.within(out.bfloat16(), out, bound, "rounded")
    wrong, _, _, _ = ref.attend(q, k, v, last - 1, 0.125)
    with pytest.raises(AssertionError):
        ref.within(wrong.bfloat16(), out, bound, "one key missing")
