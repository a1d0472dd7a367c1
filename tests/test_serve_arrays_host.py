"""Which arrays a page call may be given together: what it writes overlaps nothing that it reads or
else writes. The library refuses before it looks at the handle, so these calls need no GPU."""
import ctypes

import pytest
import torch

from gemm_overlap_gemms_gb300 import _build, ub

ARG, CUDA = ub.CODES["UB_ERR_ARG"], ub.CODES["UB_ERR_CUDA"]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ub.load()


class Memory:
    """Made-up device addresses of int32 arrays, and a handle that no refused call looks at (one that
    is not refused finds device 0 there, and no driver)."""

    def __init__(self):
        self.handle = ctypes.create_string_buffer(1 << 16)
        self.next = 1 << 40

    def new(self, words):
        at, self.next = self.next, self.next + 4 * words + 256
        return at

    def pool(self, refs, pages, table, rows, width, pitch=None):
        return ub._POOL.pack(ub._POOL.size, rows, 16, 0, pages, width, pitch or width, refs, table)


@pytest.fixture
def mem():
    return Memory()


def fork(lib, mem, refs, table, lens, source, new, copies, children=4, rows=4, width=10, pages=50, pitch=None, new_pitch=None):
    pool = mem.pool(refs, pages, table, rows, width, pitch)
    return lib.ub_kv_fork(mem.handle, pool, lens, source, children, new, new_pitch or width, copies, None)


@pytest.mark.parametrize("which", ["lens", "source"])
@pytest.mark.parametrize("at", [0, 46, 49, -3])
def test_fork_refuses_counts_that_are_its_inputs(lib, mem, which, at):
    """The counts change while the lengths and sources are read."""
    arrays = {"refs": mem.new(50), "table": mem.new(40), "lens": mem.new(4), "source": mem.new(4), "new": mem.new(40), "copies": mem.new(8)}
    arrays[which] = arrays["refs"] + 4 * at
    assert fork(lib, mem, **arrays) == ARG
    assert b"refs overlaps" in lib.ub_last_error()
