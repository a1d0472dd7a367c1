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


def rows(at, n, pitch, width):
    return {at + r * pitch + i for r in range(n) for i in range(width)}


# Not for a machine with a GPU: a call that is not refused would go on with the made-up handle.
@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls are made with made-up addresses")
def test_rows_between_rows(lib, mem):
    """Children among their parents' rows, and any other way two tables may lie in one another: refused
    exactly where a word belongs to both."""
    base, seen = 1 << 41, {ARG: 0, CUDA: 0}
    apart = {"refs": mem.new(50), "lens": mem.new(9), "source": mem.new(9), "copies": mem.new(18)}
    for n, pitch, m, new_pitch, width in [(4, 20, 4, 20, 10), (4, 20, 3, 40, 10), (3, 40, 7, 20, 10), (2, 33, 5, 13, 10), (1, 5, 4, 25, 10),
                                          (4, 11, 1, 3, 10), (2, 10, 2, 10, 10), (8, 29, 9, 31, 3), (2, 90, 3, 14, 1)]:
        table = rows(0, n, pitch, width) if n > 1 else set(range(width))
        for at in range(-130, 130):
            both = table & (rows(at, m, new_pitch, width) if m > 1 else set(range(at, at + width)))
            rc = fork(lib, mem, **apart, table=base, new=base + 4 * at, rows=n, children=m, width=width, pitch=pitch, new_pitch=new_pitch)
            assert rc == (ARG if both else CUDA), (n, pitch, m, new_pitch, width, at)
            seen[rc] += 1
    assert min(seen.values()) > 500


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls are made with made-up addresses")
def test_arrays_beside_the_rows(lib, mem):
    """Counts, lengths and copies in the columns that a table leaves free."""
    base = 1 << 41
    apart = {"refs": mem.new(50), "table": base, "lens": mem.new(4), "source": mem.new(4), "new": mem.new(40), "copies": mem.new(8)}
    for name, words in (("refs", 50), ("lens", 4), ("source", 4), ("copies", 8)):
        for at in (-60, 10, 70, 74, 75, 79, 80, 230, 250):
            both = rows(0, 4, 80, 10) & set(range(at, at + words))
            rc = fork(lib, mem, **{**apart, name: base + 4 * at}, pitch=80)
            assert rc == (ARG if both and name in ("refs", "copies") else CUDA), (name, at)
