"""The page calls on arrays that share memory: refused where a call writes what it reads, and right on
rows that lie between one another."""
import random

import pytest
import torch

import serve_ref as sr
from gemm_overlap_gemms_gb300 import ub

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def buf():
    from gemm_overlap_gemms_gb300 import _build
    _build.build()
    with ub.UserBuffer([1024, 256], 1) as b:
        yield b


def status(buf):
    torch.cuda.synchronize()
    got = buf.query_status()
    buf.clear_status()
    return got


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_fork_refuses_counts_that_are_its_inputs(buf):
    refs, table, new = ints([1, 1, 1, 1] + [0] * 46), ints([[0, 1, -1], [2, 3, -1]]), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    lens, source = ints([20, 30]), ints([0, 1])
    before = refs.tolist()
    for args in ((refs[:2], source), (refs[48:], source), (lens, refs[:2]), (lens, refs[3:5])):
        with pytest.raises(ub.UbError, match="refs overlaps"):
            buf.kv_fork(refs, table, *args, new, 16)
    assert status(buf) == ub.UB_OK and refs.tolist() == before and not new.any()


@pytest.mark.parametrize("n,width", [(1, 5), (7, 20), (60, 33)])
def test_children_between_their_parents(buf, n, width):
    """One array of rows, the children's between the parents'; the rows of a compaction too."""
    rng = random.Random(n)
    page, pages = 16, 3 * n * width
    lens = [rng.randint(0, width * page) for _ in range(n)]
    at, table = 0, []
    for length in lens:
        need = -(-length // page)
        table.append(list(range(2 * at, 2 * (at + need), 2)) + [-1] * (width - need))
        at += need
    counts = [0] * pages
    for p in range(at):
        counts[2 * p] = 1
    source = [rng.randrange(n) for _ in range(n)]
    refs, rows = ints(counts), torch.full((2 * n, width), -7, dtype=torch.int32, device="cuda")
    rows[::2] = ints(table)
    copies = buf.kv_fork(refs, rows[::2], ints(lens), ints(source), rows[1::2], page)
    want = sr.fork(counts, table, lens, source, page)
    assert status(buf) == ub.UB_OK
    assert refs.tolist() == want[0] and rows[1::2].tolist() == want[1] and copies.tolist() == want[2] and rows[::2].tolist() == table
    # all rows of the pool move; those of the array's other half are where they are written
    double = torch.full((4 * n, width), -9, dtype=torch.int32, device="cuda")
    double[::2] = rows
    moved = sr.compact(want[0], rows.tolist())
    moves, used = buf.kv_compact(refs, double[::2], table_out=double[1::2])
    assert status(buf) == ub.UB_OK
    assert refs.tolist() == moved[0] and double[1::2].tolist() == moved[1] and used.tolist() == [moved[3]]
    assert moves.tolist()[:len(moved[2])] == moved[2] and torch.equal(double[::2], rows)
