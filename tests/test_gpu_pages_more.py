"""Page calls that the plain lists of test_gpu_pages.py do not draw: empty ranges, and rows of many
pages."""
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


@pytest.mark.parametrize("begin,end", [(-1, -1), (-5, -9), (40, 0), (40, 40), (99, 33), (-1, -20), (0, -3)])
def test_taking_nothing_records_nothing(buf, begin, end):
    """A range without rows lies nowhere: a sequence that takes no part may hold any such numbers."""
    refs, table = ints([0] * 6), ints([[-1, -1], [-1, -1], [-1, -1]])
    buf.kv_take(refs, table, ints([0, begin, 16]), ints([17, end, 32]), 16)
    assert status(buf) == ub.UB_OK
    assert table.tolist() == [[0, 1], [-1, -1], [-1, 2]] and refs.tolist() == [1, 1, 1, 0, 0, 0]


@pytest.mark.parametrize("begin,end,entries", [(-1, 0, [-1, -1]), (-1, 1, [0, -1]), (32, 33, [-1, -1]), (31, 33, [-1, 0])])
def test_taking_outside_the_table_is_recorded(buf, begin, end, entries):
    refs, table = ints([0] * 6), ints([[-1, -1]])
    buf.kv_take(refs, table, ints([begin]), ints([end]), 16)
    assert status(buf) == ub.CODES["UB_ERR_ARG"]
    assert table.tolist() == [entries]


def long_rows(n, width, page, seed):
    """Lists of a pool of `n` sequences that fill most of their rows, and its order of pages."""
    rng = random.Random(seed)
    lens = [rng.randint(width * page * 3 // 4, width * page) for _ in range(n)]
    need = [-(-length // page) for length in lens]
    order = list(range(2 * sum(need) + 64))
    rng.shuffle(order)
    refs, table, at = [0] * len(order), [], 0
    for k in need:
        table.append(order[at:at + k] + [-1] * (width - k))
        at += k
    for p in order[:at]:
        refs[p] = 1
    return rng, refs, table, lens


@pytest.mark.parametrize("n,width,page,children", [(1, 8192, 16, 1), (3, 8192, 16, 9), (16, 1024, 128, 64), (64, 2500, 16, 70)])
def test_long_rows(buf, n, width, page, children):
    """Sequences of up to 131072 tokens, whose rows are thousands of entries: given up and taken again, forked,
    moved together."""
    rng, refs, table, lens = long_rows(n, width, page, n)
    d_refs, d_table, cap = ints(refs), ints(table), width * page
    begin = [rng.randint(0, length) for length in lens]
    refs, table = sr.give_up(refs, table, begin, lens, page)
    buf.kv_free(d_refs, d_table, ints(begin), ints(lens), page)
    assert status(buf) == ub.UB_OK and d_refs.tolist() == refs and d_table.tolist() == table
    refs, table, short = sr.take(refs, table, [0] * n, lens, page)
    assert not short
    buf.kv_take(d_refs, d_table, ints([0] * n), ints(lens), page)
    assert status(buf) == ub.UB_OK and d_refs.tolist() == refs and d_table.tolist() == table
    source = [rng.randrange(n) for _ in range(children)]
    new = torch.zeros(children, width, dtype=torch.int32, device="cuda")
    copies = buf.kv_fork(d_refs, d_table, ints(lens), ints(source), new, page)
    refs, rows, pairs = sr.fork(refs, table, lens, source, page)
    assert status(buf) == ub.UB_OK and d_refs.tolist() == refs and new.tolist() == rows and copies.tolist() == pairs
    whole = torch.cat((d_table, new))
    moves, used = buf.kv_compact(d_refs, whole)
    refs, rows, pairs, count = sr.compact(refs, table + rows)
    assert status(buf) == ub.UB_OK and d_refs.tolist() == refs and whole.tolist() == rows and used.tolist() == [count]
    assert moves.tolist() == pairs + [[-1, -1]] * (len(refs) // 2 - len(pairs))
    buf.kv_free(d_refs, whole, ints([0] * (n + children)), ints([cap] * (n + children)), page)
    assert status(buf) == ub.UB_OK and not d_refs.any() and (whole == -1).all()
