"""Page calls that the plain lists of test_gpu_pages.py do not draw: empty ranges, and rows of many
pages."""
import pytest
import torch

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
