"""The page calls on arrays that share memory: refused where a call writes what it reads."""
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


def test_fork_refuses_counts_that_are_its_inputs(buf):
    refs, table, new = ints([1, 1, 1, 1] + [0] * 46), ints([[0, 1, -1], [2, 3, -1]]), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    lens, source = ints([20, 30]), ints([0, 1])
    before = refs.tolist()
    for args in ((refs[:2], source), (refs[48:], source), (lens, refs[:2]), (lens, refs[3:5])):
        with pytest.raises(ub.UbError, match="refs overlaps"):
            buf.kv_fork(refs, table, *args, new, 16)
    assert status(buf) == ub.UB_OK and refs.tolist() == before and not new.any()
