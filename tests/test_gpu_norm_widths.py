"""norm_residual at the widest rows of each kernel: up to 2048 units of four elements the
backward keeps a row in registers (a ragged row of 8189 elements can lie on 2048, one of
8190 on 2049), up to 4096 the forward."""
import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp
from tests import test_gpu_norm_residual as norm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


@pytest.mark.parametrize("rows,n", [(310, 8189), (155, 8190), (9, 8187), (155, 4093), (160, 4094)])
@pytest.mark.parametrize("dt,st", [(BF, F32), (BF, BF), (F32, F32)])
def test_widest_rows_of_the_backward(rows, n, dt, st):
    norm.test_backward(rows, n, dt, st)


@pytest.mark.parametrize("rows,n", [(155, 16381), (310, 16382), (155, 8189), (2, 8189)])
@pytest.mark.parametrize("dt,st", [(BF, F32), (BF, BF), (F32, F32)])
def test_widest_rows_of_the_forward(rows, n, dt, st):
    norm.test_forward(rows, n, dt, st)
