"""AdamW with 8-bit states where its kernels differ from one call to the next: the
smallest eps, long runs of chunks without masters, calls that mix tensors with and
without masters."""
import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


@pytest.mark.parametrize("bits,eps", [(32, 1e-39), (32, 2.0 ** -126), (8, 2.0 ** -126), (8, 1e-30)])
def test_zero_gradients_over_the_smallest_eps(bits, eps):
    """0 / (0 + eps) is 0: the weights only decay.  One element of the last block has a
    gradient, and alone moves (by lr: m / root(v) is 1 at the first update)."""
    n = 3 * 128
    w = torch.full((n,), 2.0, device="cuda")
    g = torch.zeros(n, device="cuda")
    g[300] = 1e-3
    opt = tsp.AdamW([w], weight_decay=0.5, state_bits=bits, eps=eps)
    for k in range(2):
        opt.step([g], lr=0.25)                      # 1 - 0.25 * 0.5 = 0.875, exact
    assert opt.params[0].isfinite().all()
    still = torch.ones(n, dtype=torch.bool)
    still[300] = False
    assert torch.equal(w.cpu()[still], torch.full((n - 1,), 2.0 * 0.875 ** 2))
    # (a held root or m is off by at most 2^-4 of itself, for the second of the two moves of 0.25)
    want = (2.0 * 0.875 - 0.25) * 0.875 - 0.25
    assert abs(float(w[300]) - want) <= 0.25 * (3 * 2.0 ** -4 if bits == 8 else 2.0 ** -18)
