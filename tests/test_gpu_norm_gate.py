"""The gate of fp32 tensors, closed far down: sigmoid(z) and its slope keep their
relative accuracy.  u = 2^-24 is half a spacing.  e = exp(-|z|) is off by 4 u (ex2: two
spacings) and 1.5 u of the product that makes up for its argument's rounding, 1 + e by
1 u more and its reciprocal by 2 u: e / (1 + e) by 10 u at most, e / (1 + e)^2 by 14 u."""
import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


@pytest.mark.parametrize("n", [64, 250, 1001, 4096, 20000])     # every kernel
def test_sigmoid_and_slope_of_fp32_gates(n):
    rows = 300
    g = torch.Generator("cuda").manual_seed(n)
    size = torch.exp(torch.rand(rows, n, generator=g, device="cuda") * 11.3 - 6.9).clamp(max=87.0)   # 1e-3 .. 82
    z = torch.where(torch.rand(rows, n, generator=g, device="cuda") < 0.7, -size, size)
    one = torch.ones(rows, n, device="cuda")
    h, _ = tsp.norm_residual_fwd(one, torch.zeros(rows, n, device="cuda"), gate=z)
    e = torch.exp(-z.double().abs())
    want = torch.where(z >= 0, 1.0, e) / (1 + e)
    assert bool(((h.double() - want).abs() <= 10 * U * want).all())
    out = tsp.norm_residual_bwd(one, None, one, None, gate=z)
    slope = e / (1 + e) ** 2
    assert bool(((out["dgate"].double() - slope).abs() <= 14 * U * slope).all())
    assert torch.equal(out["df"], h)
