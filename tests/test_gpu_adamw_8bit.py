"""AdamW with 8-bit states where its kernels differ from one call to the next: the
smallest eps, long runs of chunks without masters, calls that mix tensors with and
without masters."""
import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp
from tests.test_gpu_adamw import B1, B2, EPS, U, UBF, dequantise, quantise, reference

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


@pytest.mark.parametrize("masters", ["none", "all but every other", "every other"])
def test_long_runs_with_and_without_masters(masters):
    """bf16 tensors large enough that a CTA takes 8 chunks in a row (4 where the first
    tensor has a master), ragged and empty ones between; tensors with a master next to
    ones without, whose weights come in 16 and in 8 bytes a lane.  On the GPU against
    elementary operations there."""
    total = 62_000_000
    sizes = [total // 2 + 77, 0, 5, 4096 * 3 + 1, 8192 + 512, 640, total // 4 + 2, 129, 4096, 8192, 3 * 4096,
             total // 4]
    gen = torch.Generator("cuda").manual_seed(7)
    r = lambda n: torch.randn(n, generator=gen, device="cuda")   # noqa: E731
    params = [(0.02 * r(n)).to(BF) for n in sizes]
    has = [masters != "none" and i % 2 == (masters == "every other") for i in range(len(sizes))]
    given = [p.float() if on else None for p, on in zip(params, has)]
    prep = [torch.zeros(n, dtype=torch.float16, device="cuda") if i % 3 else None for i, n in enumerate(sizes)]
    opt = tsp.AdamW(params, weight_decay=0.1, state_bits=8, master=given, prep=prep, betas=(B1, B2), eps=EPS)
    state = [p.float() for p in params]
    ref = [(torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")) for n in sizes]
    for k in (1, 2):
        grads = [r(n) * 1e-3 for n in sizes]
        opt.step(grads, lr=1e-3)
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            m, root = ref[i]
            w, m, v, root = reference(state[i], m, root * root, grads[i], 1e-3, 0.1, k)
            got = opt.master[i] if has[i] else opt.params[i].float()
            # quotients 4 u apart (rcp 2, product 1, division 1) of an update of at most 1e-3 *
            # sqrt(1 / 0.05): 4 u of that; numbers that far apart round to weights at most a
            # spacing further apart, 2 u of the larger (u of bf16 for a bf16 weight)
            u = U if has[i] else UBF
            big = torch.maximum(w.abs(), got.abs())
            want = w if has[i] else w.to(BF).float()
            assert bool(((got - want).abs() <= 2 * u * big + 4 * U * 5e-3).all()), (i, k)
            # all but the few that a rounding border separates are the same weight
            assert has[i] or float((got != want).float().mean()) <= 1e-3 + 1 / n
            assert torch.equal(opt.params[i], got.to(BF))
            assert prep[i] is None or torch.equal(prep[i], opt.params[i].half())
            state[i] = got.clone()
            qm, sm = quantise(m, False)
            qr, sr = quantise(root, True)
            assert torch.equal(opt.m_scale[i], sm) and torch.equal(opt.v_scale[i], sr), (i, k)
            assert torch.equal(opt.m[i].view(torch.uint8), qm.view(torch.uint8)), (i, k)
            assert torch.equal(opt.v[i].view(torch.uint8), qr.view(torch.uint8)), (i, k)
            ref[i] = dequantise(qm, sm), dequantise(qr, sr)
    assert tsp.device_status() == tsp.TSP_OK


@pytest.mark.parametrize("beta2", [0.9, B2, 0.97])
def test_held_roots_follow_their_gradients(beta2):
    """After 300 updates the gradients of every other element fall by 100, for which v
    itself needs ln(10^4) / ln(1 / beta2) updates, 302 at 0.97.  Four times that later the
    held roots are on average within half an e4m3 step, 2^-4, of the 32-bit ones, which is
    what a rounding that is not held on to leaves; so are the squares of the updates,
    whose factor is the root (twice that)."""
    n = 128 * 500
    gen = torch.Generator("cuda").manual_seed(1)
    size = torch.exp(torch.randn(n, device="cuda", generator=gen)) * 1e-3
    half = torch.arange(n, device="cuda") % 2 == 0
    opt = {b: tsp.AdamW([torch.zeros(n, device="cuda")], state_bits=b, betas=(B1, beta2)) for b in (8, 32)}
    for k in range(1500):
        if k == 300:
            size = torch.where(half, size * 0.01, size)
        if k == 1499:
            before = {b: o.params[0].clone() for b, o in opt.items()}
        g = torch.randn(n, device="cuda", generator=gen) * size
        for o in opt.values():
            o.step([g], lr=1e-3)
    ratio = dequantise(opt[8].v[0], opt[8].v_scale[0]) / opt[32].v[0].sqrt()
    for part in (half, ~half):
        assert abs(float(ratio[part].mean()) - 1) <= 2.0 ** -4
        moves = [float((opt[b].params[0] - before[b])[part].square().mean().sqrt()) for b in (8, 32)]
        assert abs(moves[0] / moves[1] - 1) <= 2.0 ** -3
