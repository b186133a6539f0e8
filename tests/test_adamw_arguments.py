"""What AdamW refuses beyond pointers and ranges: arrays that share memory (the C entry
point with made-up addresses; only where no GPU could run a call that passed) and
shapes that differ though the number of elements does not."""
import ctypes

import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp

AT = 0x100000
NAMES = ("w", "master", "g", "m", "v", "m_scale", "v_scale", "prep")
# bytes of each array of 1000 elements (bf16 weights; 8-bit states, 8 blocks)
BYTES = dict(w=2000, master=4000, g=4000, m=1000, v=1000, m_scale=32, v_scale=32, prep=2000)


@pytest.fixture(scope="module")
def lib():
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


def addresses(order):
    """Two tensors' arrays, all apart; `order` says how they lie in memory."""
    every = [(i, k) for i in range(2) for k in NAMES]
    if order == "by kind":
        every = [(i, k) for k in NAMES for i in range(2)]
    if order == "falling":
        every = every[::-1]
    return {x: AT + 0x2000 * j for j, x in enumerate(every)}


def step(lib, at, hyper=None):
    arr = (tsp.AdamwTensor * 2)()
    for i, t in enumerate(arr):
        t.n, t.weight_decay = 1000, 0.1
        for k in NAMES:
            setattr(t, k, at[i, k])
    hy = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1)
    hy.update(hyper or {})
    return lib.tsp_adamw_step(arr, 2, ctypes.byref(tsp.AdamwHyper(**hy)), 8, 1, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
@pytest.mark.parametrize("order", ["by tensor", "by kind", "falling"])
def test_arrays_that_share_memory_are_refused(lib, order):
    """Each pair of arrays, of one tensor and of two, at one address, with the one's
    last bytes in the other's first; ends that touch pass (and find no GPU here)."""
    base = addresses(order)
    assert step(lib, base) != tsp.TSP_ERR_INVALID_ARG
    for a in base:
        for b in base:
            if a == b:
                continue
            last = (BYTES[a[1]] - 1) // 16 * 16
            touch = -(-BYTES[a[1]] // 16) * 16
            refused = (a[1], b[1]) != ("g", "g")
            for shift, hit in ((0, True), (last, True), (touch, False)):
                at = dict(base)
                at[b] = base[a] + shift
                got = step(lib, at) == tsp.TSP_ERR_INVALID_ARG
                assert got == (refused and hit), (a, b, shift)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
def test_values_on_the_device_are_apart_from_what_is_written(lib):
    base = addresses("by tensor")
    for k in NAMES:
        for name, size in (("lr_dev", 4), ("step_dev", 8), ("gscale_dev", 4)):
            at = base[1, k] + BYTES[k] - size
            got = step(lib, base, {name: at - at % 8})
            assert (got == tsp.TSP_ERR_INVALID_ARG) == (k != "g"), (k, name)


def test_shapes_are_compared():
    """A transposed gradient, state, master or copy has the right number of elements;
    flat ones are taken."""
    p = [torch.zeros(6, 4).bfloat16(), torch.zeros(4, 6).bfloat16()]
    opt = tsp.AdamW(p)
    g = [torch.zeros(6, 4), torch.zeros(4, 6)]
    for bad in (g[::-1], [g[0], g[0]], [g[0].view(2, 12), g[1]], [g[0].view(6, 4, 1), g[1]],
                [g[0].view(1, 24), g[1]], g[:1], g + g[:1], []):
        with pytest.raises(ValueError, match="gradients"):
            opt.step(bad, lr=1e-3)
    for name, dt in (("m", torch.float32), ("v", torch.float32), ("master", torch.float32),
                     ("prep", torch.float16)):
        with pytest.raises(ValueError, match="tensor"):
            tsp.AdamW(p, **{name: [torch.zeros(4, 6, dtype=dt), torch.zeros(4, 6, dtype=dt)]})
        tsp.AdamW(p, **{name: [torch.zeros(24, dtype=dt), torch.zeros(4, 6, dtype=dt)]})
    assert opt.t == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
@pytest.mark.parametrize("eps,ok", [(0.0, True), (1e-8, True), (2.0 ** -126, True), (2.0 ** 100, True),
                                    (1e-39, False), (2.0 ** -149, False), (1.01 * 2.0 ** 100, False),
                                    (1e39, False), (1e-50, True)])   # (the last is 0 in fp32)
def test_an_eps_whose_reciprocal_is_no_normal_number(lib, eps, ok):
    """8-bit states divide by a reciprocal that takes subnormals for zero: 0 / 1e-39 would
    be NaN.  Such an eps is refused; in 32 bits it is divided by."""
    base = addresses("by tensor")
    assert (step(lib, base, dict(eps=eps)) == tsp.TSP_ERR_INVALID_ARG) == (not ok)
    arr = (tsp.AdamwTensor * 1)()
    arr[0].n, arr[0].w, arr[0].g, arr[0].m, arr[0].v = 1000, AT, 2 * AT, 3 * AT, 4 * AT
    hy = tsp.AdamwHyper(1e-3, 0.9, 0.95, eps, 1)
    assert lib.tsp_adamw_step(arr, 1, ctypes.byref(hy), 32, 0, None) != tsp.TSP_ERR_INVALID_ARG


def test_a_beta2_that_8_bit_states_do_not_follow(lib):
    p = [torch.zeros(300)]
    for beta2, ok in ((0.0, True), (0.95, True), (0.97, True), (0.98, False), (0.999, False)):
        if ok:
            tsp.AdamW(p, state_bits=8, betas=(0.9, beta2))
        else:
            with pytest.raises(ValueError, match="beta2"):
                tsp.AdamW(p, state_bits=8, betas=(0.9, beta2))
        tsp.AdamW(p, state_bits=32, betas=(0.9, beta2))
        if not torch.cuda.is_available():                       # (made-up addresses)
            base = addresses("by tensor")
            assert (step(lib, base, dict(beta2=beta2)) == tsp.TSP_ERR_INVALID_ARG) == (not ok)
