"""An error in the device status word holds an update back: the gradients behind it
may be what a kernel that returned without its work left.  Either every tensor of a
call is updated or none, also where the call records the error itself."""
import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp
from folded_tensor_sequence_zigzag_gb300.inputs import BlockShape, make_block_inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


def record_an_error():
    """A token id past its table."""
    tsp.embed_fwd(torch.tensor([3], device="cuda"), torch.zeros(3, 8, device="cuda"))


def held(opt):
    """Everything an update writes, as bytes."""
    every = opt.params + opt.m + opt.v + opt.m_scale + opt.v_scale + opt.master + opt.prep
    return [t.clone().view(torch.uint8) for t in every if t is not None and t.numel()]


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def make(sizes, dt, bits, master, prep, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    ps = [(0.02 * torch.randn(n, generator=gen, device="cuda")).to(dt) for n in sizes]
    gs = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
    copies = [torch.zeros(n, dtype=torch.float16, device="cuda") for n in sizes] if prep else None
    return tsp.AdamW(ps, weight_decay=0.1, state_bits=bits, master=master, prep=copies), gs


# one cluster (up to 16 chunks of 4096), single chunks, runs of chunks (8-bit states: from
# 152 * 12 chunks on) and tails; more tensors than one launch holds
SIZES = {"one": [5], "few": [1, 129, 4097, 0, 33000], "some": [4096 * 16, 3], "medium": [1_000_001, 77], "large": [9_000_001, 77], "many": [(37 * i) % 900 for i in range(300)]}


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dt,master,prep", [(F32, None, False), (BF, True, True), (BF, None, False)])
def test_an_error_holds_the_update_back(sizes, bits, dt, master, prep):
    opt, grads = make(SIZES[sizes], dt, bits, master, prep)
    other, _ = make(SIZES[sizes], dt, bits, master, prep)
    opt.step(grads, lr=1e-2)
    other.step(grads, lr=1e-2)
    before = held(opt)
    record_an_error()
    nan = [torch.full_like(g, float("nan")) for g in grads]
    for _ in range(2):
        opt.step(nan, lr=1e-2)
    assert same(before, held(opt))
    assert opt.t == 3
    assert tsp.device_status() == tsp.TSP_ERR_RANGE
    opt.t = 1
    opt.step(grads, lr=1e-2)
    other.step(grads, lr=1e-2)
    assert not same(before, held(opt)) and same(held(opt), held(other))
    assert tsp.device_status() == tsp.TSP_OK


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[9_000_001, 77, 5000], [300] * 300, [300] * 10, [40_000, 77], [300_000]])
def test_an_error_of_its_own_stops_no_part_of_an_update(bits, sizes):
    """The first weight does not fit fp16: every tensor is updated all the same, and
    the next step is held back."""
    opt, grads = make(sizes, BF, bits, True, True)
    other, _ = make(sizes, BF, bits, True, False)
    for o in (opt, other):
        o.params[0][0] = 7e4
        o.master[0][0] = 7e4
    other.step(grads, lr=1e-2)       # (before the error that would hold it back)
    opt.step(grads, lr=1e-2)
    for name in ("params", "m", "v", "master"):
        assert same([x.view(torch.uint8) for x in getattr(opt, name)],
                    [x.view(torch.uint8) for x in getattr(other, name)]), name
    assert all(torch.equal(p[1:], c[1:].to(BF)) or torch.equal(p[1:].half(), c[1:])
               for p, c in zip(opt.params, opt.prep))
    before = held(opt)
    opt.step(grads, lr=1e-2)
    assert same(before, held(opt))
    assert tsp.device_status() == tsp.TSP_ERR_RANGE and tsp.device_status() == tsp.TSP_OK


def test_replays_look_at_the_word_anew():
    """A captured step with the call in front of it that may record an error."""
    opt, grads = make([5000, 77], F32, 32, None, False)
    other, _ = make([5000, 77], F32, 32, None, False)
    ids, table = torch.tensor([0, 1], device="cuda"), torch.zeros(3, 8, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        tsp.embed_fwd(ids, table)
        opt.step(grads, lr=1e-2, step=step)
    for k, bad in enumerate([False, True, True, False]):
        ids[0] = 3 if bad else 0
        before = held(opt)
        graph.replay()
        if bad:
            assert same(before, held(opt))
        else:
            other.step(grads, lr=1e-2, step=k + 1)
            # (equal to the last bit but for the bias corrections, formed on the device
            # here: 2 u of an update of at most lr * 10 each, and the weight's rounding)
            for p, q in zip(opt.params, other.params):
                assert bool(((p - q).abs() <= 2 * 4 * 2.0 ** -24 * 0.1 + 4 * 2.0 ** -24 * q.abs()).all())
            assert all(torch.equal(x, y) for x, y in zip(opt.m + opt.v, other.m + other.v))
        assert tsp.device_status() == (tsp.TSP_ERR_RANGE if bad else tsp.TSP_OK)


def test_a_bad_token_does_not_reach_the_weights():
    """A training step whose batch holds an id past the table: the contraction kernels
    leave the gradients unwritten, and the step behind them changes nothing."""
    shape = BlockShape(S=2048, d=256, H=2, inter=384, D=4)
    cfg = tsp.make_cfg(shape.S, shape.d, shape.H, shape.inter, shape.D, BF)
    W = tsp.BlockWeights.from_dict(make_block_inputs(shape, BF, seed=1), "cuda")
    prep = tsp.prepare_weights(cfg, W)
    gen = torch.Generator().manual_seed(2)
    table = torch.randn(50, shape.d, generator=gen).to(BF).cuda()
    ids = torch.randint(0, 50, (shape.S,), generator=gen).cuda()
    dy = torch.randn(shape.S, shape.d, generator=gen).to(BF).cuda()
    opt = tsp.AdamW([table] + W.params(), prep=[None] + tsp.prep_views(cfg, prep))
    saved = tsp.empty(tsp.stack_saved_bytes(cfg, 1), torch.uint8, "cuda")

    def train():
        x = tsp.embed_fwd(ids, table, D=shape.D)
        tsp.stack_fwd(cfg, x, [W], saved=saved, preps=[prep])
        dx, grads = tsp.stack_bwd(cfg, dy, saved, [W], preps=[prep])
        dtable = tsp.embed_bwd(ids, dx, 50, D=shape.D)
        opt.step([dtable] + [grads[0][k] for k in tsp.GRAD_NAMES], lr=1e-3)
    train()
    assert tsp.device_status() == tsp.TSP_OK
    before = held(opt)
    ids[100] = 50
    train()
    assert same(before, held(opt)) and all(p.isfinite().all() for p in opt.params)
    ids[100] = 49
    train()                                        # nobody has asked for the status yet
    assert same(before, held(opt))
    assert tsp.device_status() == tsp.TSP_ERR_RANGE
    train()
    assert not same(before, held(opt)) and all(p.isfinite().all() for p in opt.params)
    assert tsp.device_status() == tsp.TSP_OK
