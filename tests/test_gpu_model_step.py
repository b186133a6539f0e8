"""The operators together, as a program uses them around the block stack."""
import math

import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp
from folded_tensor_sequence_zigzag_gb300.inputs import BlockShape, make_block_inputs

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


@pytest.mark.parametrize("dt,bits", [(torch.float32, 32), (torch.bfloat16, 8)])
def test_training_step_of_a_stack_with_its_table(dt, bits):
    """tokens -> table -> two blocks -> gradients -> one AdamW update of all 19
    tensors.  Each operator is held to what the others hand it: the stack runs on
    the embedded rows, the table's gradient is the sum of the stack's dx rows, and
    the updated weights give the forward that fresh copies of them give."""
    bf = dt == torch.bfloat16
    shape = BlockShape(S=2048, d=256, H=2, inter=384, D=4) if bf else BlockShape(S=64, d=32, H=2, inter=48, D=2)
    S, d, D, V, L = shape.S, shape.d, shape.D, 101, 2
    cfg = tsp.make_cfg(S, d, shape.H, shape.inter, D, dt)
    Ws = [tsp.BlockWeights.from_dict(make_block_inputs(shape, dt, seed=s), "cuda") for s in (1, 2)]
    gen = torch.Generator().manual_seed(3)
    table = (0.05 * torch.randn(V, d, generator=gen)).to(dt).cuda()
    ids = torch.randint(0, V - 1, (S,), generator=gen)
    ids[::9] = -1                                     # padding
    ids, scale = ids.cuda(), math.sqrt(d)
    dy = torch.randn(S, d, generator=gen).to(dt).cuda()
    preps = [tsp.prepare_weights(cfg, W) for W in Ws] if bf else None
    prep = [None] + [v for p in preps for v in tsp.prep_views(cfg, p)] if bf else None
    params = [table] + [p for W in Ws for p in W.params()]
    opt = tsp.AdamW(params, weight_decay=[0.0] + ([0.1] * 7 + [0.0] * 2) * L, state_bits=bits, prep=prep)

    x = tsp.embed_fwd(ids, table, D=D, scale=scale)
    want = torch.where((ids >= 0)[:, None], table[ids.clamp(min=0)].float() * scale, 0.0).to(dt)
    assert torch.equal(x, tsp.zigzag_permute(want, D))
    saved = tsp.empty(tsp.stack_saved_bytes(cfg, L), torch.uint8, "cuda")
    tsp.stack_fwd(cfg, x, Ws, saved=saved, preps=preps)
    dx, grads = tsp.stack_bwd(cfg, dy, saved, Ws, preps=preps)
    dtable = tsp.embed_bwd(ids, dx, V, D=D, scale=scale)
    rows = tsp.zigzag_permute(dx, D, inverse=True).double()
    there, at = ids >= 0, ids.clamp(min=0)
    ref = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, at[there], rows[there] * scale)
    mag = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, at[there], rows[there].abs() * scale)
    assert bool(((dtable.double() - ref).abs() <= (S + 3) * U * mag).all())
    assert not dtable[V - 1].any()                    # the token that no position has

    before = [p.clone() for p in params]
    opt.step([dtable] + [g[k] for g in grads for k in tsp.GRAD_NAMES], lr=1e-2)
    # the first update moves a weight by lr * g / (|g| + eps'): against its gradient, by at most lr
    for p, q, g in zip(params, before, [dtable] + [g[k] for g in grads for k in tsp.GRAD_NAMES]):
        move = p.float() - q.float()
        limit = 1e-2 * (1 + 0.1 * q.float().abs()) * 1.01 + (q.float().abs() + 1e-2) * 2.0 ** -8
        assert bool((move.abs() <= limit).all())
        seen = g.abs() > 1e-4
        assert bool((move * g)[seen & (q.float().abs() < 0.05)].le(0).all())
    assert torch.equal(table[V - 1], before[0][V - 1])
    x = tsp.embed_fwd(ids, table, D=D, scale=scale)
    y = tsp.stack_fwd(cfg, x, Ws, preps=preps)
    assert torch.equal(y, tsp.stack_fwd(cfg, x, Ws)) and y.isfinite().all()
    assert tsp.device_status() == tsp.TSP_OK


def test_sandwich_norm_around_the_bare_mlp():
    """norm_residual_fwd between two gated MLPs run without their own norm and
    residual: pre-norm in, post-norm, gate and scaled residual out.  Against the
    same chain in 64 bits on the MLPs' actual outputs, and with the pre-norm MLP
    call as the special case of no post-norm and no gate."""
    S, d, inter, D = 512, 256, 384, 2
    shape = BlockShape(S=S, d=d, H=2, inter=inter, D=D)
    W = tsp.BlockWeights.from_dict(make_block_inputs(shape, torch.bfloat16, seed=4), "cuda")
    cfg = tsp.make_cfg(S, d, 2, inter, D, torch.bfloat16)
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(S, d, generator=gen).cuda()
    gate = torch.randn(S, d, generator=gen).bfloat16().cuda()
    gp, gq = ((1 + 0.2 * torch.randn(d, generator=gen)).bfloat16().cuda() for _ in range(2))
    zero = torch.zeros(S, d, dtype=torch.bfloat16, device="cuda")
    h0, b0 = tsp.norm_residual_fwd(zero, x, g_pre=gq)        # the first pre-norm
    assert torch.equal(h0, x)
    f = tsp.gated_mlp_fwd(cfg, b0, W, norm=False, residual=False)
    h1, b1 = tsp.norm_residual_fwd(f, h0, g_post=gp, g_pre=gq, gate=gate, scale=0.5)
    f64, g64 = f.double(), gate.double()
    u = f64 * (f64.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gp.double() * torch.sigmoid(g64)
    want = x.double() + 0.5 * u
    assert bool(((h1.double() - want).abs() <= 60 * U * (0.5 * u.abs() + want.abs())).all())
    wb = h1.double() * (h1.double().square().mean(1, keepdim=True) + 1e-6).rsqrt() * gq.double()
    assert bool(((b1.double() - wb).abs() <= wb.abs() * (2.0 ** -8 + 60 * U)).all())
    f = tsp.gated_mlp_fwd(cfg, b1, W, norm=False, residual=False)
    h2, none = tsp.norm_residual_fwd(f, h1)                  # plain residual at the end
    assert none is None
    assert bool(((h2.double() - h1.double() - f.double()).abs() <= 2 * U * h2.double().abs()).all())
    assert tsp.device_status() == tsp.TSP_OK
