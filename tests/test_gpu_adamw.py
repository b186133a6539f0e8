"""AdamW over many tensors: within its roundings of the formula in 64 bits, and bit
for bit the formula's elementary fp32 operations (evaluated on the CPU) in all of
the 32-bit form and in the 8-bit form's states; operand copies, device-side step
numbers."""
import math

import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp
from folded_tensor_sequence_zigzag_gb300.inputs import BlockShape, make_block_inputs

pytestmark = pytest.mark.gpu
U, UBF = 2.0 ** -24, 2.0 ** -8
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
B1, B2, EPS = 0.9, 0.95, 1e-8


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


SIZES = [1, 3, 4, 127, 128, 129, 500, 512, 4095, 4096, 4097, 12345, 33, 65536, 2]


def f32(x):
    return torch.tensor(x, dtype=torch.float32)


def blocks(x):
    """[blocks, 128] with zeros behind the last element."""
    n = x.numel()
    return torch.cat([x.reshape(-1), x.new_zeros(-n % 128)]).view(-1, 128)


def quantise(x, root):
    """(codes, scales) by elementary fp32 operations."""
    b = blocks(x)
    top = b.abs().amax(1)
    live = ~(top < 2.0 ** -100)
    inv = torch.where(live, f32(448.0) * (f32(1.0) / top), f32(0.0))
    scale = torch.where(live, top * (f32(1.0) / f32(448.0)), f32(0.0))
    q = (b * inv[:, None]).to(E4).float()
    if root:
        q = torch.where((b > 0) & (q == 0) & live[:, None], f32(2.0 ** -9), q)
    return q.to(E4).view(-1)[:x.numel()], scale


def dequantise(q, scale):
    return (blocks(q.float()) * scale[:, None]).view(-1)[:q.numel()]


def reference(w, m, v, g, lr, wd, t, gs=1.0, dtype=F32):
    """The update on the CPU, one elementary operation of `dtype` at a time; v of an
    8-bit state comes as its value.  (w, m, v, sqrt(v))"""
    c = (lambda x: torch.tensor(float(x), dtype=dtype)) if dtype == F32 else (lambda x: float(x))
    w, m, v, g = (x.to(dtype) for x in (w, m, v, g))
    g = g * c(gs)
    m = m * c(B1) + g * c(1.0 - B1)
    v = v * c(B2) + (g * g) * c(1.0 - B2)
    root = v.sqrt()
    step, fix = c(lr / (1.0 - B1 ** t)), c(1.0 / math.sqrt(1.0 - B2 ** t))
    keep = c(1.0) - c(lr) * c(wd)
    return w * keep - step * (m / (root * fix + c(EPS))), m, v, root


def make(sizes, dt, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda n: torch.randn(n, generator=gen)   # noqa: E731
    out = []
    for i, n in enumerate(sizes):
        spread = torch.exp(1.5 * r(n)) * 1e-3
        out.append(dict(w=(0.02 * r(n)).to(dt), g=r(n) * spread, m=0.3 * r(n) * spread,
                        v=(spread * (0.2 + torch.rand(n, generator=gen))) ** 2, wd=0.1 * (i % 3)))
    return out


@pytest.mark.parametrize("dt,master", [(F32, False), (BF, True), (BF, False)])
@pytest.mark.parametrize("bits", [32, 8])
def test_update_is_the_formula(dt, master, bits):
    """Three updates of tensors of odd and even sizes in one call each."""
    ts = make(SIZES, dt)
    params = [t["w"].cuda() for t in ts]
    kw = dict(m=[t["m"].cuda() for t in ts], v=[t["v"].cuda() for t in ts])
    if bits == 8:
        for t in ts:
            t["mq"], t["ms"] = quantise(t["m"], False)
            t["vq"], t["vs"] = quantise(t["v"].sqrt(), True)
        kw = dict(m=[t["mq"].cuda() for t in ts], v=[t["vq"].cuda() for t in ts],
                  m_scale=[t["ms"].cuda() for t in ts], v_scale=[t["vs"].cuda() for t in ts])
    opt = tsp.AdamW(params, weight_decay=[t["wd"] for t in ts], state_bits=bits,
                    master=master or None, betas=(B1, B2), eps=EPS, **kw)
    state = [t["w"].float() for t in ts]
    for k in range(3):
        lr, t0, gs = 1e-3 * (k + 1), 7 + k, 0.37
        grads = [t["g"] * (1 + k) for t in ts]
        opt.step([g.cuda() for g in grads], lr=lr, step=t0, gscale=f32([gs]).cuda())
        for i, t in enumerate(ts):
            m, v = t["m"], t["v"]
            if bits == 8:
                m = dequantise(t["mq"], t["ms"])
                r = dequantise(t["vq"], t["vs"])
                v = r * r
            w, m, v, root = reference(state[i], m, v, grads[i], lr, t["wd"], t0, f32(gs).item())
            e = reference(state[i], *((t["m"], t["v"]) if bits == 32 else (
                dequantise(t["mq"], t["ms"]).double(), dequantise(t["vq"], t["vs"]).double() ** 2)),
                grads[i], lr, t["wd"], t0, f32(gs).item(), torch.float64)
            got, exact = opt.params[i].cpu(), (opt.master[i] if master else opt.params[i]).cpu().float()
            if bits == 32:
                assert torch.equal(got, w.to(dt)), (i, k)
                assert not master or torch.equal(exact, w)
            # 64 bits: 2 roundings of w, 16 of the quotient and its factors (an 8-bit
            # state's quotient is two half spacings off instead of one)
            size = (lr / (1 - B1 ** t0)) * (e[1].abs() / (e[3] / math.sqrt(1 - B2 ** t0) + EPS))
            # m is a sum that may cancel: its roundings are of its terms
            mterm = (m.abs() + 2 * grads[i].abs()).double()
            mroom = (lr / (1 - B1 ** t0)) * mterm / (e[3] / math.sqrt(1 - B2 ** t0) + EPS)
            tol = 3 * U * state[i].double().abs() + 3 * U * e[0].abs() + 16 * U * size + 8 * U * mroom
            if dt == BF and not master:
                tol = tol + e[0].abs() * UBF * (1 + UBF)
            assert bool(((exact.double() - e[0]).abs() <= tol).all())
            if master:
                assert torch.equal(got, exact.to(dt))
            state[i] = exact
            if bits == 32:
                assert torch.equal(opt.m[i].cpu(), m) and torch.equal(opt.v[i].cpu(), v)
                t["m"], t["v"] = m, v
            else:
                t["mq"], t["ms"] = quantise(m, False)
                t["vq"], t["vs"] = quantise(root, True)
                assert torch.equal(opt.m_scale[i].cpu(), t["ms"])
                assert torch.equal(opt.v_scale[i].cpu(), t["vs"])
                assert torch.equal(opt.m[i].cpu().float(), t["mq"].float())
                assert torch.equal(opt.v[i].cpu().float(), t["vq"].float())
    assert opt.t == 9 and tsp.device_status() == tsp.TSP_OK


def test_codes_are_within_half_a_step():
    """A held value is off by at most half an e4m3 step (2^-4 of it, or half of
    2^-9 of the scale), the square root of v never by rounding to zero."""
    n = 128 * 40 + 17
    gen = torch.Generator().manual_seed(2)
    g = torch.randn(n, generator=gen) * torch.exp(4 * torch.randn(n, generator=gen))
    opt = tsp.AdamW([torch.zeros(n, device="cuda")], state_bits=8, betas=(B1, B2))
    opt.step([g.cuda()], lr=1e-3)
    m64, r64 = (1 - B1) * g.double(), (1 - B2) ** 0.5 * g.double().abs()
    for q, s, want, root in ((opt.m, opt.m_scale, m64, False), (opt.v, opt.v_scale, r64, True)):
        q, s = q[0].cpu().float().double(), s[0].cpu().double()
        held = (blocks(q) * s[:, None]).view(-1)[:n]
        top = blocks(want.abs()).amax(1)
        assert bool(((s - top / 448).abs() <= 8 * U * s).all())
        step = s.repeat_interleave(128)[:n] * 2.0 ** -9
        tol = want.abs() * (2.0 ** -4 + 16 * U) + step * (0.5 if not root else 1.0)
        assert bool(((held - want).abs() <= tol).all())
        if root:
            assert bool((q[want > 0] > 0).all())


@pytest.mark.parametrize("dt,total", [(BF, 66_000_000), (F32, 31_000_000)])
def test_long_runs_of_chunks(dt, total):
    """Tensors large enough that a CTA takes several chunks in a row (4 of them),
    ragged and empty ones between: chunk ends inside tensors, runs that
    cross from one to the next, on the GPU against elementary operations there."""
    sizes = [total // 2 + 77, 0, 5, 4096 * 3 + 1, total // 4 + 2, 129, 4096, total // 4]
    gen = torch.Generator("cuda").manual_seed(3)
    r = lambda n: torch.randn(n, generator=gen, device="cuda")   # noqa: E731
    params = [(0.02 * r(n)).to(dt) for n in sizes]
    opt = tsp.AdamW(params, weight_decay=0.1, state_bits=8, betas=(B1, B2), eps=EPS)
    state = [p.float().clone() for p in params]
    ref = [(torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")) for n in sizes]
    for k in (1, 2):
        grads = [r(n) * 1e-3 for n in sizes]
        opt.step(grads, lr=1e-3)
        for i, n in enumerate(sizes):
            m, root = ref[i]
            w, m, v, root = reference(state[i], m, root * root, grads[i], 1e-3, 0.1, k)
            got = opt.master[i] if dt == BF else opt.params[i]
            # the quotients differ by 4 u (rcp 2, product 1, division 1) of an update of at
            # most 1e-3 * sqrt(1 / 0.05); two numbers that far apart round to weights at
            # most a spacing further apart, 2 u of the larger
            tol = 2 * U * torch.maximum(w.abs(), got.abs()) + 4 * U * 5e-3
            assert bool(((got - w).abs() <= tol).all()), (i, k)
            assert torch.equal(opt.params[i], got.to(dt))
            state[i] = got.clone()
            if n == 0:
                continue
            qm, sm = quantise(m, False)
            qr, sr = quantise(root, True)
            assert torch.equal(opt.m_scale[i], sm) and torch.equal(opt.v_scale[i], sr), (i, k)
            assert torch.equal(opt.m[i].view(torch.uint8), qm.view(torch.uint8)), (i, k)
            assert torch.equal(opt.v[i].view(torch.uint8), qr.view(torch.uint8)), (i, k)
            ref[i] = dequantise(qm, sm), dequantise(qr, sr)


def test_many_tensors_take_every_launch():
    """More tensors than one launch holds, empty ones among them."""
    sizes = [(7 * i) % 300 for i in range(300)]
    ts = make([n for n in sizes], F32, seed=4)
    opt = tsp.AdamW([t["w"].cuda() for t in ts], weight_decay=0.1, betas=(B1, B2), eps=EPS,
                    m=[t["m"].cuda() for t in ts], v=[t["v"].cuda() for t in ts])
    n0 = tsp.launch_count()
    opt.step([t["g"].cuda() for t in ts], lr=1e-3, step=5)
    assert tsp.launch_count() - n0 == 3
    for i, t in enumerate(ts):
        w, m, v, _ = reference(t["w"], t["m"], t["v"], t["g"], 1e-3, 0.1, 5)
        assert torch.equal(opt.params[i].cpu(), w) and torch.equal(opt.m[i].cpu(), m)


@pytest.mark.parametrize("bits", [32, 8])
def test_step_from_the_device_in_a_replayed_graph(bits):
    """lr, step and gscale as GPU tensors: a replay uses what they hold then, and
    equals calls with the numbers (the bias corrections are formed in 64 bits on
    either side and rounded to fp32: within 2 u of each other, so w is within 4 u
    of the size of its update; the states do not depend on them)."""
    ts = make([1000, 129, 4096], F32, seed=6)

    def new():
        return tsp.AdamW([t["w"].cuda() for t in ts], weight_decay=0.1, state_bits=bits,
                         betas=(B1, B2), eps=EPS)
    a, b = new(), new()
    grads = [t["g"].cuda() for t in ts]
    lr, step = f32([0.0]).cuda(), torch.zeros(1, dtype=torch.int64, device="cuda")
    gs = f32([1.0]).cuda()
    a.step(grads, lr=lr, step=step + 1, gscale=gs)   # lr 0: the weights stay, warm-up of the states
    b.step(grads, lr=0.0, step=1, gscale=gs)
    for x, y in zip(a.params + a.m, b.params + b.m):
        assert torch.equal(x.float(), y.float())
    step.fill_(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        a.step(grads, lr=lr, step=step, gscale=gs)
    for k in range(4):
        lr.fill_(1e-3 * (k + 1))
        gs.fill_(0.5 + k)
        graph.replay()
        b.step(grads, lr=float(f32(1e-3 * (k + 1))), step=2 + k, gscale=gs)
    assert int(step) == 5
    for i in range(len(ts)):
        for x, y in ((a.m[i], b.m[i]), (a.v[i], b.v[i])):
            assert torch.equal(x.float(), y.float())
        # four updates, each at most lr / (1 - beta1^t) * |m| / sqrt(v) <= 1e-2 * 10 large
        assert bool(((a.params[i] - b.params[i]).abs() <= 4 * 4 * U * 0.1
                     + 8 * U * b.params[i].abs()).all())


def test_non_finite_gradients_stay_where_the_formula_puts_them():
    n = 512
    for bits in (32, 8):
        g = torch.ones(n)
        g[5], g[300] = float("nan"), float("inf")
        opt = tsp.AdamW([torch.zeros(n, device="cuda")], state_bits=bits, betas=(B1, B2))
        opt.step([g.cuda()], lr=1e-3)
        w = opt.params[0].cpu()
        assert torch.isnan(w[5]) and torch.isnan(w[300])       # inf / inf
        w[5] = w[300] = 0
        assert w.isfinite().all()
        if bits == 8:      # a block with one of them has no finite scale, the others do
            assert opt.m_scale[0].isfinite().cpu().tolist() == [False, True, False, True]


def test_tiny_and_zero_blocks():
    g = torch.zeros(384)
    g[128:256] = 1e-35                    # m of 1e-36 is below the floor of a block
    g[256] = 1.0
    opt = tsp.AdamW([torch.zeros(384, device="cuda")], state_bits=8, betas=(B1, B2))
    for _ in range(2):
        opt.step([g.cuda()], lr=1e-3)
    assert opt.params[0].isfinite().all() and not opt.params[0][:128].any()
    assert opt.m_scale[0].cpu()[:2].tolist() == [0.0, 0.0] and opt.m_scale[0][2] > 0


def test_prepared_copies_equal_weights_prepare():
    """The fp16 operand copies an update leaves are bit for bit what
    prepare_weights makes of the updated weights, and the prepared forward runs
    on them."""
    shape = BlockShape(S=2048, d=256, H=2, inter=384, D=4)
    inp = make_block_inputs(shape, BF, seed=1, with_dy=True)
    cfg = tsp.make_cfg(shape.S, shape.d, shape.H, shape.inter, shape.D, BF)
    W = tsp.BlockWeights.from_dict(inp, "cuda")
    prep = tsp.prepare_weights(cfg, W)
    opt = tsp.AdamW(W.params(), weight_decay=0.1, prep=tsp.prep_views(cfg, prep))
    xz, dyz = (tsp.zigzag_permute(inp[k].cuda(), shape.D) for k in ("x", "dy"))
    saved = tsp.empty(tsp.saved_bytes(cfg), torch.uint8, "cuda")
    tsp.block_fwd(cfg, xz, W, saved=saved, prep=prep)
    g = tsp.block_bwd(cfg, xz, dyz, saved, W, prep=prep)
    before = [p.clone() for p in W.params()]
    opt.step([g[k] for k in tsp.GRAD_NAMES], lr=1e-2)
    assert all(not torch.equal(p, q) for p, q in zip(before, W.params()))
    fresh = tsp.prepare_weights(cfg, W)
    for a, b in zip(tsp.prep_views(cfg, prep)[:7], tsp.prep_views(cfg, fresh)[:7]):
        assert torch.equal(a, b)
    assert torch.equal(tsp.block_fwd(cfg, xz, W, prep=prep), tsp.block_fwd(cfg, xz, W))
    assert tsp.device_status() == tsp.TSP_OK


def test_a_weight_past_fp16_is_recorded():
    w = torch.tensor([1.0, 7e4, 2.0, 3.0], dtype=BF, device="cuda")
    prep = torch.zeros(4, dtype=torch.float16, device="cuda")
    opt = tsp.AdamW([w], master=None, prep=[prep])
    opt.step([torch.zeros(4, device="cuda")], lr=1e-3)
    assert tsp.device_status() == tsp.TSP_ERR_RANGE
    assert prep[0] == 1.0 and torch.equal(w.cpu(), torch.tensor([1.0, 7e4, 2.0, 3.0], dtype=BF))
    assert tsp.device_status() == tsp.TSP_OK


@pytest.mark.parametrize("bits", [32, 8])
def test_element_offsets_past_32_bits(bits):
    """A tensor of more than 2^31 elements: the same blocks become the same bits,
    wherever they are."""
    period, times, rest = 1 << 20, 2050, 5 * 128 + 3
    gen = torch.Generator("cuda").manual_seed(2)
    w = (0.02 * torch.randn(period, device="cuda", generator=gen)).to(BF)
    g = 1e-3 * torch.randn(period, device="cuda", generator=gen)

    def repeated(x):
        return torch.cat([x.repeat(times), x[:rest]])
    small = tsp.AdamW([w], weight_decay=0.1, state_bits=bits, master=None, betas=(B1, B2), eps=EPS)
    big = tsp.AdamW([repeated(w)], weight_decay=0.1, state_bits=bits, master=None, betas=(B1, B2), eps=EPS)
    grad = repeated(g)
    for _ in range(2):
        small.step([g], lr=1e-3)
        big.step([grad], lr=1e-3)
    for name in ("params", "m", "v", "m_scale", "v_scale"):
        a, b = getattr(big, name)[0], getattr(small, name)[0]
        if a is None:
            continue
        if a.dtype == E4:
            a, b = a.view(torch.uint8), b.view(torch.uint8)
        k = len(b)
        assert bool((a[:times * k].view(times, k) == b).all()), name
        tail = a[times * k:]
        if "scale" in name:      # the last block is a part of the small tensor's sixth
            tail = tail[:-1]
        whole = 5 * 128 if bits == 8 and name in ("m", "v", "params") else len(tail)
        assert torch.equal(tail[:whole], b[:whole] if "scale" not in name else b[:len(tail)]), name
    # the block that ends with the tensor has scales of its own, of the elements that are there
    q = bits == 8
    if q:
        assert bool((big.m_scale[0][-1] <= small.m_scale[0][5]) & (big.v_scale[0][-1] > 0))


def test_two_objects_at_once():
    """Steps on two streams, each with its own tensors."""
    sizes = [100_000, 77, 4096 * 40]
    ts = [make(sizes, F32, seed=s) for s in (1, 2)]

    def new():
        return [tsp.AdamW([x["w"].cuda() for x in t], state_bits=8, betas=(B1, B2), eps=EPS) for t in ts]
    one, two = new(), new()
    grads = [[x["g"].cuda() for x in t] for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    for _ in range(5):
        for o, g, s in zip(two, grads, streams):
            o.step(g, lr=1e-3, stream=s)
    torch.cuda.synchronize()
    for _ in range(5):
        for o, g in zip(one, grads):
            o.step(g, lr=1e-3)
    for a, b in zip(one, two):
        assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.m, b.m))
