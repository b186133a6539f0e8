"""The log probability and loss calls together with the rest of the framework, as a
training step, a distillation and a decode step use them; under the checked build; and
captured by a process that has not called them before."""
import math
import os
import subprocess
import sys

import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp
from folded_tensor_sequence_zigzag_gb300.inputs import BlockShape, make_block_inputs

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U, E2 = 2.0 ** -24, 2.0 ** -22


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


def sum_tolerance(V):
    """Of l and of a log probability (see the tests of the calls themselves): summands of
    8 E2 and V / 1024 + 64 roundings, logits that are far below the largest by at most 60."""
    return 8 * E2 + (V / 1024 + 64) * U + 8 * U * 68 + 8 * U * 60


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_distillation_step_with_a_tied_table(dt):
    """tokens -> table -> two blocks -> logits by the same table -> loss of the next tokens
    and of another model's eight best -> gradients -> AdamW.  Each call is held to what the
    others hand it: the loss to the logits, the table's gradient to the sum of both uses."""
    bf = dt == torch.bfloat16
    shape = BlockShape(S=2048, d=256, H=2, inter=384, D=4) if bf else BlockShape(S=64, d=32, H=2, inter=48, D=2)
    S, d, D, V, L = shape.S, shape.d, shape.D, 515, 2
    cfg = tsp.make_cfg(S, d, shape.H, shape.inter, D, dt)
    Ws = [tsp.BlockWeights.from_dict(make_block_inputs(shape, dt, seed=s), "cuda") for s in (1, 2)]
    gen = torch.Generator().manual_seed(3)
    table = (0.05 * torch.randn(V, d, generator=gen)).to(dt).cuda()
    tokens = torch.randint(0, V, (S,), generator=gen).cuda()
    target = torch.roll(tokens, -1)
    target[-1] = -1                                    # nothing follows the last token
    target[5::7] = -1                                  # padding
    live = target >= 0
    weight = torch.full((S,), 1.0 / int(live.sum()), device="cuda")

    x = tsp.embed_fwd(tokens, table, D=D, scale=math.sqrt(d))
    saved = tsp.empty(tsp.stack_saved_bytes(cfg, L), torch.uint8, "cuda")
    y = tsp.stack_fwd(cfg, x, Ws, saved=saved)
    logits = y @ table.t()
    teacher = tsp.logprobs_fwd((y @ torch.flip(table, (0,)).t()), D=D, top=8)
    before = logits.clone()
    out = tsp.token_loss_fwd(logits, target, teacher["top_ids"], teacher["top_logp"], w_ce=0.4, w_kd=0.6, D=D,
                             dloss=weight, dlogits=logits)          # the gradient takes the logits' place
    assert out["dlogits"].data_ptr() == logits.data_ptr()

    row = tsp.zigzag_permute(torch.arange(S, device="cuda").view(S, 1), D)[:, 0]   # position of each row
    z = torch.empty(S, V, dtype=torch.float64, device="cuda")
    z[row] = before.double()
    logp = torch.log_softmax(z, 1)
    q = torch.softmax(teacher["top_logp"].double(), 1)
    at = teacher["top_ids"].long()
    one = torch.arange(S, device="cuda")
    want = -0.4 * logp[one, target.clamp(min=0)] + 0.6 * (q * (q.log() - logp.gather(1, at))).sum(1)
    tol = 2 * sum_tolerance(V) + 40 * U * want.abs() + 320 * U * 30
    assert bool(((out["loss"].double() - want).abs() <= tol)[live].all()) and not out["loss"][~live].any()
    grad = logp.exp()
    grad[one, target.clamp(min=0)] -= 0.4
    grad.scatter_add_(1, at, -0.6 * q)
    grad = torch.where(live[:, None], grad * weight.double()[:, None], 0.0)
    off = (logits.double() - grad[row]).abs()
    step = 2.0 ** -8 if bf else 2 * U
    assert bool((off <= grad[row].abs() * step * 1.01 + weight[0].item() * (sum_tolerance(V) + 400 * U) + 1e-30).all())

    dy = (logits @ table).to(dt)
    dtable = (logits.float().t() @ y.float()).contiguous()
    head = dtable.clone()
    dx, grads = tsp.stack_bwd(cfg, dy, saved, Ws)
    tsp.embed_bwd(tokens, dx, V, D=D, scale=math.sqrt(d), out=dtable, accumulate=True)
    rows = tsp.zigzag_permute(dx, D, inverse=True).double() * math.sqrt(d)
    ref = head.double().index_add_(0, tokens, rows)
    mag = head.double().abs().index_add_(0, tokens, rows.abs())
    assert bool(((dtable.double() - ref).abs() <= (S + 4) * U * mag).all())
    params = [table] + [p for W in Ws for p in W.params()]
    opt = tsp.AdamW(params, weight_decay=0.0)
    old = table.clone()
    opt.step([dtable] + [g[k] for g in grads for k in tsp.GRAD_NAMES], lr=1e-3)
    seen = dtable.abs() > 1e-5
    assert bool(((table.float() - old.float()) * dtable)[seen].le(0).all()) and table.isfinite().all()
    assert tsp.device_status() == tsp.TSP_OK


def test_the_gradient_in_two_ways():
    """The policy gradient of sum(a * logp): logprobs_bwd against token_loss_bwd with -a as
    the loss's weight, which is the same function."""
    gen = torch.Generator().manual_seed(4)
    S, V, D = 96, 1003, 4
    logits = (2 * torch.randn(S, V, generator=gen)).cuda()
    ids = torch.randint(-1, V, (S,), generator=gen).cuda()
    a = torch.randn(S, generator=gen).cuda()
    f = tsp.logprobs_fwd(logits, ids, D=D, scale=0.9, stats=True)
    g = tsp.logprobs_bwd(logits, ids, f["stats"], dlogp=a, D=D, scale=0.9)
    h = tsp.token_loss_bwd(logits, f["stats"], ids, dloss=-a, D=D, scale=0.9)
    # both have p (A) + what the token adds, with A = -+ a scale and the same p: one rounding each
    assert bool(((g - h).abs() <= 4 * U * (g.abs() + h.abs()) + 2 * U * a.abs().max()).all())
    loss = tsp.token_loss_fwd(logits, ids, D=D, scale=0.9)["loss"]
    assert bool(((loss + f["logp"]).abs() <= sum_tolerance(V) * 2 + 16 * U * f["logp"].abs()).all())


def test_decoded_tokens_are_scored():
    """Prefill, then three tokens decoded; their log probabilities and alternatives are
    those of the whole sequence's logits at the same positions."""
    shape = BlockShape(S=64, d=32, H=2, inter=48, D=2)
    cfg = tsp.make_cfg(shape.S, shape.d, shape.H, shape.inter, shape.D, torch.float32)
    W = tsp.BlockWeights.from_dict(make_block_inputs(shape, torch.float32, seed=6), "cuda")
    gen = torch.Generator().manual_seed(7)
    V = 777
    table = torch.randn(V, shape.d, generator=gen).cuda()
    tokens = torch.randint(0, V, (shape.S + 3,), generator=gen).cuda()
    cache = tsp.KVCache(cfg, shape.S + 3)
    tsp.block_prefill(cfg, tsp.embed_fwd(tokens[:shape.S], table, D=shape.D), W, cache)
    y = tsp.block_decode(cfg, tsp.embed_fwd(tokens[shape.S:], table), W, cache)
    logits = y @ table.t()
    got = tsp.logprobs_fwd(logits, tokens[shape.S:].roll(-1), top=5, entropy=True, scale=0.5)
    ref = torch.log_softmax(logits.double() * 0.5, 1)
    tol = sum_tolerance(V)
    assert bool(((got["logp"].double() - ref[torch.arange(3), tokens[shape.S:].roll(-1)]).abs() <= tol).all())
    best = torch.topk(logits, 5, 1).indices
    assert torch.equal(got["top_ids"].long(), best)
    assert bool(((got["top_logp"].double() - ref.gather(1, best)).abs() <= tol).all())
    assert bool(((got["entropy"].double() + (ref.exp() * ref).sum(1)).abs() <= 20 * tol).all())


SCRIPT = r"""
import sys, torch
sys.path.insert(0, sys.argv[3])
from folded_tensor_sequence_zigzag_gb300 import tsp
tsp.load(sys.argv[1])
gen = torch.Generator().manual_seed(1)
out = {}
for S, V, D, dt, K, wide in ((24, 1000, 4, torch.bfloat16, 8, 3), (7, 50257, 1, torch.float32, 20, 0), (3, 131075, 1, torch.bfloat16, 64, 5),
                             (600, 4099, 3, torch.float32, 0, 0), (2, 40000, 1, torch.bfloat16, 200, 0), (1, 500001, 1, torch.float32, 7, 0)):
    x = (2 * torch.randn(S, V + wide, generator=gen)).to(dt).cuda()[:, :V]
    ids = torch.randint(-2, V, (S,), generator=gen).cuda()
    up = torch.rand(S, generator=gen).cuda()
    f = tsp.logprobs_fwd(x, ids, D=D, top=max(1, min(K, 250)), entropy=True, stats=True)
    d = tsp.logprobs_bwd(x, ids, f["stats"], dlogp=up, entropy=f["entropy"], dentropy=up, D=D)
    kw = dict(ids=ids, D=D, w_ce=0.5, w_kd=0.5, dloss=up)
    if K:
        kw.update(t_ids=torch.randint(-1, V, (S, K), generator=gen).int().cuda(), t_logits=torch.randn(S, K, generator=gen).cuda())
    o = tsp.token_loss_fwd(x, grad=True, stats=True, **kw)
    e = tsp.token_loss_bwd(x, o["stats"], **kw)
    other = torch.empty(S, V + 1, dtype=dt, device="cuda")[:, :V]
    tsp.token_loss_bwd(x, o["stats"], out=other, **kw)
    out.update({f"{k}{S}": v.cpu() for k, v in dict(f, d=d, e=e, other=other, **{"o" + k: v for k, v in o.items()}).items()})
torch.cuda.synchronize()
st = tsp.device_status()
if st != tsp.TSP_OK:
    raise SystemExit(f"status {st} ({tsp.strerror(st)})")
torch.save(out, sys.argv[2])
"""


def _run(script, *args):
    r = subprocess.run([sys.executable, "-c", script, *args, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]


def test_checked_build_runs_clean_and_matches(tmp_path):
    from folded_tensor_sequence_zigzag_gb300 import build
    a, b = str(tmp_path / "plain.pt"), str(tmp_path / "checked.pt")
    _run(SCRIPT, build.build(), a)
    _run(SCRIPT, build.build(check=True), b)
    plain, checked = torch.load(a), torch.load(b)
    assert plain.keys() == checked.keys()
    for k in plain:
        assert torch.equal(plain[k], checked[k]), k


FIRST_CALL = r"""
import sys, torch
sys.path.insert(0, sys.argv[2])
from folded_tensor_sequence_zigzag_gb300 import tsp
tsp.load(sys.argv[1])
tsp.zigzag_permute(torch.zeros(8, 4, device="cuda"), 2)       # (the library's own first call)
x = torch.randn(64, 32000, device="cuda").bfloat16()
t = torch.randn(2, 150000, device="cuda")
ids = torch.randint(32000, (64,), device="cuda")
torch.cuda.synchronize()
def calls():
    f = tsp.logprobs_fwd(x, ids, top=20, entropy=True, stats=True)
    o = tsp.token_loss_fwd(x, ids, f["top_ids"], f["top_logp"], grad=True)
    d = tsp.logprobs_bwd(x, ids, f["stats"], dlogp=f["logp"])
    e = tsp.token_loss_bwd(x, f["stats"], ids, f["top_ids"], f["top_logp"])
    c = tsp.logprobs_fwd(t, top=5)
    g = tsp.token_loss_fwd(t, t_ids=c["top_ids"], t_logits=c["top_logp"], grad=True)
    return [*f.values(), *o.values(), d, e, *c.values(), *g.values()]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
want = calls()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert tsp.device_status() == tsp.TSP_OK
"""


def test_first_calls_may_be_captured():
    from folded_tensor_sequence_zigzag_gb300 import build
    _run(FIRST_CALL, build.build())


def test_calls_from_several_threads():
    """Four host threads, each on a stream of its own, with sizes that take different
    kernels: the results of one after the other."""
    import threading
    g = torch.Generator("cuda").manual_seed(11)
    jobs = []
    for S, V, K in ((300, 32000, 16), (4, 128000, 5), (1000, 1001, 7), (50, 70001, 130)):
        x = torch.randn(S, V, generator=g, device="cuda").bfloat16()
        jobs.append((x, torch.randint(V, (S,), generator=g, device="cuda"), K))

    def work(x, ids, K, stream=None):
        f = tsp.logprobs_fwd(x, ids, top=K, entropy=True, stats=True, stream=stream)
        o = tsp.token_loss_fwd(x, ids, f["top_ids"], f["top_logp"], w_ce=0.5, w_kd=0.5, grad=True, stream=stream)
        return [*f.values(), *o.values()]
    want = [work(*j) for j in jobs]
    torch.cuda.synchronize()
    got, streams = [None] * 4, [torch.cuda.Stream() for _ in jobs]

    def run(i):
        for _ in range(20):
            got[i] = work(*jobs[i], stream=streams[i])
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert tsp.device_status() == tsp.TSP_OK
