"""Log probabilities, entropy, alternatives and token losses, with their gradients,
against the definitions in 64 bits.

Tolerances.  U = 2^-24 is half an fp32 step, E2 = 2^-22 the stated error of the
hardware's 2^x.  With u_j = scale (x_j - m) and l = log sum exp(u_j):
  * a summand exp(u_j) is off by E2 and 4 U |u_j|, the few renewals of a running
    reference add as much each (8 E2 in all), and a thread's sum, the warps' and the
    CTAs' add V / 1024 + 64 roundings (a thread has two sums of n <= V / 64 terms each, up
    to 128 in one warp and 500 in four; roundings have either sign and are the smaller the
    smaller the sum still is: five standard deviations, 5 U sqrt(n / 9), are 37 U at most,
    before the warps' ten and the CTAs'); so l is off by
      dl = 8 E2 + (V / 1024 + 64) U + 8 U (E|u| + 8),     E|u| = sum_j p_j |u_j|;
  * log p_j by dl + 4 U (|u_j| + |l|);
  * the entropy, l + sum p |u|, by (1 + E|u| + 8) times that without the last term;
  * p_j in a gradient relatively by E2 + 8 U (|u_j| + |l| + 2); rounding to bf16 adds 2^-8
    of the value, a step of the smallest bf16 numbers 2^-126 (flushed results).
"""
import math

import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp

pytestmark = pytest.mark.gpu
U, E2 = 2.0 ** -24, 2.0 ** -22
INF, NAN = math.inf, math.nan
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    yield tsp.load()
    assert tsp.device_status() == tsp.TSP_OK


def rows(gen, S, V, dt, wide=0, at=0, std=3.0, ban=0.0):
    """Logits [S, V] whose rows lie V + wide apart, from the at-th element of a buffer
    that is NaN everywhere else."""
    x = torch.randn(S, V, generator=gen) * std
    if ban:
        x[torch.rand(S, V, generator=gen) < ban] = -INF
    ld = V + wide
    buf = torch.full((at + S * ld,), NAN, dtype=dt, device="cuda")
    view = buf[at:].view(S, ld)[:, :V]
    view.copy_(x.to(dt))
    return view


def untouched(view):
    """What lies around the rows is still NaN."""
    assert int(view._base.isnan().sum()) == view._base.numel() - view.numel()


def zigzag_rows(S, D):
    """Row of each position."""
    p = torch.arange(S)
    if D == 1:
        return p
    c = S // (2 * D)
    j = p // c
    return torch.where(j < D, 2 * j, 2 * (2 * D - 1 - j) + 1) * c + p % c


class Ref:
    """Everything of the logits' rows in 64 bits, in the order of positions."""

    def __init__(self, logits, D=1, scale=1.0):
        self.x = logits.cpu().double()[zigzag_rows(logits.shape[0], D)]
        self.scale, (self.S, self.V) = float(torch.tensor(scale, dtype=F32)), self.x.shape
        self.m = self.x.max(1, keepdim=True).values
        self.u = self.scale * (self.x - self.m)
        self.l = self.u.exp().sum(1, keepdim=True).log()
        self.logp = self.u - self.l
        self.p = self.logp.exp()
        self.eu = torch.where(self.p > 0, self.p * -self.u, 0.0).sum(1)
        self.entropy = self.l[:, 0] + self.eu
        self.dl = 8 * E2 + (self.V / 1024 + 64) * U + 8 * U * (self.eu + 8)
        self.d_logp = self.dl[:, None] + 4 * U * (self.u.abs() + self.l.abs())
        self.d_entropy = (1 + self.eu + 8) * self.dl
        self.rel_p = E2 + 8 * U * (self.u.abs() + self.l.abs() + 2)

    def order(self, top):
        """The top alternatives by (largest logit, lowest token); -1 past the tokens there are."""
        i = torch.sort(-(self.x + 0.0), dim=1, stable=True).indices[:, :top]
        logp = self.logp.gather(1, i)
        tol = self.d_logp.gather(1, i)
        i = torch.where(logp > -INF, i, -1)
        more = top - i.shape[1]
        if more > 0:
            i = torch.nn.functional.pad(i, (0, more), value=-1)
            logp = torch.nn.functional.pad(logp, (0, more), value=-INF)
            tol = torch.nn.functional.pad(tol, (0, more))
        return i, logp, tol


def near(got, want, tol, what=""):
    got = got.detach().cpu().double()
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), what
    assert torch.equal(got.isnan(), want.isnan()), what
    off = (got - want).abs()[fine] - tol.expand_as(want)[fine]
    assert off.numel() == 0 or off.max() <= 0, f"{what}: {off.max():.3e} past the tolerance"


def as_rows(positions, D):
    """[S, ...] in the order of positions as rows."""
    out = torch.empty_like(positions)
    out[zigzag_rows(positions.shape[0], D)] = positions
    return out


SHAPES = [  # S, V, D, wide, at
    (1, 1, 1, 0, 0), (3, 2, 1, 0, 1), (5, 7, 1, 0, 0), (4, 8, 2, 0, 0), (6, 9, 1, 4, 3), (2, 15, 1, 1, 0),
    (16, 17, 4, 0, 5), (7, 31, 1, 0, 0), (64, 100, 8, 3, 0), (33, 1000, 1, 0, 2), (12, 2049, 3, 0, 0),
    (5, 4097, 1, 8, 0), (8, 32000, 2, 0, 0), (3, 50257, 1, 0, 1), (1, 128000, 1, 0, 0), (2, 131071, 1, 1, 7),
    (1, 300001, 1, 0, 0)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("S,V,D,wide,at", SHAPES)
def test_logprobs_fwd(S, V, D, wide, at, dt):
    gen = torch.Generator().manual_seed(V + S)
    scale = 0.7
    x = rows(gen, S, V, dt, wide, at)
    ids = torch.randint(0, V, (S,), generator=gen)
    top = min(V + 2, 20)
    r = Ref(x, D, scale)
    got = tsp.logprobs_fwd(x, ids.cuda(), D=D, scale=scale, top=top, entropy=True, stats=True)
    one = torch.arange(S)
    near(got["logp"], r.logp[one, ids], r.d_logp[one, ids], "logp")
    near(got["entropy"], r.entropy, r.d_entropy, "entropy")
    assert torch.equal(got["stats"][:, 0].cpu().double(), r.m[:, 0])
    near(got["stats"][:, 1], r.l[:, 0], r.dl + 2 * U * r.l[:, 0].abs(), "l")
    i, logp, tol = r.order(top)
    assert torch.equal(got["top_ids"].cpu().long(), i)
    near(got["top_logp"], logp, tol, "top_logp")
    # each result by itself, int32 ids (other kernels, which add up in other orders): held to
    # the definition in the same way
    some = tsp.logprobs_fwd(x, ids.int().cuda(), D=D, scale=scale)
    near(some["logp"], r.logp[one, ids], r.d_logp[one, ids], "logp alone")
    some = tsp.logprobs_fwd(x, D=D, scale=scale, entropy=True)
    near(some["entropy"], r.entropy, r.d_entropy, "entropy alone")
    some = tsp.logprobs_fwd(x, D=D, scale=scale, stats=True)
    near(some["stats"][:, 1], r.l[:, 0], r.dl + 2 * U * r.l[:, 0].abs(), "l alone")
    some = tsp.logprobs_fwd(x, D=D, scale=scale, top=top)
    assert torch.equal(some["top_ids"].cpu().long(), i)
    near(some["top_logp"], logp, tol, "top_logp alone")
    # once more: the same bits
    again = tsp.logprobs_fwd(x, ids.cuda(), D=D, scale=scale, top=top, entropy=True, stats=True)
    assert all(torch.equal(again[k], got[k]) for k in got)


def grad_tolerance(r, weight, adds, dt):
    """Of p_j * weight_j (each part's magnitude) + adds."""
    t = r.p * weight * (r.rel_p + 8 * U) + 4 * U * adds.abs()
    value = r.p * weight + adds.abs()
    return t * 1.01 + (2.0 ** -8 * value if dt == BF else 2 * U * value) + 2.0 ** -125


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("what", ["logp", "entropy", "both"])
@pytest.mark.parametrize("S,V,D,wide,at", SHAPES)
def test_logprobs_bwd(S, V, D, wide, at, what, dt):
    gen = torch.Generator().manual_seed(V + S + 1)
    scale = 1.3
    x = rows(gen, S, V, dt, wide, at)
    ids = torch.randint(0, V, (S,), generator=gen)
    ids[::5] = -1 if S > 5 else ids[::5]
    r = Ref(x, D, scale)
    dl = torch.randn(S, generator=gen) if what != "entropy" else torch.zeros(S)
    de = torch.randn(S, generator=gen) if what != "logp" else torch.zeros(S)
    fwd = tsp.logprobs_fwd(x, ids.cuda(), D=D, scale=scale, entropy=True, stats=True)
    kw = dict(D=D, scale=scale)
    if what != "entropy":
        kw["dlogp"] = dl.cuda()
    if what != "logp":
        kw.update(entropy=fwd["entropy"], dentropy=de.cuda())
    before = x.clone()
    got = tsp.logprobs_bwd(x, ids.cuda(), fwd["stats"], **kw)
    assert torch.equal(x, before) and got.stride() == x.stride() or S == 1
    live = (ids >= 0).double()
    dl, de = dl.double() * live, de.double() * live
    adds = torch.zeros_like(r.p)
    adds[torch.arange(S), ids.clamp(min=0)] = r.scale * dl
    lh = torch.where(r.p > 0, r.logp + r.entropy[:, None], 0.0)
    want = adds - r.scale * r.p * (dl[:, None] + de[:, None] * lh)
    size = r.scale * (dl.abs()[:, None] + de.abs()[:, None] * (lh.abs() + r.entropy[:, None]))
    # the statistics are themselves off by dl, the entropy by d_entropy
    slack = r.p * (size * r.dl[:, None] + r.scale * de.abs()[:, None] * (r.d_entropy + r.dl)[:, None] * 2)
    tol = grad_tolerance(r, size, adds, dt) + slack * 1.01
    near(got, as_rows(want, D), as_rows(tol, D), "dlogits")
    # by elements (rows that lie otherwise) and in place: the same bits
    other = torch.full((1 + S * (V + 5),), NAN, dtype=dt, device="cuda")[1:].view(S, V + 5)[:, :V]
    assert torch.equal(tsp.logprobs_bwd(x, ids.cuda(), fwd["stats"], out=other, **kw), got)
    assert torch.equal(tsp.logprobs_bwd(x, ids.cuda(), fwd["stats"], out=x, **kw), got)
    assert torch.equal(x, got)
    untouched(x)


def teacher_lists(gen, S, V, K, dt, short=True):
    ids = torch.stack([torch.randperm(V, generator=gen)[:K] if K <= V else torch.randint(0, V, (K,), generator=gen)
                       for _ in range(S)]).int()
    y = (torch.randn(S, K, generator=gen) * 2).to(dt)
    if short:
        ids[torch.rand(S, K, generator=gen) < 0.2] = -1
        y[torch.rand(S, K, generator=gen) < 0.1] = -INF
        ids[0] = -1                                   # a position without entries
    if K > 2:
        ids[-1, 1] = ids[-1, 2]                       # a token listed twice
    return ids, y


def loss_reference(r, ids, w_ce, t_ids, t_y, w_kd, t_scale):
    """(loss, its tolerance, q on the row's tokens, weight of p) per position."""
    S, V = r.p.shape
    live = torch.ones(S, dtype=torch.bool) if ids is None else ids >= 0
    loss, tol = torch.zeros(S, dtype=torch.float64), torch.zeros(S, dtype=torch.float64)
    adds, weight = torch.zeros(S, V, dtype=torch.float64), torch.zeros(S, dtype=torch.float64)
    one = torch.arange(S)
    if ids is not None and w_ce:
        t = ids.clamp(min=0)
        loss -= w_ce * r.logp[one, t]
        tol += abs(w_ce) * r.d_logp[one, t] + 2 * U * abs(w_ce) * r.logp[one, t].abs()
        adds[one, t] -= w_ce
        weight += w_ce
    if t_ids is not None and w_kd:
        ts = float(torch.tensor(t_scale, dtype=F32))
        there = (t_ids >= 0) & (t_y > -INF)
        any_ = there.any(1)
        z = torch.where(there, t_y.double() * ts, -INF)
        q = torch.where(any_[:, None], torch.softmax(z, 1), 0.0).nan_to_num(0.0)
        at = t_ids.long().clamp(min=0)
        logp, dlp = r.logp.gather(1, at), r.d_logp.gather(1, at)
        logq = torch.where(q > 0, q.log(), 0.0)
        kl = torch.where(q > 0, q * (logq - logp), 0.0).sum(1)
        # log q and its weights: exp of t_scale (y - max), within 300 U of a list of 256
        size = torch.where(q > 0, q * (logq.abs() + logp.abs() + 1 + (z - z.max(1, keepdim=True).values).abs().nan_to_num(0.0)), 0.0).sum(1)
        loss += w_kd * kl
        tol += abs(w_kd) * (torch.where(q > 0, q * dlp, 0.0).sum(1) + 320 * U * size)
        adds.scatter_add_(1, at, -w_kd * q)
        weight += w_kd * any_
    loss = torch.where(live, loss, 0.0)
    return loss, tol + 4 * U * loss.abs(), adds * live[:, None], weight * live


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K,w_ce,w_kd", [(0, 1.0, 0.0), (1, 0.0, 1.0), (8, 0.3, 0.7), (64, 0.0, 2.0), (256, 0.5, -0.25)])
@pytest.mark.parametrize("S,V,D,wide,at", SHAPES)
def test_token_loss(S, V, D, wide, at, K, w_ce, w_kd, dt):
    gen = torch.Generator().manual_seed(V + S + 2 + K)
    scale, t_scale = 0.5, 1.5
    x = rows(gen, S, V, dt, wide, at)
    ids = torch.randint(0, V, (S,), generator=gen) if w_ce or K == 1 else None
    if ids is not None and S > 5:
        ids[::5] = -1
    t_ids, t_y = teacher_lists(gen, S, V, K, dt if K == 8 else F32) if K else (None, None)
    dloss = torch.rand(S, generator=gen) if K != 64 else None
    r = Ref(x, D, scale)
    loss, tol, adds, weight = loss_reference(r, ids, w_ce, t_ids, t_y, w_kd, t_scale)
    c = lambda t: None if t is None else t.cuda()
    kw = dict(ids=c(ids), t_ids=c(t_ids), t_logits=c(t_y), w_ce=w_ce, w_kd=w_kd, D=D, scale=scale, t_scale=t_scale)
    got = tsp.token_loss_fwd(x, stats=True, **kw)
    near(got["loss"], loss, tol, "loss")
    want_stats = tsp.logprobs_fwd(x, c(ids), D=D, scale=scale, stats=True)["stats"]
    # (a long list takes more threads, which add the row up in another order: each is
    # within dl of the definition, so they are within 2 dl and a rounding of each other)
    assert torch.equal(got["stats"][:, 0], want_stats[:, 0])
    near(got["stats"][:, 1], want_stats[:, 1].cpu().double(),
         torch.where(want_stats[:, 1].cpu() == -INF, 0.0, 2 * r.dl + 2 * U * r.l[:, 0].abs()), "l")
    up = r.scale * (torch.ones(S, dtype=torch.float64) if dloss is None else dloss.double())
    want = up[:, None] * (weight[:, None] * r.p + adds)
    size = (up * weight.abs())[:, None].expand_as(r.p)
    parts = up[:, None] * adds.abs()                 # q is off by 320 U
    gtol = grad_tolerance(r, size, parts, dt) + 320 * U * parts + 1.01 * r.p * size * r.dl[:, None]
    before = x.clone()
    d = tsp.token_loss_bwd(x, got["stats"], dloss=c(dloss), **kw)
    near(d, as_rows(want, D), as_rows(gtol, D), "gradient")
    # loss and gradient in one pass
    both = tsp.token_loss_fwd(x, stats=True, grad=True, dloss=c(dloss), **kw)
    near(both["loss"], loss, tol, "loss (with gradient)")
    near(both["stats"][:, 1], got["stats"][:, 1].cpu().double(), 2 * r.dl + 2 * U * r.l[:, 0].abs(), "l (with gradient)")
    near(both["dlogits"], as_rows(want, D), as_rows(gtol, D), "gradient (one pass)")
    assert torch.equal(x, before)
    # rows that lie otherwise, and in place: the same bits
    other = torch.full((1 + S * (V + 5),), NAN, dtype=dt, device="cuda")[1:].view(S, V + 5)[:, :V]
    assert torch.equal(tsp.token_loss_bwd(x, got["stats"], dloss=c(dloss), out=other, **kw), d)
    other = torch.full((1 + S * (V + 5),), NAN, dtype=dt, device="cuda")[1:].view(S, V + 5)[:, :V]
    near(tsp.token_loss_fwd(x, dloss=c(dloss), dlogits=other, **kw)["dlogits"], as_rows(want, D), as_rows(gtol, D), "elsewhere")
    tsp.token_loss_fwd(x, dloss=c(dloss), dlogits=x, **kw)
    assert torch.equal(x, both["dlogits"])
    x.copy_(before)
    tsp.token_loss_bwd(x, got["stats"], dloss=c(dloss), out=x, **kw)
    assert torch.equal(x, d)
    untouched(x)
    untouched(other)


def special(V, dt):
    """Rows that a language model's logits can be, and some that they cannot."""
    low = torch.finfo(dt).min
    gen = torch.Generator().manual_seed(V)
    base = torch.randn(V, generator=gen).to(dt).float()
    out = {"ordinary": base.clone()}
    out["nothing left"] = torch.full((V,), -INF)
    out["one left"] = torch.full((V,), -INF)
    out["one left"][V // 2] = 3.0
    out["lowest"] = torch.full((V,), low)
    out["lowest and nothing"] = torch.full((V,), -INF)
    out["lowest and nothing"][::3] = low
    out["masked by lowest"] = base.clone()
    out["masked by lowest"][1::2] = low
    out["last left"] = torch.full((V,), -INF)
    out["last left"][-1] = -7.0
    out["equal"] = torch.zeros(V)
    out["zeros of both signs"] = torch.zeros(V)
    out["zeros of both signs"][::2] = -0.0
    out["rising"] = torch.arange(V).float() / 16
    out["falling"] = -torch.arange(V).float() / 16
    out["huge"] = base * 1e30
    out["large"] = base + 30000.0
    out["far apart"] = base * 400
    out["one thread's"] = base.clone()
    out["one thread's"][::8 * 512] += 40.0           # the largest logits all with the same few threads
    for n in (128, 256, 512):
        out[f"every {n}th unit"] = base.clone()
        out[f"every {n}th unit"].view(-1)[torch.arange(V) // 8 % n == 3] += 20.0
        out[f"every {n}th unit of fp32"] = base.clone()
        out[f"every {n}th unit of fp32"][torch.arange(V) // 4 % n == 3] += 20.0
    return {k: v.to(dt) for k, v in out.items()}


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [1, 5, 40, 1000, 33001, 130000])
@pytest.mark.parametrize("top", [1, 5, 200])
def test_special_rows(V, top, dt):
    named = special(V, dt)
    x = torch.stack(list(named.values())).cuda()
    S = x.shape[0]
    ids = torch.full((S,), V - 1)
    for scale in (1.0, 0.25):
        r = Ref(x, 1, scale)
        dead = (r.x == -INF).all(1)
        none = lambda v, to: torch.where(dead, torch.tensor(to, dtype=torch.float64), v)
        got = tsp.logprobs_fwd(x, ids.cuda(), scale=scale, top=top, entropy=True, stats=True)
        near(got["stats"][:, 0], none(r.m[:, 0], 0.0), torch.tensor(0.0), "m")
        near(got["stats"][:, 1], none(r.l[:, 0], -INF), r.dl.nan_to_num(0.0) + 2 * U * r.l[:, 0].abs().nan_to_num(0.0), "l")
        near(got["logp"], none(r.logp[:, V - 1], -INF), r.d_logp[:, V - 1].nan_to_num(0.0, posinf=0.0), "logp")
        near(got["entropy"], none(r.entropy, 0.0), r.d_entropy.nan_to_num(0.0), "entropy")
        r.logp[dead] = -INF
        i, logp, tol = r.order(top)
        for k, name in enumerate(named):
            assert torch.equal(got["top_ids"][k].cpu().long(), i[k]), name
        near(got["top_logp"], logp, tol.nan_to_num(0.0, posinf=0.0), "top_logp")
        # gradients: zero in a row of nothing, and at every token that is left out
        one = torch.ones(S, device="cuda")
        d = tsp.logprobs_bwd(x, ids.cuda(), got["stats"], dlogp=one, entropy=got["entropy"], dentropy=one, scale=scale)
        assert d.isfinite().all() and not d[dead].any()
        out_of = (x == -INF)
        out_of[:, V - 1] = False
        assert not d[out_of].any()
        fine = ~dead & r.u[:, V - 1].isfinite()
        lh = torch.where(r.p > 0, r.logp + r.entropy[:, None], 0.0)
        want = -r.scale * r.p * (1 + lh)
        want[:, V - 1] += r.scale
        size = r.scale * (1 + lh.abs() + r.entropy[:, None])
        tol = grad_tolerance(r, size, r.scale * torch.ones_like(size), dt) + r.p * (size * r.dl[:, None] + 2 * r.scale * (r.d_entropy + r.dl)[:, None])
        near(d[fine.cuda()], want[fine], tol[fine].nan_to_num(0.0), "gradient")
        loss = tsp.token_loss_fwd(x, ids.cuda(), scale=scale, grad=True)
        near(loss["loss"], none(-r.logp[:, V - 1], INF), r.d_logp[:, V - 1].nan_to_num(0.0, posinf=0.0) * 1.01, "loss")
        assert loss["dlogits"].isfinite().all() and not loss["dlogits"][dead].any()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [9, 5003, 130000])
def test_rows_without_a_distribution(V, dt):
    """NaN or +inf anywhere: NaN results and gradients in that row alone, no alternatives."""
    gen = torch.Generator().manual_seed(3)
    x = rows(gen, 7, V, dt)
    bad = [1, 3, 5, 6]
    x[1, 0], x[3, V // 2], x[5, V - 1] = NAN, INF, INF
    x[6] = -INF
    x[6, V // 3] = NAN
    good = [0, 2, 4]
    ids = torch.full((7,), 2, device="cuda")
    t_ids = torch.arange(5, dtype=torch.int32, device="cuda").repeat(7, 1)
    t_y = torch.randn(7, 5, generator=gen).cuda()
    got = tsp.logprobs_fwd(x, ids, top=4, entropy=True, stats=True)
    y = x.clone()
    y[bad] = 0.0
    alone = tsp.logprobs_fwd(y, ids, top=4, entropy=True, stats=True)
    for k in alone:
        assert torch.equal(got[k][good], alone[k][good]), k
    assert (got["top_ids"][bad] == -1).all()
    for k in ("logp", "entropy", "top_logp"):
        assert got[k][bad].isnan().all(), k
    d = tsp.logprobs_bwd(x, ids, got["stats"], dlogp=ids.float())
    assert d[bad].isnan().all() and d[good].isfinite().all()
    both = tsp.token_loss_fwd(x, ids, t_ids, t_y, grad=True)
    assert both["loss"][bad].isnan().all() and both["loss"][good].isfinite().all()
    assert both["dlogits"][bad].isnan().all() and both["dlogits"][good].isfinite().all()
    # padding is not looked at
    ids[bad] = -1
    got = tsp.logprobs_fwd(x, ids, top=4, entropy=True, stats=True)
    assert not got["logp"][bad].any() and not got["entropy"][bad].any() and (got["top_ids"][bad] == -1).all()
    assert (got["top_logp"][bad] == -INF).all() and (got["stats"][bad].cpu() == torch.tensor([0.0, -INF])).all()
    both = tsp.token_loss_fwd(x, ids, t_ids, t_y, grad=True)
    assert not both["loss"][bad].any() and not both["dlogits"][bad].any()


def test_teachers_that_say_little():
    """Lists with nothing in them, teachers of one token, teachers with NaN and +inf,
    huge logits, and a model that has left out what the teacher lists."""
    gen = torch.Generator().manual_seed(4)
    V, S, K = 1001, 8, 6
    x = rows(gen, S, V, F32)
    t_ids = torch.stack([torch.randperm(V, generator=gen)[:K] for _ in range(S)]).int()
    y = torch.randn(S, K, generator=gen)
    t_ids[0] = -1
    y[1] = -INF
    t_ids[2, 1:] = -1
    y[3, 2] = NAN
    y[4, 2] = INF
    y[5] = torch.tensor([3.4e38, -3.4e38, 3.4e38, -INF, 0.0, 1e30])
    y[7] = torch.finfo(F32).min
    x[6, t_ids[6, 0].long()] = -INF
    kw = dict(t_ids=t_ids.cuda(), t_logits=y.cuda(), t_scale=2.0)
    got = tsp.token_loss_fwd(x, stats=True, **kw)
    both = tsp.token_loss_fwd(x, grad=True, **kw)
    d = tsp.token_loss_bwd(x, got["stats"], **kw)
    r = Ref(x)
    assert not got["loss"][:2].any() and not d[:2].any()
    near(got["loss"][2], -r.logp[2, t_ids[2, 0].long()], r.d_logp[2, t_ids[2, 0].long()] * 1.1, "one token")
    for k in (3, 4):
        assert got["loss"][k].isnan() and both["loss"][k].isnan() and d[k, t_ids[k].long()].isnan().any()
    a, b = t_ids[5, 0].long(), t_ids[5, 2].long()
    near(got["loss"][5], math.log(0.5) - (r.logp[5, a] + r.logp[5, b]) / 2, r.d_logp[5].max() * 1.1, "two tokens")
    assert got["loss"][6] == INF and both["loss"][6] == INF and d[6].isfinite().all()
    want = r.p[7].clone()
    want[t_ids[7].long()] -= 1 / K
    near(d[7], want, r.rel_p[7] * r.p[7] + r.p[7] * r.dl[7] + 40 * U * want.abs(), "all lowest")
    same = ~d.isnan()
    near(both["dlogits"][same], d[same].cpu().double(), 16 * (E2 + 30 * U) * d[same].cpu().double().abs() + 1e-9, "one pass")


def test_ids_past_the_logits():
    x = torch.randn(6, 50, device="cuda")
    ids = torch.tensor([1, 50, 2, 1 << 40, -5, 3], device="cuda")
    got = tsp.logprobs_fwd(x, ids, top=3, entropy=True, stats=True)
    assert tsp.device_status() == tsp.TSP_ERR_RANGE
    pad = torch.tensor([1, -1, 2, -1, -1, 3], device="cuda")
    want = tsp.logprobs_fwd(x, pad, top=3, entropy=True, stats=True)
    assert all(torch.equal(got[k], want[k]) for k in got)
    assert tsp.device_status() == tsp.TSP_OK
    d = tsp.logprobs_bwd(x, ids, got["stats"], dlogp=got["logp"])
    assert tsp.device_status() == tsp.TSP_ERR_RANGE
    assert torch.equal(d, tsp.logprobs_bwd(x, pad, got["stats"], dlogp=got["logp"]))
    t_ids = torch.tensor([[3, 50, 7]] * 6, dtype=torch.int32, device="cuda")
    none = torch.tensor([[3, -1, 7]] * 6, dtype=torch.int32, device="cuda")
    y = torch.randn(6, 3, device="cuda")
    for grad in (False, True):
        a = tsp.token_loss_fwd(x, t_ids=t_ids, t_logits=y, grad=grad)
        assert tsp.device_status() == tsp.TSP_ERR_RANGE
        b = tsp.token_loss_fwd(x, t_ids=none, t_logits=y, grad=grad)
        assert all(torch.equal(a[k], b[k]) for k in a)
    assert tsp.device_status() == tsp.TSP_OK


@pytest.mark.parametrize("S,V,dt", [(3000, 300, BF), (700, 32000, BF), (400, 50257, F32), (200, 150001, BF), (40, 700001, BF), (2, 2000000, F32)])
def test_many_rows_and_long_ones(S, V, dt):
    """More rows than the GPU holds at once, and rows longer than its shared memory:
    rows taken at random against the definitions, all of them against each other."""
    g = torch.Generator("cuda").manual_seed(5)
    x = (torch.randn(S, V, generator=g, device="cuda") * 2).to(dt)
    ids = torch.randint(V, (S,), generator=g, device="cuda")
    K = 50
    t_ids = torch.randint(V, (S, K), generator=g, device="cuda").int()
    t_y = torch.randn(S, K, generator=g, device="cuda")
    some = sorted({0, 1, S // 2, S - 1})
    got = tsp.logprobs_fwd(x, ids, top=30, entropy=True, stats=True)
    r = Ref(x[some])
    pick, one = ids[some].cpu(), torch.arange(len(some))
    near(got["logp"][some], r.logp[one, pick], r.d_logp[one, pick], "logp")
    near(got["entropy"][some], r.entropy, r.d_entropy, "entropy")
    i, logp, tol = r.order(30)
    assert torch.equal(got["top_ids"][some].cpu().long(), i)
    kw = dict(ids=ids, t_ids=t_ids, t_logits=t_y, w_ce=0.5, w_kd=0.5)
    loss, ltol, adds, weight = loss_reference(r, pick, 0.5, t_ids[some].cpu(), t_y[some].cpu(), 0.5, 1.0)
    both = tsp.token_loss_fwd(x, stats=True, grad=True, **kw)
    near(both["loss"][some], loss, ltol, "loss")
    want = weight[:, None] * r.p + adds
    gtol = grad_tolerance(r, weight[:, None].expand_as(r.p), adds, dt) + 320 * U * adds.abs() + 1.01 * r.p * r.dl[:, None]
    near(both["dlogits"][some], want, gtol, "gradient")
    # a row's gradient adds up to nothing
    total = both["dlogits"].double().sum(1).abs()
    assert total.max() <= (V * 2.0 ** -24 + 2) * (2.0 ** -8 if dt == BF else 2.0 ** -16)
    d = tsp.token_loss_bwd(x, both["stats"], **kw)
    mag = both["dlogits"].float().abs()
    assert ((d.float() - both["dlogits"].float()).abs() <= mag * (2.0 ** -6 if dt == BF else 2.0 ** -15) + 1e-12).all()
    del mag, d
    again = tsp.token_loss_fwd(x, stats=True, grad=True, **kw)
    assert all(torch.equal(again[k], both[k]) for k in both)


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31."""
    V, far = 4099, (1 << 30) + 8
    buf = torch.empty(3 * far + V, dtype=BF, device="cuda")
    x = torch.as_strided(buf, (4, V), (far, 1))
    gen = torch.Generator().manual_seed(6)
    x.copy_(torch.randn(4, V, generator=gen).to(BF))
    # (rows that lie as far from 16-byte boundaries are added up in the same order)
    dense, ids = torch.empty(4, V + 5, dtype=BF, device="cuda")[:, :V], torch.arange(4, device="cuda") + V - 4
    dense.copy_(x)
    a, b = (tsp.logprobs_fwd(t, ids, top=9, entropy=True, stats=True) for t in (x, dense))
    assert all(torch.equal(a[k], b[k]) for k in a)
    up = torch.ones(4, device="cuda")
    want = tsp.logprobs_bwd(dense, ids, a["stats"], dlogp=up)
    t_ids, y = a["top_ids"], a["top_logp"]
    both = tsp.token_loss_fwd(dense, ids, t_ids, y, grad=True)
    assert torch.equal(tsp.token_loss_fwd(x, ids, t_ids, y, dlogits=x)["loss"], both["loss"])
    near(x.contiguous(), both["dlogits"].cpu().double(), 2.0 ** -7 * both["dlogits"].cpu().double().abs() + 1e-9, "one pass")
    x.copy_(dense)
    tsp.logprobs_bwd(x, ids, a["stats"], dlogp=up, out=x)
    assert torch.equal(x.contiguous(), want)


@pytest.mark.parametrize("V", [37, 700])
def test_gradients_against_differences(V):
    """Central differences of the calls themselves along random directions: off by
    h^2 / 6 of a third derivative below 8 and by the results' rounding over h."""
    gen = torch.Generator().manual_seed(7)
    S, K, h = 4, 5, 2.0 ** -5
    x = rows(gen, S, V, F32, std=1.0)
    ids = torch.randint(0, V, (S,), generator=gen).cuda()
    t_ids = torch.stack([torch.randperm(V, generator=gen)[:K] for _ in range(S)]).int().cuda()
    y = torch.randn(S, K, generator=gen).cuda()
    up, ue = torch.rand(S, generator=gen).cuda(), torch.rand(S, generator=gen).cuda()
    kw = dict(t_ids=t_ids, t_logits=y, w_ce=0.4, w_kd=0.6, scale=0.8)

    def score(z):
        o = tsp.logprobs_fwd(z, ids, entropy=True, scale=0.8)
        return (o["logp"].double() * up.double() + o["entropy"].double() * ue.double()).sum().item()

    def loss(z):
        return (tsp.token_loss_fwd(z, ids, **kw)["loss"].double() * up.double()).sum().item()
    f = tsp.logprobs_fwd(x, ids, entropy=True, stats=True, scale=0.8)
    d1 = tsp.logprobs_bwd(x, ids, f["stats"], dlogp=up, entropy=f["entropy"], dentropy=ue, scale=0.8)
    d2 = tsp.token_loss_fwd(x, ids, grad=True, dloss=up, **kw)["dlogits"]
    for _ in range(4):
        v = torch.sign(torch.randn(S, V, generator=gen)).cuda()
        for fn, d in ((score, d1), (loss, d2)):
            diff = (fn(x + h * v) - fn(x - h * v)) / (2 * h)
            assert abs(diff - (d.double() * v).sum().item()) <= S * (h * h / 6 * 8 + 2 * 20 * U * math.log(V) / h)


def test_streams_and_graphs():
    """A call on another stream than the current one; two streams at once; a captured
    forward, loss and gradient replayed on new values."""
    g = torch.Generator("cuda").manual_seed(8)
    S, V, K = 64, 32000, 16
    xs = [(torch.randn(S, V, generator=g, device="cuda") * 2).to(BF) for _ in range(4)]
    ids = torch.randint(V, (S,), generator=g, device="cuda")

    def chain(x, stream=None):
        f = tsp.logprobs_fwd(x, ids, top=K, entropy=True, stats=True, stream=stream)
        d = tsp.logprobs_bwd(x, ids, f["stats"], dlogp=f["logp"], entropy=f["entropy"], dentropy=f["logp"], stream=stream)
        o = tsp.token_loss_fwd(x, ids, f["top_ids"], f["top_logp"], w_ce=0.5, w_kd=0.5, grad=True, stream=stream)
        return {**f, "d": d, **{"o" + k: v for k, v in o.items()}}
    want = [chain(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [chain(x, streams[i % 2]) for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(a[k], b[k]) for k in b)
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(x)
    for i in (1, 3, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[i][k]) for k in out)


def test_a_model_is_its_own_teacher():
    """Alternatives as a teacher's list: over every token the divergence is nothing and
    so is its gradient; a list cut short is as the definition says."""
    gen = torch.Generator().manual_seed(9)
    S, V = 16, 200
    x = rows(gen, S, V, F32, ban=0.3)
    f = tsp.logprobs_fwd(x, top=V)
    o = tsp.token_loss_fwd(x, t_ids=f["top_ids"], t_logits=f["top_logp"], grad=True)
    r = Ref(x)
    assert (o["loss"].abs().cpu() <= 2 * r.d_logp.nan_to_num(0.0, posinf=0.0).max(1).values + 700 * U).all()
    near(o["dlogits"], torch.zeros(S, V, dtype=torch.float64), 2 * r.p * (r.rel_p.nan_to_num(0.0, posinf=0.0) + r.dl[:, None] + 320 * U), "gradient")
    f = tsp.logprobs_fwd(x, top=7)
    o = tsp.token_loss_fwd(x, t_ids=f["top_ids"], t_logits=f["top_logp"])
    i, logp, _ = r.order(7)
    want = -logp.exp().sum(1).log()                  # KL(p restricted to the list || p)
    assert ((o["loss"].cpu().double() - want).abs() <= 2 * r.dl + 700 * U).all()


@pytest.mark.parametrize("K", [40, 256])
@pytest.mark.parametrize("V", [64, 320])
def test_positions_with_and_without_entries_by_turns(V, K):
    """Many short rows one after the other: none takes the neighbour's list.  The rows are
    whole lines, so that every position comes out as it does alone with its own kind."""
    S = 20000
    x = torch.randn(S, V, device="cuda", generator=torch.Generator("cuda").manual_seed(V)).bfloat16()
    gen = torch.Generator().manual_seed(K)
    t_ids, t_y = torch.randint(0, V, (S, K), generator=gen).int(), torch.randn(S, K, generator=gen)
    t_ids[::2] = -1
    t_ids, t_y = t_ids.cuda(), t_y.cuda()
    for grad in (False, True):
        got = tsp.token_loss_fwd(x, None, t_ids, t_y, grad=grad)
        assert not got["loss"][::2].any() and got["loss"][1::2].all()
        alone = tsp.token_loss_fwd(x[1::2].contiguous(), None, t_ids[1::2].contiguous(), t_y[1::2].contiguous(), grad=grad)
        assert torch.equal(got["loss"][1::2], alone["loss"])
        if grad:
            assert not got["dlogits"][::2].any() and torch.equal(got["dlogits"][1::2], alone["dlogits"])


@pytest.mark.parametrize("S,V,dt", [(600, 130000, BF), (600, 70000, F32), (3, 40000, BF)])
def test_in_place_over_parts_of_a_row(S, V, dt):
    """A gradient that takes the logits' place: the given token's logit is read by one CTA
    and written over by another."""
    gen = torch.Generator("cuda").manual_seed(S)
    x = torch.randn(S, V, device="cuda", generator=gen).to(dt)
    t_ids = torch.randint(0, V, (S, 16), generator=gen, device="cuda").int()
    t_y = torch.randn(S, 16, generator=gen, device="cuda")
    for kw in (dict(), dict(t_ids=t_ids, t_logits=t_y)):
        for k in range(4):
            ids = torch.randint(0, V, (S,), generator=gen, device="cuda")
            want = tsp.token_loss_fwd(x, ids, grad=True, **kw)
            y = x.clone()
            got = tsp.token_loss_fwd(y, ids, dlogits=y, **kw)
            assert torch.equal(got["loss"], want["loss"]) and torch.equal(y, want["dlogits"])


@pytest.mark.parametrize("dt", [BF, F32])
def test_last_positions_of_a_batch(dt):
    """Rows a whole sequence apart: the gradient takes their own room, not the batch's."""
    gen = torch.Generator().manual_seed(3)
    B, L, V = 5, 300, 1003
    x = (torch.randn(B, L, V, generator=gen) * 2).to(dt).cuda()[:, -1]
    ids = torch.randint(0, V, (B,), generator=gen).cuda()
    got = tsp.token_loss_fwd(x, ids, grad=True, stats=True)
    assert got["dlogits"]._base is None or got["dlogits"]._base.numel() < (B + 1) * (V + 64)
    r = Ref(x)
    loss, tol, adds, weight = loss_reference(r, ids.cpu(), 1.0, None, None, 0.0, 1.0)
    near(got["loss"], loss, tol, "loss")
    size = torch.ones_like(r.p)
    gtol = grad_tolerance(r, size, adds.abs(), dt) + 1.01 * r.p * r.dl[:, None]
    near(got["dlogits"], r.p + adds, gtol, "gradient (one pass)")
    near(tsp.token_loss_bwd(x, got["stats"], ids), r.p + adds, gtol, "gradient")
    one = tsp.token_loss_fwd(x[:1], ids[:1], grad=True)
    assert one["dlogits"].is_contiguous()


# as many rows as there are CTAs of one or two warps on the GPU, which take short rows then
MANY = [(3700, 1, 1, 0, 0), (4000, 9, 4, 0, 3), (3800, 257, 1, 5, 1), (4096, 1000, 8, 0, 0), (3700, 2047, 1, 1, 7), (1900, 5003, 1, 0, 0), (1840, 8192, 2, 8, 0)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("S,V,D,wide,at", MANY)
def test_many_short_rows(S, V, D, wide, at, dt):
    test_logprobs_fwd(S, V, D, wide, at, dt)
    test_logprobs_bwd(S, V, D, wide, at, "both" if S % 3 else "logp", dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K,w_ce,w_kd", [(0, 1.0, 0.0), (3, 0.3, 0.7), (32, 0.0, 2.0), (33, 0.5, 1.0), (64, 0.5, -0.25), (65, 1.0, 1.0)])
@pytest.mark.parametrize("S,V,D,wide,at", [s for s in MANY if s[1] in (1, 9, 257, 1000, 5003)])
def test_losses_of_many_short_rows(S, V, D, wide, at, K, w_ce, w_kd, dt):
    test_token_loss(S, V, D, wide, at, K, w_ce, w_kd, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V,top", [(9, 3), (700, 1), (1003, 21), (1000, 22), (2500, 5), (2501, 64), (5003, 85), (5003, 86)])
def test_many_special_rows(V, top, dt):
    named = special(V, dt)
    one = torch.stack(list(named.values()))
    n = one.shape[0]
    R = -(-3700 // n)
    x = one.cuda().repeat(R, 1)
    ids = torch.full((n * R,), V - 1, device="cuda")
    r = Ref(one)
    dead = (r.x == -INF).all(1)
    none = lambda v, to: torch.where(dead, torch.tensor(to, dtype=torch.float64), v).repeat(R)
    got = tsp.logprobs_fwd(x, ids, top=top, entropy=True, stats=True)
    near(got["stats"][:, 0], none(r.m[:, 0], 0.0), torch.tensor(0.0), "m")
    near(got["stats"][:, 1], none(r.l[:, 0], -INF), (r.dl.nan_to_num(0.0) + 2 * U * r.l[:, 0].abs().nan_to_num(0.0)).repeat(R), "l")
    near(got["logp"], none(r.logp[:, V - 1], -INF), r.d_logp[:, V - 1].nan_to_num(0.0, posinf=0.0).repeat(R), "logp")
    near(got["entropy"], none(r.entropy, 0.0), r.d_entropy.nan_to_num(0.0).repeat(R), "entropy")
    r.logp[dead] = -INF
    i, logp, tol = r.order(top)
    off = (got["top_ids"].cpu().long().view(R, n, top) != i).any(2).any(0)
    assert not off.any(), [name for name, o in zip(named, off) if o]
    near(got["top_logp"], logp.repeat(R, 1), tol.nan_to_num(0.0, posinf=0.0).repeat(R, 1), "top_logp")
    loss = tsp.token_loss_fwd(x, ids, grad=True)
    near(loss["loss"], none(-r.logp[:, V - 1], INF), r.d_logp[:, V - 1].nan_to_num(0.0, posinf=0.0).repeat(R) * 1.01, "loss")
    assert loss["dlogits"].isfinite().all() and not loss["dlogits"].view(R, n, V)[:, dead.cuda()].any()
