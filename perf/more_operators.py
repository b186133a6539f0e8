"""Performance cases of the operators behind the block stack, on the logits of the output projection:

* ``score``   log probabilities of given tokens, with entropy and top alternatives, and their gradient;
* ``loss``    cross entropy of given tokens and distillation from a teacher's top logits: forward,
              gradient, or both in one pass.

``run`` computes a case in elementary torch operations, or with ``own`` set through the
framework's entry points.  ``exact`` gives the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
LARGEST = 8192 * 128000         # logits of the largest case
LARGEST_TOP = 4096 * 128000     # the same with alternatives


# ---------------------------------------------------------------------------- cases
def _score(**kw):
    return {**dict(kind="score", D=1, dtype="bf16", temp=1.0, ids=64, top=0, entropy=True, pad=0.0, ban=0.0, wide=0), **kw}


def _loss(kind, **kw):
    return {**dict(kind=kind, D=1, dtype="bf16", temp=1.0, ids=64, K=0, ce=1.0, kd=0.0, pad=0.0, ban=0.0, wide=0, short=False), **kw}


def listed():
    return [
        # one token answered, with five alternatives
        _score(name="answer1", S=1, V=32000, top=5, temp=0.7),
        # eight decoded tokens under a grammar that bans a third of a large vocabulary, fp32 logits
        _score(name="answer8_constrained", S=8, V=128000, dtype="fp32", top=20, ban=0.33),
        # a 16384-token prompt scored in the zigzag order of eight ranks
        _score(name="score_prompt16k", S=16384, D=8, V=32000),
        # a teacher's 64 best tokens for each position, as the distillation below reads them
        _score(name="teacher_top64", S=4096, V=128000, top=64, ids=0, entropy=False),
        # a padded batch of ragged rows: odd vocabulary, fp32, few alternatives
        _score(name="score_ragged", S=4095, V=50257, dtype="fp32", top=10, ids=32, pad=0.2),
        # gradient of a policy objective with an entropy bonus, prompt positions left out
        _score(name="policy_grad8k", kind="score_bwd", S=8192, D=4, V=32000, pad=0.3),
        # the same without the bonus on ragged fp32 rows
        _score(name="score_grad_ragged", kind="score_bwd", S=1023, V=50257, dtype="fp32", entropy=False, ids=32),
        # validation loss of a distilled model
        _loss(name="loss_eval8k", kind="loss_fwd", S=8192, V=32000, K=32, ce=0.5, kd=0.5),
        # the training loss of a 16384-token step and its gradient
        _loss(name="loss_train16k", kind="loss_train", S=16384, D=8, V=32000, pad=0.1),
        # distillation step over a large vocabulary, both terms, softened
        _loss(name="distill_train8k", kind="loss_train", S=8192, V=128000, K=64, ce=0.1, kd=0.9, temp=2.0),
        # gradient alone: rows padded to a multiple of 16 elements, teacher lists of differing lengths
        _loss(name="distill_grad_ragged", kind="loss_bwd", S=4093, V=50257, K=20, ce=0.0, kd=1.0, ids=0, wide=15, short=True),
        # a small fp32 model: all launch latency
        _loss(name="loss_tiny", kind="loss_train", S=64, D=4, V=1000, dtype="fp32", K=8, ce=0.5, kd=0.5, ids=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges: one to 16384 rows of 1000 to 160000 logits, odd sizes among them."""
    kind = rng.choice(["score", "score", "score_bwd", "loss_fwd", "loss_bwd", "loss_train", "loss_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    V = _log(rng, 1000, 160000)
    if rng.random() < 0.5:
        V = V // 64 * 64
    top = _log(rng, 1, 128) if kind == "score" and rng.random() < 0.6 else 0
    most = (LARGEST_TOP if top else LARGEST) // (2 if dtype == "fp32" else 1)
    S, D = min(_log(rng, 1, 16384), most // V), rng.choice([1, 1, 2, 4, 8])
    if S < 2 * D:
        D = 1
    if D > 1:
        S = S // (2 * D) * 2 * D
    c = dict(S=S, V=V, D=D, dtype=dtype, temp=rng.choice([1.0, 1.0, 0.7, 2.0]), ids=rng.choice([32, 64]), pad=rng.choice([0.0, 0.0, 0.3]),
             ban=rng.choice([0.0, 0.0, 0.3]), wide=rng.choice([0, 0, rng.randint(1, 64)]))
    if kind.startswith("score"):
        return _score(**c, kind=kind, top=top, entropy=rng.random() < 0.6)
    K = rng.choice([0, _log(rng, 1, 128)])
    both = rng.random() < 0.6
    return _loss(kind, **c, K=K, ce=1.0 if K == 0 else 0.3 if both else 0.0, kd=0.0 if K == 0 else 0.7 if both else 1.0, short=rng.random() < 0.3)


# ---------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(int(seed))
    return g


def _zigzag_positions(S, D):
    """Global position of each row of the rank-major layout: rank r holds chunks r and 2D-1-r of 2D."""
    pos = torch.arange(S, device="cuda")
    if D == 1:
        return pos
    r = torch.arange(D, device="cuda")
    return pos.view(2 * D, -1)[torch.stack([r, 2 * D - 1 - r], 1).view(-1)].reshape(-1)


def prepare(case, seed):
    """Logits as a language model's: most tokens far below a few likely ones, of which the given token and the teacher's are."""
    c, g = case, _gen(seed)
    S, V, dt = c["S"], c["V"], DTYPES[c["dtype"]]
    buf = torch.empty(S, V + c["wide"], dtype=dt, device="cuda")
    step = max(1, (1 << 27) // buf.shape[1])
    for a in range(0, S, step):
        part = torch.randn(min(step, S - a), buf.shape[1], generator=g, device="cuda").mul_(2.0)
        if c["ban"]:
            part.masked_fill_(torch.rand(part.shape, generator=g, device="cuda") < c["ban"], -math.inf)
        buf[a:a + step] = part
    del part
    logits = buf[:, :V]
    # per position: the likely tokens (all different), how they stand with this model and with the teacher
    n = max(16, c.get("K", 0))
    start = torch.randint(V, (S, 1), generator=g, device="cuda")
    stride = 1 + torch.randint(V // n, (S, 1), generator=g, device="cuda")
    k = torch.arange(n, device="cuda")
    likely = (start + stride * k) % V
    level = 11.0 - 1.5 * torch.log1p(k.float()) + torch.randn(S, n, generator=g, device="cuda")
    pos = _zigzag_positions(S, c["D"])
    logits.scatter_(1, likely[pos], (level + torch.randn(S, n, generator=g, device="cuda"))[pos].to(dt))
    s = dict(case=c, logits=logits, scale=1.0 / c["temp"], ids=None)
    if c["ids"]:
        pick = (torch.rand(S, 1, generator=g, device="cuda") ** 3 * n).long().clamp_(max=n - 1)
        ids = likely.gather(1, pick).view(S)
        if c["pad"]:
            ids[1:] = torch.where(torch.rand(S, generator=g, device="cuda") < c["pad"], -1, ids)[1:]
        s["ids"] = ids.to(torch.int32 if c["ids"] == 32 else torch.int64)
    if c.get("K"):
        s["t_ids"], s["t_logits"] = likely[:, :c["K"]].to(torch.int32), level[:, :c["K"]].contiguous()
        if c["short"]:
            n_here = torch.randint(1, c["K"] + 1, (S, 1), generator=g, device="cuda")
            s["t_ids"] = torch.where(k[:c["K"]] < n_here, s["t_ids"], -1)
    if c["kind"] in ("score_bwd", "loss_bwd"):
        # what the forward has left, and the upstream gradients
        s["stats"], s["entropy"] = _stats(s)
        s["up"] = torch.randn(S, generator=g, device="cuda") / S if c["kind"] == "score_bwd" else torch.full((S,), 1.0 / S, device="cuda")
        s["up_entropy"] = torch.full((S,), 0.01 / S, device="cuda")
    if c["kind"] == "loss_train":
        s["up"] = torch.full((S,), 1.0 / S, device="cuda")
    return s


def _stats(s):
    """Each position's (largest logit, log sum of exp(scale * (logit - largest))), and the entropy, in the order of positions."""
    c = s["case"]
    stats, ent = torch.empty(c["S"], 2, device="cuda"), torch.empty(c["S"], device="cuda")
    pos = _zigzag_positions(c["S"], c["D"])
    step = max(1, (1 << 26) // c["V"])
    for a in range(0, c["S"], step):
        x = s["logits"][a:a + step].double()
        m = x.amax(1, keepdim=True)
        u = (x - m) * s["scale"]
        e = u.exp()
        total = e.sum(1)
        stats[pos[a:a + step]] = torch.stack([m[:, 0], total.log()], 1).float()
        ent[pos[a:a + step]] = (total.log() - (e * u.clamp(min=-1e4)).sum(1) / total).float()
    if s["ids"] is not None:   # positions without a token are not looked at
        stats[s["ids"] < 0] = torch.tensor([0.0, -math.inf], device="cuda")
        ent[s["ids"] < 0] = 0.0
    return stats, ent


# ---------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from folded_tensor_sequence_zigzag_gb300 import tsp
    c = s["case"]
    k, place = c["kind"], dict(D=c["D"], scale=s["scale"])
    if k == "score":
        return tsp.logprobs_fwd(s["logits"], s["ids"], top=c["top"], entropy=c["entropy"], stats=True, **place)
    if k == "score_bwd":
        more = dict(entropy=s["entropy"], dentropy=s["up_entropy"]) if c["entropy"] else {}
        return tsp.logprobs_bwd(s["logits"], s["ids"], s["stats"], dlogp=s["up"], **more, **place)
    args = dict(ids=s["ids"], w_ce=c["ce"], w_kd=c["kd"], t_scale=s["scale"], **place)
    if c["K"]:
        args.update(t_ids=s["t_ids"], t_logits=s["t_logits"])
    if k == "loss_fwd":
        return tsp.token_loss_fwd(s["logits"], stats=True, **args)
    if k == "loss_train":
        return tsp.token_loss_fwd(s["logits"], grad=True, dloss=s["up"], **args)
    return tsp.token_loss_bwd(s["logits"], s["stats"], dloss=s["up"], **args)


def _run_plain(s):
    return {"score": _plain_score, "score_bwd": _plain_score_bwd}.get(s["case"]["kind"], _plain_loss)(s)


def _order(c):
    """(position of each row, row of each position)"""
    pos = _zigzag_positions(c["S"], c["D"])
    return pos, torch.empty_like(pos).index_copy_(0, pos, torch.arange(c["S"], device="cuda"))


def _sums(s):
    """scale * (logits - largest) in the order of rows, and (largest, log of the sum) in the order of positions."""
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    u = (x - m) * s["scale"]
    return u, m, u.exp().sum(1, keepdim=True).log()


def _plain_score(s):
    c, out = s["case"], {}
    pos, row = _order(c)
    u, m, l = _sums(s)
    live = torch.ones(c["S"], dtype=torch.bool, device="cuda") if s["ids"] is None else s["ids"] >= 0
    if s["ids"] is not None:
        got = u[row, s["ids"].long().clamp(min=0)] - l[row, 0]
        out["logp"] = torch.where(live, got, 0.0)
    if c["entropy"]:
        h = l[:, 0] - (u.exp() * u.clamp(min=-1e4)).sum(1) / l[:, 0].exp()
        out["entropy"] = torch.where(live, h[row], 0.0)
    out["stats"] = torch.where(live[:, None], torch.cat([m, l], 1)[row], torch.tensor([0.0, -math.inf], device="cuda"))
    if c["top"]:
        # the larger logit first, the lower token of equal ones: one key of both
        bits = (s["logits"].float() + 0.0).view(torch.int32)
        key = ((bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32) - torch.arange(c["V"], device="cuda")
        best = key.topk(min(c["top"], c["V"]), 1).indices
        del key, bits
        logp = u.gather(1, best) - l
        best = torch.where(logp > -math.inf, best, -1)   # a banned token is no alternative
        out["top_ids"] = torch.where(live[:, None], best[row], -1).to(torch.int32)
        out["top_logp"] = torch.where(live[:, None], logp[row], -math.inf)
    return out


def _plain_score_bwd(s):
    c = s["case"]
    pos, _ = _order(c)
    x, (m, l) = s["logits"].float(), s["stats"][pos].unbind(1)
    logp = (x - m[:, None]) * s["scale"] - l[:, None]
    live = torch.isfinite(l)
    up = torch.where(live, s["up"][pos], 0.0)[:, None]
    factor = -up
    if c["entropy"]:
        factor = factor - torch.where(live, s["up_entropy"][pos], 0.0)[:, None] * (logp.clamp(min=-1e4) + s["entropy"][pos][:, None])
    d = torch.where(live[:, None], logp.exp() * factor, 0.0)
    d.scatter_add_(1, s["ids"][pos].long().clamp(min=0)[:, None], up)
    return (d * s["scale"]).to(s["logits"].dtype)


def _plain_loss(s):
    c, k = s["case"], s["case"]["kind"]
    S = c["S"]
    pos, row = _order(c)
    if k == "loss_bwd":
        (m, l), x = s["stats"][pos].unbind(1), s["logits"].float()
        m, l = m[:, None], l[:, None]
        u = (x - m) * s["scale"]
    else:
        u, m, l = _sums(s)
    live = torch.ones(S, dtype=torch.bool, device="cuda") if s["ids"] is None else s["ids"] >= 0
    loss, weight = torch.zeros(S, device="cuda"), torch.zeros(S, device="cuda")
    if c["ce"]:
        t = s["ids"].long().clamp(min=0)
        loss, weight = loss + c["ce"] * (l[row, 0] - u[row, t]), weight + c["ce"]
    if c["K"]:
        there = s["t_ids"] >= 0
        z = torch.where(there, s["t_logits"].float() * s["scale"], -math.inf)
        logq = z - z.amax(1, keepdim=True)
        logq = logq - logq.exp().sum(1, keepdim=True).log()
        q, at = logq.exp(), s["t_ids"].long().clamp(min=0)
        logp = u[row[:, None], at] - l[row]
        loss = loss + c["kd"] * torch.where(q > 0, q * (logq.clamp(min=-1e4) - logp), 0.0).sum(1)
        weight = weight + c["kd"]
    loss = torch.where(live, loss, 0.0)
    out = {"loss": loss} if k != "loss_bwd" else {}
    if k == "loss_fwd":
        out["stats"] = torch.where(live[:, None], torch.cat([m, l], 1)[row], torch.tensor([0.0, -math.inf], device="cuda"))
        return out
    up = torch.where(live, s["up"], 0.0) * s["scale"]
    d = torch.where(live[pos][:, None], (u - l).exp(), 0.0).mul_((up * weight)[pos][:, None])
    if c["ce"]:
        d.scatter_add_(1, t[pos][:, None], (-c["ce"] * up)[pos][:, None])
    if c["K"]:
        d.scatter_add_(1, at[pos], (-c["kd"] * up[:, None] * q)[pos])
    out["dlogits"] = d.to(s["logits"].dtype)
    return out["dlogits"] if k == "loss_bwd" else out


# ---------------------------------------------------------------------------- work, exact
def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    c, k = case, case["kind"]
    S, n, e = c["S"], c["S"] * c["V"], 2 if c["dtype"] == "bf16" else 4
    read = int(n * (1 - c["pad"])) if c["ids"] else n        # rows of padding are not looked at
    small = S * (c["ids"] // 8) + S * 8 * c.get("K", 0)
    if k == "score":
        out = S * (4 * bool(c["ids"]) + 4 * c["entropy"] + 8 + 8 * c["top"])
        return {"bytes": read * e + small + out, "flops": (5 + 2 * c["entropy"]) * read}
    if k == "score_bwd":
        return {"bytes": (read + n) * e + small + S * (12 + 8 * c["entropy"]), "flops": (5 + 3 * c["entropy"]) * read}
    if k == "loss_fwd":
        return {"bytes": read * e + small + 12 * S, "flops": 5 * read}
    return {"bytes": (read + n) * e + small + (8 if k == "loss_train" else 12) * S, "flops": (9 if k == "loss_train" else 5) * read}


def exact(case, seed):
    """What run() returns for these inputs, position by position from the definitions in 64 bits."""
    s = prepare(case, seed)
    c, k, got = case, case["kind"], []
    S, V = c["S"], c["V"]
    rows = torch.arange(S, device="cuda")
    if c["D"] > 1:   # chunk j < D lies in slot 0 of rank j, chunk j >= D in slot 1 of rank 2D-1-j
        n = S // (2 * c["D"])
        j = rows // n
        rows = torch.where(j < c["D"], 2 * j, 2 * (2 * c["D"] - 1 - j) + 1) * n + rows % n
    big = S * V > 2 ** 29   # (a gradient of 64 bits a value would take half a minute to hand on)
    grad = torch.zeros(S, V, dtype=torch.float32 if big else torch.float64, device="cuda") if k not in ("score", "loss_fwd") else None
    step = max(1, (1 << 25) // V)
    for a in range(0, S, step):
        at = slice(a, min(S, a + step))
        r = rows[at]
        o, d = _exact_part(s, s["logits"][r].double(), at)
        got.append(o)
        if grad is not None:
            grad[r] = d.float() if big else d
    out = {name: torch.cat([o[name] for o in got]) for name in got[0]}
    if k in ("score_bwd", "loss_bwd"):
        return grad
    if grad is not None:
        out["dlogits"] = grad
    if k == "score" and c["top"]:
        out["top_ids"] = None
    return out


def _exact_part(s, x, at):
    c, k, scale = s["case"], s["case"]["kind"], s["scale"]
    n = x.shape[0]
    live = s["ids"][at] >= 0 if s["ids"] is not None else torch.ones(n, dtype=torch.bool, device="cuda")
    one = torch.arange(n, device="cuda")
    here = live.double()
    if k in ("score_bwd", "loss_bwd"):   # from the sums that were handed over
        st = s["stats"][at].double()
        logp = scale * x - (scale * st[:, :1] + st[:, 1:])
        logp[~live] = -math.inf
    else:
        logp = torch.log_softmax(scale * x, 1)
    p = torch.where(live[:, None], torch.exp(logp), 0.0)
    plogp = torch.special.xlogy(p, p)
    o, d = {}, None
    t = s["ids"][at].long() if s["ids"] is not None else None
    if k == "score":
        if t is not None:
            o["logp"] = torch.where(live, logp[one, t.clamp(min=0)], 0.0)
        if c["entropy"]:
            o["entropy"] = -plogp.sum(1) * here
        top = x.max(1).values
        st = torch.stack([top, torch.logsumexp(scale * x, 1) - scale * top], 1)
        o["stats"] = torch.where(live[:, None], st, torch.tensor([0.0, -math.inf], dtype=torch.float64, device="cuda"))
        if c["top"]:
            best = torch.topk(logp, min(c["top"], c["V"]), 1).values
            o["top_logp"] = torch.where(live[:, None], best, -math.inf)
        return o, d
    if k == "score_bwd":
        up = s["up"][at].double() * here
        d = -p * up[:, None]
        d[one[live], t[live]] += up[live]
        if c["entropy"]:
            d -= (plogp + p * s["entropy"][at].double()[:, None]) * s["up_entropy"][at].double()[:, None]
        return o, d * scale
    loss, d = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros_like(p)
    if c["ce"]:
        loss -= c["ce"] * logp[one, t.clamp(min=0)]
        d += c["ce"] * p
        d[one[live], t[live]] -= c["ce"]
    if c["K"]:
        ids = s["t_ids"][at].long()
        q = torch.softmax((s["t_logits"][at].double() * scale).masked_fill(ids < 0, -math.inf), 1)
        loss += c["kd"] * (torch.special.xlogy(q, q) - torch.where(q > 0, q * logp.gather(1, ids.clamp(min=0)), 0.0)).sum(1)
        d += c["kd"] * p
        d.scatter_add_(1, ids.clamp(min=0), -c["kd"] * q * here[:, None])
    o["loss"] = torch.where(live, loss, 0.0)
    if k == "loss_fwd":
        top = x.max(1).values
        st = torch.stack([top, torch.logsumexp(scale * x, 1) - scale * top], 1)
        o["stats"] = torch.where(live[:, None], st, torch.tensor([0.0, -math.inf], dtype=torch.float64, device="cuda"))
        return o, None
    return o, d * (scale * s["up"][at].double())[:, None]
