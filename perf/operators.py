"""Performance cases of the operators around the block stack of a training or serving step:

* ``embed``   token embedding with a scale into the zigzag rank-major order, and its gradient;
* ``norm``    a sub-layer's output normalised, gated, scaled and added to the residual stream,
              with the next sub-layer's pre-norm of the result, and its gradient;
* ``adamw``   one AdamW update of many tensors, with 32-bit or block-scaled 8-bit states, that also
              writes the fp16 operand copies the prepared block calls read.

``run`` computes a case in elementary torch operations, or with ``own`` set through the
framework's entry points.  ``exact`` gives the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6                      # RMSNorm
LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-4, 0.9, 0.95, 1e-8, 0.1
BLOCK = 128                     # elements that share one scale of an 8-bit state
E4M3_MAX, E4M3_TINY = 448.0, 2.0 ** -9
SCALE_FLOOR = 2.0 ** -100       # a block whose largest magnitude is below this is held as zeros


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # eight new tokens of a decode step enter the model
        dict(name="embed_decode8", kind="embed_fwd", S=8, D=1, V=32000, d=4096, dtype="bf16", scaled=False, ids=64, pad=0.0),
        # the 131072-token prompt of the long-context workload, laid out for 8 ranks
        dict(name="embed_prompt128k", kind="embed_fwd", S=131072, D=8, V=32000, d=4096, dtype="bf16", scaled=True, ids=64, pad=0.0),
        # the table's gradient in a 32768-token training step (fp32 residual-stream gradient)
        dict(name="embed_grad32k", kind="embed_bwd", S=32768, D=8, V=32000, d=4096, dtype="fp32", scaled=True, ids=64, pad=0.0, add=False),
        # a tied table: the gradient is added to the head's; odd vocabulary, padded batch, 16-bit gradient
        dict(name="embed_grad_tied", kind="embed_bwd", S=16380, D=2, V=50257, d=1000, dtype="bf16", scaled=False, ids=32, pad=0.2, add=True),
        # one decoded token between two sub-layers
        dict(name="norm_decode1", kind="norm_fwd", rows=1, n=4096, dtype="bf16", stream="bf16", gate=False, post=True, pre=True, scaled=False),
        # a 16384-token prompt: post-norm, gate, scaled residual on the fp32 stream, next pre-norm
        dict(name="norm_prompt16k", kind="norm_fwd", rows=16384, n=4096, dtype="bf16", stream="fp32", gate=True, post=True, pre=True, scaled=True),
        # the same in training, gradients of everything
        dict(name="norm_grad32k", kind="norm_bwd", rows=32768, n=4096, dtype="bf16", stream="fp32", gate=True, post=True, pre=True, scaled=True),
        # small fp32 model of ragged width, no gate
        dict(name="norm_grad_ragged", kind="norm_bwd", rows=4099, n=1001, dtype="fp32", stream="fp32", gate=False, post=True, pre=True, scaled=True),
        # the nine tensors of the tiny fp32 block: all launch latency
        dict(name="adamw_tiny", kind="adamw", d=64, inter=128, layers=1, V=0, dtype="fp32", bits=32, master=False, prep=False, clip=False),
        # twelve ragged fp32 layers with their table: many tensors of sizes that no tile divides
        dict(name="adamw_many", kind="adamw", d=250, inter=683, layers=12, V=5003, dtype="fp32", bits=8, master=False, prep=False, clip=True),
        # one 7B-shaped block: bf16 weights with fp32 masters, operand copies refreshed
        dict(name="adamw_block7b", kind="adamw", d=4096, inter=11008, layers=1, V=0, dtype="bf16", bits=32, master=True, prep=True, clip=True),
        # the same with 8-bit states
        dict(name="adamw_block7b_8bit", kind="adamw", d=4096, inter=11008, layers=1, V=0, dtype="bf16", bits=8, master=True, prep=True, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges: one to 131072 rows, widths 64 to 8192, odd sizes among them."""
    kind = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd", "adamw", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind == "adamw":
        d = _log(rng, 64, 2048)
        if rng.random() < 0.6:
            d = max(64, d // 64 * 64)
        bf, inter, V = dtype == "bf16", max(d, int(d * rng.uniform(1.5, 3.0))), rng.choice([0, _log(rng, 1000, 30000)])
        layers = max(1, min(rng.randint(1, 12), (150_000_000 - V * d) // (4 * d * d + 3 * d * inter)))
        return dict(kind=kind, d=d, inter=inter, layers=layers, V=V, dtype=dtype,
                    bits=rng.choice([8, 32]), master=bf and rng.random() < 0.8, prep=bf and rng.random() < 0.7, clip=rng.random() < 0.5)
    width = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        width = max(64, width // 64 * 64)
    rows = _log(rng, 1, 131072)
    rows = max(1, min(rows, 134_000_000 // width))
    if kind.startswith("norm"):
        post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        return dict(kind=kind, rows=rows, n=width, dtype=dtype, stream="fp32" if dtype == "fp32" else rng.choice(["fp32", "bf16"]), gate=rng.random() < 0.5, post=post, pre=pre,
                    scaled=rng.random() < 0.5)
    D = rng.choice([1, 2, 4, 8])
    if D > 1:
        rows = max(1, rows // (2 * D)) * 2 * D
    V = _log(rng, 1000, min(130000, 200_000_000 // width))
    c = dict(kind=kind, S=rows, D=D, V=V, d=width, dtype=dtype, scaled=rng.random() < 0.5, ids=rng.choice([32, 64]), pad=rng.choice([0.0, 0.0, 0.3]))
    if kind == "embed_bwd":
        c["add"] = rng.random() < 0.4
    return c


# ---------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _ids(c, g):
    """Token ids with the falling frequencies of text (rank r about as often as 1/r), scattered over the table; -1 marks padding."""
    u = torch.rand(c["S"], generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(c["V"])).long().clamp_(max=c["V"]) - 1
    ids = (rank * 7919 + 13) % c["V"]
    if c["pad"]:
        ids = torch.where(torch.rand(c["S"], generator=g, device="cuda") < c["pad"], -1, ids)
    return ids.to(torch.int32 if c["ids"] == 32 else torch.int64)


def _zigzag_positions(S, D):
    """Global position of each row of the rank-major layout: rank r holds chunks r and 2D-1-r of 2D."""
    pos = torch.arange(S, device="cuda")
    if D == 1:
        return pos
    r = torch.arange(D, device="cuda")
    return pos.view(2 * D, -1)[torch.stack([r, 2 * D - 1 - r], 1).view(-1)].reshape(-1)


def _tensor_sizes(c):
    """Elements of the decayed matrices (table, then each layer's seven) and of the undecayed gains (two a layer)."""
    d, i = c["d"], c["inter"]
    mats = ([c["V"] * d] if c["V"] else []) + [d * d] * 4 * c["layers"] + [i * d] * 3 * c["layers"]
    return mats, [d] * 2 * c["layers"]


def _starts(sizes, at=0):
    """Places of tensors in a flat buffer, each at a multiple of the state block, and the buffer's end."""
    starts = []
    for n in sizes:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    return starts, at


def _quantise(x, keep_positive):
    """(codes, scales) of a flat 32-bit tensor: e4m3 values of x * (448 / largest of the block)."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1)
    live = ~(top < SCALE_FLOOR)
    inv = torch.where(live, E4M3_MAX / top, 0.0)
    scale = torch.where(live, top / E4M3_MAX, 0.0)
    q = (b * inv[:, None]).to(torch.float8_e4m3fn)
    if keep_positive:
        q = torch.where((b > 0) & (q.float() == 0) & live[:, None], torch.full_like(b, E4M3_TINY), q.float()).to(torch.float8_e4m3fn)
    return q.view(-1), scale


def _adamw_state(c, g):
    mats, gains = _tensor_sizes(c)
    ms, mid = _starts(mats)
    gs, end = _starts(gains, mid)
    dt = DTYPES[c["dtype"]]
    used = torch.zeros(end, dtype=torch.bool, device="cuda")
    for at, n in zip(ms + gs, mats + gains):
        used[at:at + n] = True
    # weights as after some training, second moments and gradients that differ by tensor region and element
    w = _normal(g, end, 0.02)
    w[mid:] += 1.0
    spread = torch.exp(_normal(g, end, 1.0)) * 1e-3
    grad = _normal(g, end, 1.0) * spread
    m = _normal(g, end, 0.3) * spread
    v = (spread * (0.5 + torch.rand(end, generator=g, device="cuda"))) ** 2
    del spread
    for t in (w, grad, m, v):
        t.masked_fill_(~used, 0.0)
    s = dict(case=c, mid=mid, end=end, grad=grad, sizes=mats + gains, starts=ms + gs, step=1000,
             clip=torch.tensor([0.37], device="cuda") if c["clip"] else None)
    s["w"] = w.to(dt)
    s["master"] = w if c["master"] else None
    s["prep"] = torch.zeros(mid, dtype=torch.float16, device="cuda") if c["prep"] else None
    if c["bits"] == 8:
        s["m"], s["m_scale"] = _quantise(m, False)
        s["v"], s["v_scale"] = _quantise(v.sqrt(), True)   # an 8-bit state holds the square root
    else:
        s["m"], s["v"] = m, v
    return s


def _pieces(s, flat, blocks=False, count=None):
    """The tensors' own views of a flat buffer (of a buffer of block scales)."""
    k = [(a // BLOCK, -(-n // BLOCK)) if blocks else (a, n) for a, n in zip(s["starts"], s["sizes"])]
    return [flat[a:a + n] for a, n in (k if count is None else k[:count])]


def prepare(case, seed):
    g, k = _gen(seed), case["kind"]
    if k.startswith("embed"):
        s = dict(case=case, ids=_ids(case, g), scale=math.sqrt(case["d"]) if case["scaled"] else 1.0)
        dt = DTYPES[case["dtype"]]
        if k == "embed_fwd":
            s["table"] = _normal(g, (case["V"], case["d"]), 0.02, dt)
        else:
            s["dx"] = _normal(g, (case["S"], case["d"]), 1.0, dt)
            # a tied table's buffer holds the head's gradient
            s["grad"] = _normal(g, (case["V"], case["d"]), 1.0) if case["add"] else None
    elif k.startswith("norm"):
        shape, n, dt, st = (case["rows"], case["n"]), case["n"], DTYPES[case["dtype"]], DTYPES[case["stream"]]
        s = dict(case=case, scale=0.7 if case["scaled"] else 1.0, f=_normal(g, shape, 0.5, dt), gate=_normal(g, shape, 1.5, dt) if case["gate"] else None)
        s["post"] = (1 + _normal(g, n, 0.2)).to(dt) if case["post"] else None
        s["pre"] = (1 + _normal(g, n, 0.2)).to(dt) if case["pre"] else None
        x = _normal(g, shape, 2.0, st)
        if k == "norm_fwd":
            s["x"] = x
        else:
            s["dh"] = _normal(g, shape, 1.0)
            s["db"] = _normal(g, shape, 1.0) if case["pre"] else None
            # what the forward has left: its output and the two rows of inverse norms
            s["h"] = x
            s["rstd_f"] = torch.rsqrt(s["f"].float().square().mean(1) + EPS) if case["post"] else None
            s["rstd_h"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS) if case["pre"] else None
    else:
        s = _adamw_state(case, g)
        if own:
            # the optimizer object that a program keeps over its steps
            from folded_tensor_sequence_zigzag_gb300 import tsp
            mats = len(_tensor_sizes(case)[0])
            s["opt"] = tsp.AdamW(_pieces(s, s["w"]), weight_decay=[DECAY] * mats + [0.0] * (len(s["sizes"]) - mats), state_bits=case["bits"],
                                 master=None if s["master"] is None else _pieces(s, s["master"]), m=_pieces(s, s["m"]), v=_pieces(s, s["v"]),
                                 m_scale=_pieces(s, s["m_scale"], True) if case["bits"] == 8 else None, v_scale=_pieces(s, s["v_scale"], True) if case["bits"] == 8 else None,
                                 prep=None if s["prep"] is None else _pieces(s, s["prep"], count=mats) + [None] * (len(s["sizes"]) - mats),
                                 betas=(BETA1, BETA2), eps=ADAM_EPS)
            s["grads"] = _pieces(s, s["grad"])
    return s


# ---------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from folded_tensor_sequence_zigzag_gb300 import tsp
    c = s["case"]
    k = c["kind"]
    if k == "embed_fwd":
        return tsp.embed_fwd(s["ids"], s["table"], D=c["D"], scale=s["scale"])
    if k == "embed_bwd":
        return tsp.embed_bwd(s["ids"], s["dx"], c["V"], D=c["D"], scale=s["scale"], out=s["grad"], accumulate=c["add"])
    if k == "norm_fwd":
        return tsp.norm_residual_fwd(s["f"], s["x"], g_post=s["post"], g_pre=s["pre"], gate=s["gate"], scale=s["scale"], eps=EPS, with_rstd=True)
    if k == "norm_bwd":
        return tsp.norm_residual_bwd(s["dh"], s["db"], s["f"], s["h"], g_post=s["post"], g_pre=s["pre"], rstd_f=s["rstd_f"], rstd_h=s["rstd_h"], gate=s["gate"], scale=s["scale"])
    s["opt"].step(s["grads"], lr=LR, step=s["step"], gscale=s["clip"])
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {n: s[n] for n in ("w", "master", "prep", "m", "v", "m_scale", "v_scale") if s.get(n) is not None}


def _run_plain(s):
    return {"embed_fwd": _embed_fwd, "embed_bwd": _embed_bwd, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "adamw": _adamw}[s["case"]["kind"]](s)


def _embed_fwd(s):
    c = s["case"]
    ids = s["ids"].long()[_zigzag_positions(c["S"], c["D"])]
    x = s["table"][ids.clamp(min=0)].float() * s["scale"]
    return torch.where((ids >= 0)[:, None], x, 0.0).to(s["table"].dtype)


def _embed_bwd(s):
    c = s["case"]
    ids = s["ids"].long()[_zigzag_positions(c["S"], c["D"])]
    rows = s["dx"].float() * s["scale"]
    grad = s["grad"] if c["add"] else torch.zeros(c["V"], c["d"], device="cuda")
    return grad.index_add_(0, ids.clamp(min=0), torch.where((ids >= 0)[:, None], rows, 0.0))


def _norm_fwd(s):
    f, rstd_f, rstd_h, b = s["f"].float(), None, None, None
    if s["post"] is not None:
        rstd_f = torch.rsqrt(f.square().mean(1) + EPS)
        f = f * rstd_f[:, None] * s["post"].float()
    if s["gate"] is not None:
        f = f * torch.sigmoid(s["gate"].float())
    h = (s["x"].float() + s["scale"] * f).to(s["x"].dtype)
    if s["pre"] is not None:
        r = h.float()   # the norm is that of the stream as it is stored
        rstd_h = torch.rsqrt(r.square().mean(1) + EPS)
        b = (r * rstd_h[:, None] * s["pre"].float()).to(s["f"].dtype)
    return h, b, rstd_f, rstd_h


def _norm_bwd(s):
    out, dt = {}, s["f"].dtype
    dx = s["dh"]
    if s["pre"] is not None:
        nh = s["h"].float() * s["rstd_h"][:, None]
        gd = s["db"] * s["pre"].float()
        dx = dx + s["rstd_h"][:, None] * (gd - nh * (gd * nh).mean(1, keepdim=True))
        out["dg_pre"] = (s["db"] * nh).sum(0)
    out["dx"] = dx.clone() if dx is s["dh"] else dx
    f = s["f"].float()
    nf = f if s["post"] is None else f * s["rstd_f"][:, None]
    u = nf if s["post"] is None else nf * s["post"].float()
    du = s["scale"] * dx
    if s["gate"] is not None:
        z = s["gate"].float()
        sig = torch.sigmoid(z)
        out["dgate"] = (du * u * sig * torch.sigmoid(-z)).to(dt)
        du = du * sig
    if s["post"] is not None:
        out["dg_post"] = (du * nf).sum(0)
        gd = du * s["post"].float()
        du = s["rstd_f"][:, None] * (gd - nf * (gd * nf).mean(1, keepdim=True))
    out["df"] = du.to(dt)
    return out


def _adamw(s):
    c, mid = s["case"], s["mid"]
    g = s["grad"] if s["clip"] is None else s["grad"] * s["clip"]
    if c["bits"] == 8:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        r = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).view(-1)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    root = v.sqrt()
    w = (s["w"] if s["master"] is None else s["master"]).float()
    step = LR / (1 - BETA1 ** s["step"])
    fix = 1 / math.sqrt(1 - BETA2 ** s["step"])
    keep = torch.cat([w[:mid] * (1 - LR * DECAY), w[mid:]])
    w = keep - step * (m / (root * fix + ADAM_EPS))
    if c["bits"] == 8:
        q, scale = _quantise(m, False)
        s["m"].copy_(q), s["m_scale"].copy_(scale)
        q, scale = _quantise(root, True)
        s["v"].copy_(q), s["v_scale"].copy_(scale)
    else:
        s["m"].copy_(m), s["v"].copy_(v)
    if s["master"] is not None:
        s["master"].copy_(w)
    s["w"].copy_(w)
    if s["prep"] is not None:
        s["prep"].copy_(s["w"][:mid])
    return _adamw_outputs(s)


# ---------------------------------------------------------------------------- work, exact
def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    c, k = case, case["kind"]
    if k == "adamw":
        mats, gains = _tensor_sizes(c)
        n, nm = sum(mats) + sum(gains), sum(mats)
        e = 2 if c["dtype"] == "bf16" else 4
        state = 2 * 8 * n if c["bits"] == 32 else 2 * (2 * n + 8 * n // BLOCK)
        weight = 8 * n + e * n if c["master"] else 2 * e * n
        return {"bytes": 4 * n + state + weight + (2 * nm if c["prep"] else 0), "flops": 16 * n}
    e = 2 if c["dtype"] == "bf16" else 4
    if k.startswith("embed"):
        S, d, V = c["S"], c["d"], c["V"]
        kept = int(S * (1 - c["pad"]))
        # distinct ids of falling frequencies: rank r is drawn with probability log(1 + 1/r) / log V
        r = torch.arange(1, V + 1, dtype=torch.float64)
        distinct = int((1 - (1 - torch.log1p(1 / r) / math.log(V)).clamp(min=0) ** kept).sum().item())
        if k == "embed_fwd":
            return {"bytes": S * c["ids"] // 8 + distinct * d * e + S * d * e, "flops": S * d}
        out = 2 * distinct * d * 4 if c["add"] else V * d * 4
        return {"bytes": S * c["ids"] // 8 + kept * d * e + out, "flops": 2 * kept * d}
    n, t = c["n"], c["rows"] * c["n"]
    s = 4 if c["stream"] == "fp32" else 2
    gains = (c["post"] + c["pre"]) * n
    if k == "norm_fwd":
        b = t * (e + e * c["gate"] + 2 * s + e * c["pre"]) + gains * e + 4 * c["rows"] * (c["post"] + c["pre"])
        return {"bytes": b, "flops": t * (10 + 6 * c["gate"])}
    b = t * (4 + 4 + e + e + (s + 4) * c["pre"] + 2 * e * c["gate"]) + gains * (e + 4) + 4 * c["rows"] * (c["post"] + c["pre"])
    return {"bytes": b, "flops": t * (22 + 10 * c["gate"])}


def exact(case, seed):
    """What run() returns for the first pass on these inputs, from the definitions in 64 bits."""
    s = _adamw_state(case, _gen(seed)) if case["kind"] == "adamw" else prepare(case, seed)
    k = case["kind"]
    if k == "embed_fwd":
        return _exact_embed_fwd(s)
    if k == "embed_bwd":
        return _exact_embed_bwd(s)
    if k == "norm_fwd":
        return _exact_norm_fwd(s)
    if k == "norm_bwd":
        return _exact_norm_bwd(s)
    return _exact_adamw(s)


def _row_of_position(S, D):
    """Row of each global position: chunk j < D is slot 0 of rank j, chunk j >= D slot 1 of rank 2D-1-j."""
    p = torch.arange(S, device="cuda")
    if D == 1:
        return p
    n = S // (2 * D)
    j = p // n
    return torch.where(j < D, 2 * j, 2 * (2 * D - 1 - j) + 1) * n + p % n


def _exact_embed_fwd(s):
    c = s["case"]
    out = torch.zeros(c["S"], c["d"], dtype=torch.float32 if c["S"] * c["d"] > 2 ** 28 else torch.float64, device="cuda")
    row, there = _row_of_position(c["S"], c["D"]), s["ids"] >= 0
    for at in range(0, c["d"], 512):   # one product of two values of the table's type fits 64 bits
        x = s["table"][:, at:at + 512].double() * s["scale"]
        out[row[there], at:at + 512] = x[s["ids"][there].long()].to(out.dtype)
    return out


def _exact_embed_bwd(s):
    c = s["case"]
    row, there = _row_of_position(c["S"], c["D"]), s["ids"] >= 0
    ids = s["ids"][there].long()
    out = torch.empty(c["V"], c["d"], dtype=torch.float64, device="cuda")
    for at in range(0, c["d"], 256):
        x = s["dx"][:, at:at + 256].double()[row[there]] * s["scale"]
        part = s["grad"][:, at:at + 256].double() if c["add"] else torch.zeros(c["V"], x.shape[1], dtype=torch.float64, device="cuda")
        out[:, at:at + 256] = part.index_put_((ids,), x, accumulate=True)
    return out


def _by_rows(rows, n):
    step = max(1, (1 << 25) // n)
    return [(a, min(rows, a + step)) for a in range(0, rows, step)]


def _exact_norm_fwd(s):
    got, c = [], s["case"]
    for a, e in _by_rows(c["rows"], c["n"]):
        u = s["f"][a:e].double()
        rf = rh = b = None
        if s["post"] is not None:
            rf = 1 / torch.sqrt((u * u).sum(1) / c["n"] + EPS)
            u = torch.einsum("rn,r,n->rn", u, rf, s["post"].double())
        if s["gate"] is not None:
            u = u / (1 + torch.exp(-s["gate"][a:e].double()))
        h = s["x"][a:e].double() + u * s["scale"]
        if s["pre"] is not None:
            q = h.to(s["x"].dtype).double()
            rh = 1 / torch.sqrt((q * q).sum(1) / c["n"] + EPS)
            b = torch.einsum("rn,r,n->rn", q, rh, s["pre"].double())
        got.append((h.float() if c["dtype"] == "bf16" else h, b, rf, rh))
    return tuple(None if p[0] is None else torch.cat(p) for p in zip(*got))


def _exact_norm_bwd(s):
    """From the derivative of u / sqrt(mean(u^2) + eps) along a row, (d - y <d, y> / n) / sqrt(mean(u^2) + eps), y the normalised row."""
    c, n = s["case"], s["case"]["n"]
    rows, sums = [], {}
    for a, e in _by_rows(c["rows"], n):
        f = s["f"][a:e].double()
        total = s["dh"][a:e].double()
        if s["pre"] is not None:
            rh = s["rstd_h"][a:e].double().unsqueeze(1)
            y, d = s["h"][a:e].double() * rh, s["db"][a:e].double()
            sums["dg_pre"] = sums.get("dg_pre", 0) + torch.einsum("rn,rn->n", d, y)
            d = d * s["pre"].double()
            total = total + rh * (d - y * torch.einsum("rn,rn->r", d, y).unsqueeze(1) / n)
        o = {"dx": total}
        y = f if s["post"] is None else f * s["rstd_f"][a:e].double().unsqueeze(1)
        gain = 1.0 if s["post"] is None else s["post"].double()
        d = total * s["scale"]
        if s["gate"] is not None:
            p = 1 / (1 + torch.exp(-s["gate"][a:e].double()))
            o["dgate"] = d * y * gain * p * (1 - p)
            d = d * p
        if s["post"] is not None:
            sums["dg_post"] = sums.get("dg_post", 0) + torch.einsum("rn,rn->n", d, y)
            d = d * gain
            d = s["rstd_f"][a:e].double().unsqueeze(1) * (d - y * torch.einsum("rn,rn->r", d, y).unsqueeze(1) / n)
        o["df"] = d
        rows.append({k: v.float() if c["rows"] * n > 2 ** 27 else v for k, v in o.items()})
    return {**{k: torch.cat([r[k] for r in rows]) for k in rows[0]}, **sums}


def _exact_codes(x, root):
    """e4m3 values of a block's elements (64 bits), and the scales."""
    b = x.view(-1, BLOCK)
    top = b.abs().max(1).values
    scale = torch.where(top < SCALE_FLOOR, 0.0, top / E4M3_MAX)
    y = torch.where(scale[:, None] > 0, b / scale.clamp(min=1e-300)[:, None], 0.0)
    # spacing of e4m3: three bits below the leading one, not finer than 2^-9
    step = torch.exp2((torch.frexp(y).exponent - 4).clamp(min=-9).double())
    q = torch.round(y / step) * step
    if root:
        q = torch.where((b > 0) & (q == 0) & (scale > 0)[:, None], E4M3_TINY, q)
    return q.view(-1).float(), scale


def _exact_adamw(s):
    c, mid, end = s["case"], s["mid"], s["end"]
    out = {k: [] for k in ("w", "m", "v", "m_scale", "v_scale")}
    b1, b2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
    cuts = sorted({0, mid, end, *range(0, end, 1 << 25)})
    for a, e in zip(cuts, cuts[1:]):
        g = s["grad"][a:e].double() * (1.0 if s["clip"] is None else s["clip"].double())
        m, v = s["m"][a:e].double(), s["v"][a:e].double()
        if c["bits"] == 8:
            m = m * s["m_scale"][a // BLOCK:e // BLOCK].double().repeat_interleave(BLOCK)
            v = (v * s["v_scale"][a // BLOCK:e // BLOCK].double().repeat_interleave(BLOCK)) ** 2
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        w = (s["w"] if s["master"] is None else s["master"])[a:e].double()
        w = w - LR * ((m / b1) / (torch.sqrt(v / b2) + ADAM_EPS) + (DECAY if a < mid else 0.0) * w)
        out["w"].append(w.float() if c["bits"] == 8 or end > 2 ** 26 else w)
        if c["bits"] == 8:
            for name, x in (("m", m), ("v", torch.sqrt(v))):
                q, scale = _exact_codes(x, name == "v")
                out[name].append(q)
                out[name + "_scale"].append(scale)
        else:
            out["m"].append(m.float()), out["v"].append(v.float())
    got = {k: torch.cat(p) for k, p in out.items() if p}
    if s["master"] is not None:
        got["master"] = got["w"]
    if s["prep"] is not None:
        got["prep"] = got["w"][:mid]
    return got
