"""h = x + s sigmoid(z) rms(f; g_post), b = rms(h; g_pre) and their gradients
against the formulas in 64 bits.  u = 2^-24 is half a spacing of fp32, 2^-8 of
bf16.  A row sum of squares or products is formed by chains of at most 64
additions and two rounds of 5 pairwise ones (rows here are at most 64 * 1024
wide), so it is off by at most 80 u of the sum of magnitudes; an inverse norm
by half that, 2 spacings of rsqrtf and a division: 45 u."""
import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp

pytestmark = pytest.mark.gpu
U, UBF = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


def inputs(rows, n, dt, st, gate, post, pre, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 7 + n)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    t = dict(f=r(rows, n).to(dt), x=(2 * r(rows, n)).to(st), gate=(2 * r(rows, n)).to(dt) if gate else None,
             g_post=(1 + 0.3 * r(n)).to(dt) if post else None,
             g_pre=(1 + 0.3 * r(n)).to(dt) if pre else None)
    if rows > 2:                       # an all-zero row, a huge and a tiny one
        t["f"][1] = 0
        t["f"][2] *= 1e4 if dt == F32 else 1e3
        t["f"][0] *= 1e-4
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def d64(t):
    return None if t is None else t.double()


def ref_fwd(f, x, gate, g_post, g_pre, s):
    """(h, b, rstd_f, rstd_h) without any rounding; 64-bit inputs."""
    rf = rh = b = None
    u = f
    if g_post is not None:
        rf = (f.square().mean(1) + EPS).rsqrt()
        u = f * rf[:, None] * g_post
    if gate is not None:
        u = u / (1 + torch.exp(-gate))
    h = x + s * u
    if g_pre is not None:
        rh = (h.square().mean(1) + EPS).rsqrt()
        b = h * rh[:, None] * g_pre
    return h, b, rf, rh


SHAPES = [(2600, 1000), (5003, 261), (640, 8192), (700, 5003), (1000, 1), (300, 2), (701, 5), (613, 27), (2003, 29), (650, 255), (1300, 513), (155, 8191),
          (153, 12290), (1, 1), (1, 8), (3, 7), (1, 4096), (2, 16384), (5, 64), (300, 256), (7, 1001), (4, 250),
          (9, 2057), (3, 8192), (2, 8200), (1000, 24), (3, 20000), (2, 40001), (700, 1000)]
MODES = [(True, True, True), (False, True, True), (True, False, True), (False, True, False),
         (True, False, False), (False, False, True)]   # gate, post, pre


@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("dt,st", [(BF, F32), (BF, BF), (F32, F32)])
def test_forward(rows, n, dt, st):
    for gate, post, pre in MODES:
        t = inputs(rows, n, dt, st, gate, post, pre)
        s = 0.75
        h, b, rf, rh = tsp.norm_residual_fwd(t["f"], t["x"], t["g_post"], t["g_pre"], t["gate"], s,
                                             EPS, with_rstd=True)
        a = {k: d64(v) for k, v in t.items()}
        wh, _, wrf, _ = ref_fwd(a["f"], a["x"], a["gate"], a["g_post"], None, s)
        us = UBF if st == BF else 0
        # u: 45 u of the norm, 3 products, 4 u of the sigmoid (expf 2, sum, quotient, product)
        tol = (wh - a["x"]).abs() * 55 * U + wh.abs() * 2 * U
        assert bool(((h.double() - wh).abs() <= tol + (wh.abs() + tol) * us).all()), (gate, post, pre)
        if post:
            assert bool(((rf.double() - wrf).abs() <= 45 * U * wrf).all())
        assert (b is None) == (not pre) and (rf is None) == (not post) and (rh is None) == (not pre)
        if pre:   # of the stored h
            hh = h.double()
            wrh = (hh.square().mean(1) + EPS).rsqrt()
            assert bool(((rh.double() - wrh).abs() <= 45 * U * wrh).all())
            wb = hh * wrh[:, None] * a["g_pre"]
            ub = UBF if dt == BF else 0
            assert bool(((b.double() - wb).abs() <= wb.abs() * (50 * U + ub * (1 + 50 * U))
                         + 1e-38).all()), (gate, post, pre)


def test_in_place_and_equal_to_rmsnorm():
    """h may be x; b is what rmsnorm_fwd gives for the stored h, up to the order
    of one fp32 row sum."""
    t = inputs(40, 512, BF, BF, True, True, True)
    h, b = tsp.norm_residual_fwd(t["f"], t["x"], t["g_post"], t["g_pre"], t["gate"])
    x = t["x"].clone()
    h2, b2 = tsp.norm_residual_fwd(t["f"], x, t["g_post"], t["g_pre"], t["gate"], h=x)
    assert h2 is x and torch.equal(h, h2) and torch.equal(b, b2)
    ref = tsp.rmsnorm_fwd(h, t["g_pre"], EPS).double()
    assert bool(((b.double() - ref).abs() <= ref.abs() * (2 * UBF + 100 * U)).all())


@pytest.mark.parametrize("z", [float("-inf"), -3e38, -100.0, -0.0, 100.0, 3e38, float("inf"),
                               float("nan")])
def test_gate_at_its_ends(z):
    """A closed gate leaves x, an open one adds all of f; slopes end at 0; a NaN
    reaches its own elements only."""
    n = 64
    f, x = torch.full((2, n), 2.0).cuda(), torch.ones(2, n).cuda()
    gate = torch.zeros(2, n).cuda()
    gate[1] = z
    h, _ = tsp.norm_residual_fwd(f, x, gate=gate)
    g = torch.sigmoid(torch.tensor(z, dtype=torch.float64)).item()
    assert torch.equal(h[0].cpu(), torch.full((n,), 2.0))
    want = torch.full((n,), 1 + 2 * g, dtype=torch.float64)
    assert torch.allclose(h[1].double().cpu(), want, rtol=4 * U, atol=0, equal_nan=True)
    out = tsp.norm_residual_bwd(x, None, f, None, gate=gate)
    slope = torch.full((n,), 2 * g * (1 - g), dtype=torch.float64)
    assert torch.allclose(out["dgate"][1].double().cpu(), slope, rtol=8 * U, atol=1e-38, equal_nan=True)
    assert torch.allclose(out["df"][1].double().cpu(), torch.full((n,), g, dtype=torch.float64),
                          rtol=4 * U, atol=1e-38, equal_nan=True)
    assert torch.equal(out["df"][0].cpu(), torch.full((n,), 0.5))


def test_rows_of_zeros_and_of_infinities():
    t = inputs(4, 128, BF, F32, False, True, True)
    t["f"][:] = 0
    t["x"][:2] = 0
    t["f"][3, 5] = float("inf")
    h, b = tsp.norm_residual_fwd(t["f"], t["x"], t["g_post"], t["g_pre"])
    assert torch.equal(h[:3], t["x"][:3]) and not b[:2].any() and b[2].isfinite().all()
    assert not h[3].isfinite().all()      # the norm of an infinite row is not finite
    assert h[:3].isfinite().all()


def ref_bwd(a, h, dh, db, rf, rh, s):
    """Gradients, and the size of the terms each is the sum of (for its tolerance)."""
    out, mag = {}, {}
    zero = torch.zeros_like(a["f"])
    dx, m = (zero, zero) if dh is None else (dh, dh.abs())
    if a["g_pre"] is not None:
        y, gd = h * rh[:, None], db * a["g_pre"]
        dx = dx + rh[:, None] * (gd - y * (gd * y).mean(1, keepdim=True))
        m = m + rh[:, None] * (gd.abs() + y.abs() * (gd * y).abs().mean(1, keepdim=True))
        out["dg_pre"], mag["dg_pre"] = (db * y).sum(0), (db * y).abs().sum(0)
    out["dx"], mag["dx"] = dx, m
    y = a["f"] if rf is None else a["f"] * rf[:, None]
    g = 1.0 if a["g_post"] is None else a["g_post"]
    sig = 1.0 if a["gate"] is None else torch.sigmoid(a["gate"])
    du, mu = s * sig * dx, abs(s) * sig * m
    if a["gate"] is not None:
        slope = sig * torch.sigmoid(-a["gate"])
        out["dgate"] = s * dx * y * g * slope
        mag["dgate"] = abs(s) * m * (y * g).abs() * slope
    if rf is not None:
        out["dg_post"], mag["dg_post"] = (du * y).sum(0), (mu * y.abs()).sum(0)
        gd, mg = du * g, mu * abs(g)
        du = rf[:, None] * (gd - y * (gd * y).mean(1, keepdim=True))
        mu = rf[:, None] * (mg + y.abs() * (mg * y.abs()).mean(1, keepdim=True))
    out["df"], mag["df"] = du, mu
    return out, mag


@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("dt,st", [(BF, F32), (BF, BF), (F32, F32)])
def test_backward(rows, n, dt, st):
    for gate, post, pre in MODES:
        t = inputs(rows, n, dt, st, gate, post, pre)
        s = 0.75
        h, _, rf, rh = tsp.norm_residual_fwd(t["f"], t["x"], t["g_post"], t["g_pre"], t["gate"], s,
                                             EPS, with_rstd=True)
        g = torch.Generator().manual_seed(5)
        dh = torch.randn(rows, n, generator=g).cuda() if not (pre and gate) else None
        db = torch.randn(rows, n, generator=g).cuda() if pre else None
        got = tsp.norm_residual_bwd(dh, db, t["f"], h, t["g_post"], t["g_pre"], rf, rh, t["gate"], s)
        a = {k: d64(v) for k, v in t.items()}
        ref, mag = ref_bwd(a, h.double(), d64(dh), d64(db), d64(rf), d64(rh), s)
        assert set(got) == set(ref)
        for k, v in got.items():
            # row sums 80 u of their magnitudes, at most 20 roundings of products and of the
            # sigmoid beside them, for df those of dx and a second row sum: 200 u in all; the
            # gains' column sums run over the rows
            tol = mag[k] * U * (200 + (rows if k.startswith("dg_") else 0))
            if k in ("df", "dgate"):
                tol = tol + (ref[k].abs() + tol) * (UBF if dt == BF else 0)
            err = (v.double() - ref[k]).abs()
            assert bool((err <= tol + 1e-38).all()), (k, gate, post, pre, float((err - tol).max()))
        again = tsp.norm_residual_bwd(dh, db, t["f"], h, t["g_post"], t["g_pre"], rf, rh, t["gate"], s)
        assert all(torch.equal(got[k], again[k]) for k in got)     # nothing is atomic
        if dh is not None:                                          # dx in place of dh
            mine = dh.clone()
            out = tsp.norm_residual_bwd(mine, db, t["f"], h, t["g_post"], t["g_pre"], rf, rh,
                                        t["gate"], s, dx=mine)
            assert out["dx"] is mine and all(torch.equal(got[k], out[k]) for k in got)


def test_gradients_against_differences():
    """Central differences of the 64-bit forward along random directions, every
    input at once and each alone."""
    rows, n, s = 6, 40, 1.25
    t = inputs(rows, n, F32, F32, True, True, True, seed=3)
    t["f"][:] = torch.randn(rows, n, generator=torch.Generator().manual_seed(8)).cuda()
    h, _, rf, rh = tsp.norm_residual_fwd(t["f"], t["x"], t["g_post"], t["g_pre"], t["gate"], s, EPS,
                                         with_rstd=True)
    g = torch.Generator().manual_seed(6)
    dh, db = (torch.randn(rows, n, generator=g).cuda() for _ in range(2))
    got = tsp.norm_residual_bwd(dh, db, t["f"], h, t["g_post"], t["g_pre"], rf, rh, t["gate"], s)
    names = dict(f="df", x="dx", gate="dgate", g_post="dg_post", g_pre="dg_pre")
    a = {k: d64(v) for k, v in t.items()}

    def loss(v):
        hh, bb, _, _ = ref_fwd(v["f"], v["x"], v["gate"], v["g_post"], v["g_pre"], s)
        return float((dh.double() * hh).sum() + (db.double() * bb).sum())
    for which in [list(names)] + [[k] for k in names]:
        way = {k: torch.randn(a[k].shape, generator=g, dtype=torch.float64).cuda() for k in which}
        e = 1e-5
        diff = (loss({k: a[k] + e * way[k] if k in way else a[k] for k in a})
                - loss({k: a[k] - e * way[k] if k in way else a[k] for k in a})) / (2 * e)
        size = sum(float((got[names[k]].double() * way[k]).abs().sum()) for k in which)
        mine = sum(float((got[names[k]].double() * way[k]).sum()) for k in which)
        # the kernel's fp32 (200 u of its terms, which are a few times the result's size), and
        # the differences' own error: e^2 times a third derivative of order one, and 2^-53 / e
        assert abs(diff - mine) <= size * (1000 * U + 1e-8) + 1e-6


def test_single_row_side_stream_and_capture():
    t = inputs(1, 4096, BF, F32, True, True, True)
    args = (t["f"], t["x"], t["g_post"], t["g_pre"], t["gate"])
    want = tsp.norm_residual_fwd(*args, with_rstd=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tsp.norm_residual_fwd(*args, with_rstd=True, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    dh, db = torch.randn(1, 4096).cuda(), torch.randn(1, 4096).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, b, rf, rh = tsp.norm_residual_fwd(*args, with_rstd=True)
        grads = tsp.norm_residual_bwd(dh, db, t["f"], h, t["g_post"], t["g_pre"], rf, rh, t["gate"])
    t["f"].copy_(torch.randn(1, 4096))
    t["x"].copy_(torch.randn(1, 4096))
    graph.replay()
    torch.cuda.synchronize()
    want = tsp.norm_residual_fwd(*args, with_rstd=True)
    assert all(torch.equal(x, y) for x, y in zip(want, (h, b, rf, rh)))
    again = tsp.norm_residual_bwd(dh, db, t["f"], h, t["g_post"], t["g_pre"], rf, rh, t["gate"])
    assert all(torch.equal(grads[k], again[k]) for k in grads)


def test_element_offsets_past_32_bits():
    """2^31 elements and more, of ragged rows: rows that hold the same and start at the
    same element of a unit give the same bits, wherever they are."""
    n, period, times = 2049, 1024, 1024          # 2.15e9 elements; the period is whole units
    t = inputs(period, n, BF, BF, True, True, True)
    gen = torch.Generator("cuda").manual_seed(1)
    dh, db = (torch.randn(period, n, device="cuda", generator=gen) for _ in range(2))
    args = (t["g_post"], t["g_pre"])
    want = tsp.norm_residual_fwd(t["f"], t["x"], *args, t["gate"], 0.5, with_rstd=True)
    grad = tsp.norm_residual_bwd(dh, db, t["f"], want[0], *args, *want[2:], t["gate"], 0.5)

    def all_equal(big, small):
        return bool((big.view(times, *small.shape) == small).all())
    f, gate, h = (t[k].repeat(times, 1) for k in ("f", "gate", "x"))
    got = tsp.norm_residual_fwd(f, h, *args, gate, 0.5, h=h, with_rstd=True)
    for a, b in zip(got, want):
        assert all_equal(a, b)
    out = tsp.norm_residual_bwd(dh.repeat(times, 1), db.repeat(times, 1), f, h, *args, *got[2:], gate, 0.5)
    for k in ("dx", "df", "dgate"):
        assert all_equal(out[k], grad[k])
    # dg_pre: a CTA (152 of them at least) adds up at most 2^20 / 152 = 6899 rows, then come
    # the sums of the CTAs' parts, 43 additions deep at most; a term is off by 4 u (the
    # product, h times its inverse norm): below 7000 u of the terms' magnitudes.
    hh = want[0].double() * want[3].double()[:, None]
    terms = db.double() * hh
    tol = 7000 * U * terms.abs().sum(0) * times
    assert bool(((out["dg_pre"].double() - terms.sum(0) * times).abs() <= tol).all())


def test_two_calls_at_once():
    """Calls on two streams, each with what is its own."""
    ts = [inputs(3000 + i, 1024, BF, F32, True, True, True, seed=i) for i in range(2)]
    grads = [torch.randn(3000 + i, 1024, generator=torch.Generator().manual_seed(i)).cuda() for i in range(2)]

    def step(t, g, stream=None):
        h, b, rf, rh = tsp.norm_residual_fwd(t["f"], t["x"], t["g_post"], t["g_pre"], t["gate"],
                                             with_rstd=True, stream=stream)
        out = tsp.norm_residual_bwd(g, g, t["f"], h, t["g_post"], t["g_pre"], rf, rh, t["gate"], stream=stream)
        return [h, b, *out.values()]
    want = [step(t, g) for t, g in zip(ts, grads)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(5):
        got = [step(t, g, s) for t, g, s in zip(ts, grads, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(want, got) for a, b in zip(x, y))
