"""Token embedding into the zigzag order and its table gradient, against plain
64-bit sums.  u = 2^-24 is half a spacing of fp32, 2^-8 of bf16."""
import math

import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


def row_of_pos(S, D):
    if D == 1:
        return list(range(S))
    c = S // (2 * D)
    out = []
    for p in range(S):
        j = p // c
        r, slot = (j, 0) if j < D else (2 * D - 1 - j, 1)
        out.append((2 * r + slot) * c + p % c)
    return out


def make_ids(kind, S, V, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        return torch.randint(0, V, (S,), generator=g)
    if kind == "one":                      # every position the same token
        return torch.full((S,), V - 1)
    if kind == "few":                      # long runs of few tokens, first and last among them
        return torch.tensor([0, V - 1, V // 2])[torch.randint(0, 3, (S,), generator=g)]
    if kind == "padded":
        ids = torch.randint(0, V, (S,), generator=g)
        return torch.where(torch.rand(S, generator=g) < 0.4, torch.tensor(-1), ids)
    assert kind == "all_padding"
    return torch.full((S,), -7)


def expect_fwd(ids, table, D, scale):
    S = ids.shape[0]
    ref = torch.zeros(S, table.shape[1], dtype=torch.float64)
    t64 = table.double().cpu()
    for p, r in enumerate(row_of_pos(S, D)):
        if 0 <= ids[p] < table.shape[0]:
            ref[r] = t64[ids[p]] * scale
    return ref


FWD = [(1, 1, 7, 1, BF), (1, 1, 50, 64, BF), (5, 1, 50, 33, BF), (8, 1, 1000, 4096, BF),
       (48, 3, 97, 250, BF), (64, 4, 11, 1001, F32), (6, 3, 11, 2, F32), (200, 1, 33, 1000, F32),
       (4096, 8, 501, 768, BF), (514, 1, 64, 2057, BF)]


@pytest.mark.parametrize("S,D,V,d,dt", FWD)
@pytest.mark.parametrize("kind", ["uniform", "padded"])
@pytest.mark.parametrize("scale", [1.0, 22.627417])
def test_forward(S, D, V, d, dt, kind, scale):
    ids = make_ids(kind, S, V, seed=S + d)
    table = torch.randn(V, d, generator=torch.Generator().manual_seed(d)).to(dt)
    for idt in (torch.int32, torch.int64):
        got = tsp.embed_fwd(ids.to(idt).cuda(), table.cuda(), D=D, scale=scale).double().cpu()
        ref = expect_fwd(ids, table, D, scale)
        # one fp32 product of the fp32 scale, one rounding to the table's type
        s32 = torch.tensor(scale, dtype=torch.float32).double().item()
        tol = ref.abs() * ((UBF if dt == BF else 0) + 2 * U32 + abs(s32 / scale - 1))
        assert bool(((got - ref).abs() <= (0 if scale == 1.0 else tol)).all())
    assert tsp.device_status() == tsp.TSP_OK


def test_forward_keeps_nan_and_infinity_of_their_rows_only():
    table = torch.ones(4, 64, dtype=BF)
    table[1, 3], table[2, 5] = float("nan"), float("-inf")
    got = tsp.embed_fwd(torch.tensor([0, 1, 2, -1]).cuda(), table.cuda(), scale=2.0).cpu().float()
    assert torch.isnan(got[1, 3]) and got[2, 5] == float("-inf")
    got[1, 3] = got[2, 5] = 2.0
    assert torch.equal(got, torch.tensor([2.0, 2.0, 2.0, 0.0])[:, None].expand(4, 64))


def expect_bwd(ids, dx, V, D, scale, base=None):
    """(sum, sum of magnitudes, occurrences) in 64 bits."""
    rows = torch.tensor(row_of_pos(ids.shape[0], D))
    there = (ids >= 0) & (ids < V)
    x = dx.double().cpu()[rows[there]]
    at = ids[there]
    s = torch.zeros(V, dx.shape[1], dtype=torch.float64).index_add_(0, at, x * scale)
    a = torch.zeros(V, dx.shape[1], dtype=torch.float64).index_add_(0, at, x.abs() * abs(scale))
    n = torch.zeros(V, dtype=torch.float64).index_add_(0, at, torch.ones(at.shape[0], dtype=torch.float64))
    if base is not None:
        s, a = s + base.double(), a + base.double().abs()
    return s, a, n


def bwd_tol(a, n, scale):
    # n - 1 additions of the fp32 sum in whatever grouping, the scaling, the
    # scale's own rounding, the addition to the table
    return a * ((n[:, None] + 3) * U32)


BWD = [(1, 1, 5, 1), (1, 1, 40, 64), (7, 1, 40, 4096), (31, 1, 9, 33), (64, 4, 700, 256),
       (96, 3, 50, 1000), (514, 1, 20, 257), (1000, 1, 100000, 12), (4096, 8, 1000, 512),
       (4098, 1, 77, 130), (4864, 4, 3000, 40), (4865, 1, 3000, 40), (20000, 2, 513, 68), (33000, 1, 262145, 4), (70000, 1, 512, 36)]


@pytest.mark.parametrize("S,D,V,d", BWD)
@pytest.mark.parametrize("kind", ["uniform", "few", "padded"])
@pytest.mark.parametrize("dt", [F32, BF])
def test_backward(S, D, V, d, kind, dt):
    ids = make_ids(kind, S, V, seed=S)
    dx = torch.randn(S, d, generator=torch.Generator().manual_seed(1)).to(dt)
    scale = math.sqrt(d)
    ref, mag, n = expect_bwd(ids, dx, V, D, scale)
    got = tsp.embed_bwd(ids.cuda(), dx.cuda(), V, D=D, scale=scale)
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= bwd_tol(mag, n, scale)).all()), float((err - bwd_tol(mag, n, scale)).max())
    # the same call gives the same bits; so does another id type
    again = tsp.embed_bwd(ids.int().cuda(), dx.cuda(), V, D=D, scale=scale)
    assert torch.equal(got, again)
    # added to a table's gradient: rows of absent tokens keep their bits
    base = torch.randn(V, d, generator=torch.Generator().manual_seed(2))
    out = base.cuda()
    tsp.embed_bwd(ids.cuda(), dx.cuda(), V, D=D, scale=scale, out=out, accumulate=True)
    ref, mag, _ = expect_bwd(ids, dx, V, D, scale, base)
    assert bool(((out.double().cpu() - ref).abs() <= bwd_tol(mag, n, scale)).all())
    assert torch.equal(out.cpu()[n == 0], base[n == 0])
    assert tsp.device_status() == tsp.TSP_OK


@pytest.mark.parametrize("kind", ["one", "all_padding"])
@pytest.mark.parametrize("S,d", [(2, 8), (9, 4096), (12345, 300)])
def test_backward_of_one_token_and_of_none(S, d, kind):
    V = 130
    ids = make_ids(kind, S, V, 0)
    dx = torch.randn(S, d, generator=torch.Generator().manual_seed(3))
    ref, mag, n = expect_bwd(ids, dx, V, 1, 1.0)
    got = tsp.embed_bwd(ids.cuda(), dx.cuda(), V)
    assert bool(((got.double().cpu() - ref).abs() <= bwd_tol(mag, n, 1.0)).all())
    assert not got[n.cuda() == 0].any()


def test_padding_rows_may_hold_anything():
    """The gradient rows of padding are not read into any sum."""
    ids = torch.tensor([3, -1, 3, 2, -5, -1])
    dx = torch.ones(6, 20)
    dx[ids < 0] = float("nan")
    got = tsp.embed_bwd(ids.cuda(), dx.cuda(), 5).cpu()
    assert torch.equal(got[:, 0], torch.tensor([0.0, 0.0, 1.0, 2.0, 0.0])) and got.isfinite().all()


def test_id_past_the_table_is_recorded_and_touches_nothing():
    ids = torch.tensor([0, 9, 2, 2 ** 40 + 1, -2 ** 40])
    table = torch.ones(9, 16)
    assert tsp.device_status() == tsp.TSP_OK
    got = tsp.embed_fwd(ids.cuda(), table.cuda())
    assert tsp.device_status() == tsp.TSP_ERR_RANGE
    assert torch.equal(got.cpu()[:, 0], torch.tensor([1.0, 0.0, 1.0, 0.0, 0.0]))
    grad = tsp.embed_bwd(ids.cuda(), torch.ones(5, 16, device="cuda"), 9)
    assert tsp.device_status() == tsp.TSP_ERR_RANGE
    want = torch.zeros(9)
    want[0] = want[2] = 1
    assert torch.equal(grad.cpu()[:, 5], want)
    # -2^40 alone is padding
    tsp.embed_fwd(ids[4:].cuda(), table.cuda())
    assert tsp.device_status() == tsp.TSP_OK


def test_gradient_against_differences():
    """d/dE of sum(dx * forward(E)) by central differences of the 64-bit forward
    (linear in E, so a step of 1 has no truncation error)."""
    S, D, V, d, scale = 24, 2, 10, 6, 1.5
    ids = make_ids("padded", S, V, 5)
    E = torch.randn(V, d, generator=torch.Generator().manual_seed(4))
    dx = torch.randn(S, d, generator=torch.Generator().manual_seed(5))
    got = tsp.embed_bwd(ids.cuda(), dx.cuda(), V, D=D, scale=scale).double().cpu()
    for v in range(V):
        for c in range(d):
            step = torch.zeros(V, d)
            step[v, c] = 1.0
            diff = ((expect_fwd(ids, E + step, D, scale) - expect_fwd(ids, E - step, D, scale))
                    * dx.double()).sum() / 2
            # E + step is rounded to fp32: one half spacing of values below 8 on each side
            assert abs(diff - got[v, c]) <= S * scale * 8 * U32 * float(dx.abs().max()) * 2 + \
                abs(diff) * 8 * U32


def test_more_positions_than_tiles_of_the_sort():
    """Over 512 * 1024 positions a CTA of the sort takes several tiles in a row."""
    S, V, d = 600002, 3001, 4
    gen = torch.Generator("cuda").manual_seed(1)
    ids = torch.randint(-50, V, (S,), generator=gen, device="cuda")
    ids[200000:260000] = 17
    dx = torch.randn(S, d, generator=gen, device="cuda")
    got = tsp.embed_bwd(ids, dx, V)
    there = ids >= 0
    z = lambda t, w: torch.zeros(V, w, dtype=torch.float64, device="cuda").index_add_(0, ids[there], t[there])   # noqa: E731
    ref, mag = z(dx.double(), d), z(dx.double().abs(), d)
    n = z(torch.ones(S, 1, dtype=torch.float64, device="cuda"), 1)
    assert bool(((got.double() - ref).abs() <= mag * ((n + 3) * U32)).all())
    assert torch.equal(got, tsp.embed_bwd(ids, dx, V))


@pytest.mark.parametrize("S", [3, 1000, 9000])
def test_huge_vocabulary(S):
    """Tokens of 27 bits: too wide to be counted in one word with their position,
    three passes of the sort; nearly all rows are absent."""
    V, d = (1 << 26) + 5, 2
    gen = torch.Generator().manual_seed(S)
    ids = torch.randint(0, V, (S,), generator=gen)
    ids[0], ids[-1] = V - 1, 0
    ids[S // 2] = ids[S // 3]
    dx = torch.randn(S, d, generator=gen)
    got = tsp.embed_bwd(ids.cuda(), dx.cuda(), V)
    at, back = ids.unique(return_inverse=True)
    ref = torch.zeros(len(at), d, dtype=torch.float64).index_add_(0, back, dx.double())
    assert bool(((got[at.cuda()].double().cpu() - ref).abs() <= 4 * U32 * (ref.abs() + 8)).all())
    assert int((got != 0).any(1).sum()) == len(at)


def test_row_offsets_past_32_bits():
    """A table of more than 2^31 elements: the last rows are read and written."""
    V, d = 530000, 4096                     # 2.17e9 elements
    table = torch.zeros(V, d, dtype=BF, device="cuda")
    table[V - 1], table[V - 3] = 3.0, 5.0
    ids = torch.tensor([V - 1, 0, V - 3, V - 1]).cuda()
    got = tsp.embed_fwd(ids, table)
    assert torch.equal(got[:, 0].float().cpu(), torch.tensor([3.0, 0.0, 5.0, 3.0]))
    del table
    dx = torch.ones(4, d, device="cuda")
    grad = tsp.embed_bwd(ids, dx, V)
    assert grad[V - 1].eq(2.0).all() and grad[V - 3].eq(1.0).all() and grad[0].eq(1.0).all()
    assert float(grad.sum(dtype=torch.float64)) == 4.0 * d


def test_workspaces_are_checked():
    ids, dx = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(4, 8, device="cuda")
    n = tsp.embed_bwd_workspace_bytes(4, 3, 8)
    for ws in (torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            tsp.embed_bwd(ids, dx, 3, ws=ws)
    with pytest.raises(tsp.TspError) as e:
        tsp.embed_bwd(ids, dx, 3, ws=torch.zeros(n - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.code == tsp.TSP_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        tsp.embed_fwd(ids.cpu(), torch.ones(3, 8, device="cuda"))


def test_zigzag_forward_is_gather_then_permute():
    S, D, V, d = 512, 8, 100, 256
    ids = make_ids("uniform", S, V, 1).cuda()
    table = torch.randn(V, d).to(BF).cuda()
    assert torch.equal(tsp.embed_fwd(ids, table, D=D), tsp.zigzag_permute(table[ids], D))


def test_side_stream_and_captured_calls():
    """On a stream of its own, and captured: a replay reads what the tensors
    hold then; two graphs may share a workspace when they run in order."""
    S, V, d = 640, 50, 128
    ids = make_ids("uniform", S, V, 1).cuda()
    dx = torch.randn(S, d).cuda()
    table = torch.randn(V, d).cuda()
    want_x, want_g = tsp.embed_fwd(ids, table), tsp.embed_bwd(ids, dx, V)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = tsp.embed_fwd(ids, table, stream=side), tsp.embed_bwd(ids, dx, V, stream=side)
    side.synchronize()
    assert torch.equal(a, want_x) and torch.equal(b, want_g)
    ws = torch.empty(tsp.embed_bwd_workspace_bytes(S, V, d), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty(V, d, device="cuda") for _ in range(2)], []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x = tsp.embed_fwd(ids, table)
            tsp.embed_bwd(ids, dx, V, scale=1.0 + k, out=outs[k], ws=ws)
        graphs.append((g, x))
    new = make_ids("padded", S, V, 9).cuda()
    ids.copy_(new)
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for k, (_, x) in enumerate(graphs):
        assert torch.equal(x, tsp.embed_fwd(ids, table))
        assert torch.equal(outs[k], tsp.embed_bwd(ids, dx, V, scale=1.0 + k))


def test_position_offsets_past_32_bits():
    """x_z and dx_z of more than 2^31 elements, in the zigzag order: the sums of ones are
    counts, exact in fp32."""
    S, D, V, d = 530000, 8, 9, 4096
    ids = make_ids("padded", S, V, 3).cuda()
    table = (torch.arange(V).float()[:, None] + torch.arange(d) / 64).to(BF).cuda()
    x = tsp.embed_fwd(ids, table, D=D)
    back = tsp.zigzag_permute(x, D, inverse=True)
    for v in range(V):
        assert bool((back[ids == v] == table[v]).all())
    assert not bool(back[ids < 0].any())
    del back
    grad = tsp.embed_bwd(ids, x.fill_(1.0), V, D=D)
    count = torch.stack([(ids == v).sum() for v in range(V)]).float()
    assert torch.equal(grad, count[:, None].expand(V, d))
