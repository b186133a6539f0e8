"""Arguments of the embedding, norm-residual and AdamW entry points, checked on
the host before any launch (no GPU needed): the C ABI with made-up addresses,
the binding with CPU tensors."""
import ctypes

import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp

OK, MIS = 0x10000, 0x10008
BIG = 1 << 40
INV, UNS = tsp.TSP_ERR_INVALID_ARG, tsp.TSP_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


@pytest.mark.parametrize("code,bad", [
    (INV, dict(S=0)), (INV, dict(S=-4)), (INV, dict(D=0)), (INV, dict(D=65, S=130)),
    (INV, dict(S=18, D=4)), (INV, dict(V=0)), (INV, dict(d=0)), (INV, dict(ids=None)),
    (INV, dict(ids=0x10004)), (INV, dict(id_bytes=2)), (INV, dict(table=None)),
    (INV, dict(table=MIS)), (INV, dict(x=MIS)), (INV, dict(x=2 * OK)), (INV, dict(x=OK)),
    # the last 16 bytes of the table and of the ids, and the other way round
    (INV, dict(x=2 * OK + 1584)), (INV, dict(x=OK + 112)), (INV, dict(x=2 * OK - 240)),
    (INV, dict(x=OK - 240)), (INV, dict(scale=float("nan"))),
    (INV, dict(scale=float("inf"))), (INV, dict(dtype=2)),
    (UNS, dict(S=(1 << 30) + 2, D=1)), (UNS, dict(V=(1 << 31) - 1)), (UNS, dict(d=(1 << 24) + 1))])
def test_embed_fwd_refuses(lib, code, bad):
    a = dict(ids=OK, id_bytes=8, table=2 * OK, x=3 * OK, S=16, D=4, V=100, d=8, scale=1.0, dtype=1)
    a.update(bad)
    assert lib.tsp_embed_fwd(a["ids"], a["id_bytes"], a["table"], a["x"], a["S"], a["D"], a["V"],
                             a["d"], a["scale"], a["dtype"], None) == code


@pytest.mark.parametrize("bad", [
    dict(S=0), dict(S=18, D=4), dict(V=0), dict(ids=None), dict(id_bytes=16), dict(dx=MIS),
    dict(dtable=None), dict(ws=None), dict(ws=MIS), dict(short=1), dict(dtype=3),
    dict(scale=float("nan")), dict(dtable=2 * OK), dict(ws=3 * OK),
    dict(dtable=2 * OK + 496), dict(ws=3 * OK + 3184), dict(ws=2 * OK + 496), dict(ws=OK),
    dict(dtable=OK + 48)])
def test_embed_bwd_refuses(lib, bad):
    a = dict(ids=OK, id_bytes=4, dx=2 * OK, dtype=0, dtable=3 * OK, S=16, D=4, V=100, d=8, scale=1.0,
             ws=4 * OK, short=0)
    a.update(bad)
    nb = lib.tsp_embed_bwd_workspace_bytes(16, 100, 8) - a["short"]
    assert lib.tsp_embed_bwd(a["ids"], a["id_bytes"], a["dx"], a["dtype"], a["dtable"], a["S"],
                             a["D"], a["V"], a["d"], a["scale"], 0, a["ws"], nb, None) == INV


def test_workspace_sizes(lib):
    f = lib.tsp_embed_bwd_workspace_bytes
    assert f(0, 10, 8) == 0 and f(16, 0, 8) == 0 and f(16, 10, 0) == 0
    assert f((1 << 30) + 1, 10, 8) == 0
    # tokens and rows twice, digit counts, two partial rows for each chunk of 16 to 64 positions
    S, V, d = 32768, 32000, 4096
    assert 4 * S * 4 + S // 64 * 2 * d * 4 <= f(S, V, d) <= 6 * S * 4 + S // 16 * 2 * d * 4 + 2048
    g = lib.tsp_norm_residual_bwd_workspace_bytes
    assert g(0, 8) == 0 and g(4, 0) == 0 and g(4, (1 << 24) + 1) == 0
    assert g(1, 100) == 2 * 100 * 4
    assert g(1 << 20, 4096) <= 1024 * 2 * 4096 * 4


@pytest.mark.parametrize("code,bad", [
    (INV, dict(f=None)), (INV, dict(f=MIS)), (INV, dict(x=None)), (INV, dict(h=None)),
    (INV, dict(b=None)), (INV, dict(g_pre=None)), (INV, dict(gate=MIS)), (INV, dict(rows=0)),
    (INV, dict(n=0)), (INV, dict(eps=-1.0)), (INV, dict(eps=float("nan"))),
    (INV, dict(scale=float("inf"))), (INV, dict(dtype=2)), (INV, dict(dtype=0, sdt=1)),
    (INV, dict(rstd_f=MIS)), (INV, dict(g_post=None)), (UNS, dict(n=(1 << 24) + 1)),
    (INV, dict(h="f")), (INV, dict(b="f")), (INV, dict(b="x")), (INV, dict(b="h")),
    (INV, dict(h="x", b="x")), (INV, dict(rstd_f="rstd_h")), (INV, dict(f="x", h="x")),
    (INV, dict(b=OK + 48)), (INV, dict(b=OK - 48)), (INV, dict(h=OK + 0x1000 + 16)),
    (INV, dict(rstd_f=OK + 0x1000 + 112)), (INV, dict(b=OK + 0x3000)),
    (UNS, dict(rows=1 << 31))])
def test_norm_residual_fwd_refuses(lib, code, bad):
    names = ("f", "x", "gate", "g_post", "g_pre", "h", "b", "rstd_f", "rstd_h")
    a = {k: OK + 0x1000 * i for i, k in enumerate(names)}
    a.update(gate=None, rows=4, n=8, scale=1.0, eps=1e-6, dtype=1, sdt=0)
    a.update({k: a[v] if isinstance(v, str) else v for k, v in bad.items()})
    assert lib.tsp_norm_residual_fwd(*a.values(), None) == code


@pytest.mark.parametrize("code,bad", [
    (INV, dict(f=None)), (INV, dict(dx=None)), (INV, dict(df=MIS)), (INV, dict(dgate=None)),
    (INV, dict(gate=None)), (INV, dict(db=None)), (INV, dict(h=None)), (INV, dict(rstd_h=None)),
    (INV, dict(rstd_f=None)), (INV, dict(dg_post=None)), (INV, dict(dg_pre=None)),
    (INV, dict(g_post=None)), (INV, dict(g_pre=None)), (INV, dict(rows=-1)), (INV, dict(n=0)),
    (INV, dict(ws=None)), (INV, dict(short=1)), (INV, dict(dtype=0, sdt=1)),
    (UNS, dict(n=(1 << 24) + 1)), (INV, dict(df="f")), (INV, dict(dgate="gate")),
    (INV, dict(dx="db")), (INV, dict(df="dx")), (INV, dict(dg_post="g_post")),
    (INV, dict(dg_post="dg_pre")), (INV, dict(dx=OK + 16)), (INV, dict(df=OK + 0x2000 + 48)),
    (INV, dict(dg_pre=OK + 0x1000 + 112)), (INV, dict(ws=OK + 0x1000)), (INV, dict(ws="dg_pre")),
    (INV, dict(ws="df")), (UNS, dict(rows=1 << 31))])
def test_norm_residual_bwd_refuses(lib, code, bad):
    names = ("dh", "db", "f", "gate", "h", "g_post", "g_pre", "rstd_f", "rstd_h", "dx", "df",
             "dgate", "dg_post", "dg_pre")
    a = {k: OK + 0x1000 * i for i, k in enumerate(names)}
    a.update(rows=4, n=8, scale=1.0, dtype=1, sdt=0, ws=2 * OK, short=0)
    a.update({k: a[v] if isinstance(v, str) else v for k, v in bad.items()})
    nb = lib.tsp_norm_residual_bwd_workspace_bytes(4, 8) - a.pop("short")
    assert lib.tsp_norm_residual_bwd(*a.values(), nb, None) == code


def test_norm_residual_bwd_needs_a_gradient(lib):
    """Without g_pre the only gradient is dh."""
    assert lib.tsp_norm_residual_bwd(None, None, OK, None, None, None, None, None, None, OK, OK,
                                     None, None, None, 4, 8, 1.0, 1, 0, None, 0, None) == INV


def _adamw(lib, hyper=None, count=2, bits=32, dtype=1, **bad):
    arr = (tsp.AdamwTensor * 2)()
    for i, t in enumerate(arr):
        at = OK + i * 0x10000
        t.n, t.w, t.g, t.m, t.v, t.master, t.prep = 1000, at, at, at, at, at, at
        t.weight_decay = 0.1
        if bits == 8:
            t.m_scale, t.v_scale = at, at
    for k, v in bad.items():
        setattr(arr[1], k, v)
    hy = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1)
    hy.update(hyper or {})
    return lib.tsp_adamw_step(arr, count, ctypes.byref(tsp.AdamwHyper(**hy)), bits, dtype, None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(w=None), dict(w=MIS), dict(g=None), dict(g=MIS), dict(m=None), dict(v=MIS),
    dict(master=MIS), dict(prep=MIS), dict(weight_decay=float("nan")), dict(m_scale=OK),
    dict(bits=8, m_scale=None), dict(bits=8, v_scale=None), dict(bits=8, v_scale=0x10002),
    dict(bits=4), dict(dtype=2),
    dict(dtype=0),                       # fp32 weights: no master, no fp16 copy
    dict(count=-1), dict(w=OK), dict(w=OK + 1984),     # a weight twice, two that overlap
    dict(hyper=dict(beta1=1.0)), dict(hyper=dict(beta2=-0.1)), dict(hyper=dict(eps=-1e-8)),
    dict(hyper=dict(lr=float("nan"))), dict(hyper=dict(step=0)),
    dict(hyper=dict(step_dev=0x10004)), dict(hyper=dict(gscale_dev=0x10002))])
def test_adamw_refuses(lib, bad):
    assert _adamw(lib, **bad) == INV


def test_adamw_of_nothing(lib):
    """No tensors, or only empty ones (whose pointers may be NULL): nothing to launch."""
    before = tsp.launch_count()
    assert _adamw(lib, count=0) == tsp.TSP_OK
    arr = (tsp.AdamwTensor * 1)()
    hy = tsp.AdamwHyper(1e-3, 0.9, 0.95, 1e-8, 1)
    assert lib.tsp_adamw_step(arr, 1, ctypes.byref(hy), 32, 0, None) == tsp.TSP_OK
    assert lib.tsp_adamw_step(arr, 1, None, 32, 0, None) == INV
    assert lib.tsp_adamw_step(None, 1, ctypes.byref(hy), 32, 0, None) == INV
    assert tsp.launch_count() == before


def test_binding_refuses_what_the_library_cannot_see():
    """Types, shapes and strides are the binding's to check; CPU tensors reach
    no launch."""
    ids, table = torch.zeros(4, dtype=torch.int64), torch.zeros(10, 8)
    for a, k in (((ids.float(), table), {}), ((ids.view(2, 2), table), {}),
                 ((ids, table.half()), {}), ((ids, table.t()), {}), ((ids[::2], table), {}),
                 ((ids, table), dict(out=torch.zeros(4, 9))), ((ids, table), {})):
        with pytest.raises(ValueError):
            tsp.embed_fwd(*a, **k)
    dx = torch.zeros(4, 8)
    for a, k in (((ids, dx, 10), dict(accumulate=True)), ((ids, dx[:3], 10), {}),
                 ((ids, dx.double(), 10), {}), ((ids, dx, 10), dict(out=torch.zeros(10, 8).half())),
                 ((ids, dx, 10), {})):
        with pytest.raises(ValueError):
            tsp.embed_bwd(*a, **k)
    f, g = torch.zeros(4, 8, dtype=torch.bfloat16), torch.ones(8, dtype=torch.bfloat16)
    x = torch.zeros(4, 8)
    for a, k in (((f, x[:3]), {}), ((f, x), dict(g_post=g.float())), ((f, x), dict(g_pre=g[:7])),
                 ((f, x), dict(gate=x)), ((f.half(), x), {}), ((f, x), dict(h=f)), ((f, x), {})):
        with pytest.raises(ValueError):
            tsp.norm_residual_fwd(*a, **k)
    for k in (dict(rstd_f=torch.zeros(3)), dict(g_post=g, rstd_f=torch.zeros(4).half()),
              dict(dx=f), {}):
        with pytest.raises(ValueError):
            tsp.norm_residual_bwd(x, None, f, x, **k)


def test_adamw_object_checks_its_tensors():
    p = [torch.zeros(300), torch.zeros(5, 7)]
    with pytest.raises(ValueError):
        tsp.AdamW([])
    for k in (dict(state_bits=16), dict(weight_decay=[0.1]), dict(m=[torch.zeros(300)]),
              dict(m=[torch.zeros(300), torch.zeros(34)]), dict(v_scale=[None, None]),
              dict(m=[torch.zeros(300).half(), torch.zeros(35)]), dict(prep=[None]),
              dict(master=[torch.zeros(300).half(), torch.zeros(35)])):
        with pytest.raises(ValueError):
            tsp.AdamW(p, **k)
    with pytest.raises(ValueError):
        tsp.AdamW([torch.zeros(3), torch.zeros(3).bfloat16()])
    with pytest.raises(ValueError):
        tsp.AdamW([torch.zeros(6, 4).t()])
    opt = tsp.AdamW(p, state_bits=8)
    assert [t.numel() for t in opt.m_scale] == [3, 1] and opt.m[1].dtype == torch.float8_e4m3fn
    for grads in ([p[0]], [p[0], p[1].half()], [p[0], p[0]], p):
        with pytest.raises(ValueError):
            opt.step(grads, lr=1e-3)
    assert opt.t == 0
    # states that are one another, a weight that is another's master, overlapping copies
    m, w16 = torch.zeros(335), [torch.zeros(300).bfloat16(), torch.zeros(40).bfloat16()]
    copies = torch.zeros(400).half()
    for args, k in ((p, dict(m=[m[:300], m[:35]])), (p, dict(m=[m[:300], m[299:334]])),
                    (p, dict(m=[m[:300], m[300:]], v=[torch.zeros(300), m[300:]])),
                    ([p[0], p[0][:100]], {}), (w16, dict(prep=[copies[:300], copies[296:336]]))):
        with pytest.raises(ValueError, match="share memory"):
            tsp.AdamW(args, **k)
    tsp.AdamW(p, m=[m[:300], m[300:]])
    # it holds addresses: an exchanged state or moved weight does not pass unseen
    with pytest.raises(TypeError):
        opt.m[0] = torch.zeros(300)
    p[0].data = torch.ones(300)
    with pytest.raises(ValueError, match="memory"):
        opt.step([torch.zeros(300), torch.zeros(35)], lr=1e-3)


def test_prep_views_are_the_prepared_copies(lib):
    """The views of a prepared-weights buffer follow the library's layout: the
    matrices in gradient order, each at the next multiple of 256 bytes."""
    cfg = tsp.make_cfg(2048, 256, 2, 384, 4, torch.bfloat16)
    buf = torch.zeros(tsp.block_weights_bytes(cfg), dtype=torch.uint8)
    views = tsp.prep_views(cfg, buf)
    assert [v.numel() for v in views[:7]] == [256 * 256] * 4 + [384 * 256] * 3
    assert views[7:] == [None, None]
    ends = [(v.data_ptr() - buf.data_ptr(), 2 * v.numel()) for v in views[:7]]
    at = 0
    for a, n in ends:
        assert a == at
        at += (n + 255) // 256 * 256
    assert at == buf.numel()
