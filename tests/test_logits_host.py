"""Arguments of the log probability and token loss entry points, checked on the
host before any launch (no GPU needed): the C ABI with made-up addresses, the
binding with CPU tensors."""
import ctypes

import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp

OK, STEP = 0x100000, 0x100000
INV, UNS = tsp.TSP_ERR_INVALID_ARG, tsp.TSP_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


def _rows(bad):
    a = dict(logits=OK, ld=10, S=16, V=10, D=4, scale=1.0, dtype=1)
    return tsp.Logits(*[bad.get(k, v) for k, v in a.items()])


ROWS = [(INV, dict(logits=None)), (INV, dict(logits=OK + 1)), (INV, dict(ld=9)), (INV, dict(S=0)),
        (INV, dict(S=-1)), (INV, dict(S=12)), (INV, dict(V=0)), (INV, dict(D=0)),
        (INV, dict(D=65, S=130)), (INV, dict(scale=0.0)), (INV, dict(scale=-1.0)),
        (INV, dict(scale=NAN)), (INV, dict(scale=INF)), (INV, dict(scale=2.0 ** 17)),
        (INV, dict(scale=2.0 ** -17)), (INV, dict(dtype=2)), (INV, dict(dtype=0, logits=OK + 2)),
        (UNS, dict(S=(1 << 30) + 8)), (UNS, dict(V=(1 << 30) + 1, ld=1 << 31)),
        (UNS, dict(ld=(1 << 32) + 1)), (INV, dict(ids=OK + 4)), (INV, dict(id_bytes=2)),
        (INV, dict(id_bytes=0))]


def _call(lib, name, order, bad):
    a = {k: OK + STEP * (i + 1) for i, k in enumerate(order)}
    a.update(id_bytes=8, top=3, w_ce=0.5, ld_d=10)
    x = bad.get("x", _rows(bad))
    t = dict(ids=OK + 30 * STEP, logits=OK + 31 * STEP, K=5, scale=1.0, weight=0.5, dtype=0)
    t.update({k[2:]: v for k, v in bad.items() if k.startswith("t_")})
    a["teacher"] = ctypes.byref(tsp.Teacher(*t.values()))
    a.update({k: a[v] if isinstance(v, str) else v for k, v in bad.items() if k in order})
    return getattr(lib, name)(None if x is None else ctypes.byref(x), *[a[k] for k in order], None)


FWD = ("ids", "id_bytes", "logp", "entropy", "stats", "top_ids", "top_logp", "top")
BWD = ("ids", "id_bytes", "stats", "entropy", "dlogp", "dentropy", "dlogits", "ld_d")
LOSS = ("ids", "id_bytes", "w_ce", "teacher", "loss", "stats", "dloss", "dlogits", "ld_d")
LOSS_BWD = ("ids", "id_bytes", "w_ce", "teacher", "stats", "dloss", "dlogits", "ld_d")


@pytest.mark.parametrize("code,bad", ROWS + [
    (INV, dict(x=None)), (INV, dict(ids=None)), (INV, dict(logp=None, entropy=None, stats=None, top=0,
                                                           top_ids=None, top_logp=None)),
    (INV, dict(top=-1)), (INV, dict(top=257)), (INV, dict(top=0)), (INV, dict(top_ids=None)),
    (INV, dict(top_logp=None)), (INV, dict(logp=OK + 2)), (INV, dict(stats=OK + 2)),
    (INV, dict(logp="entropy")), (INV, dict(stats=OK)), (INV, dict(stats=OK + 316)),
    (INV, dict(logp="ids")), (INV, dict(top_ids="top_logp")), (INV, dict(top_logp=OK + STEP + 124)),
    (INV, dict(entropy=OK - 60))])
def test_logprobs_fwd_refuses(lib, code, bad):
    assert _call(lib, "tsp_logprobs_fwd", FWD, bad) == code


@pytest.mark.parametrize("code,bad", ROWS + [
    (INV, dict(x=None)), (INV, dict(ids=None)), (INV, dict(stats=None)), (INV, dict(entropy=None)),
    (INV, dict(dentropy=None)), (INV, dict(dlogp=None, dentropy=None, entropy=None)),
    (INV, dict(dlogits=None)), (INV, dict(ld_d=9)), (INV, dict(ld_d=(1 << 32) + 1)),
    (INV, dict(dlogits=OK + STEP * 50 + 1)), (INV, dict(stats=OK + 2)),
    (INV, dict(dlogits=OK, ld_d=11)), (INV, dict(dlogits=OK + 2)), (INV, dict(dlogits=OK + 318)),
    (INV, dict(dlogits="stats")), (INV, dict(dlogits="dlogp")), (INV, dict(dlogits="ids"))])
def test_logprobs_bwd_refuses(lib, code, bad):
    assert _call(lib, "tsp_logprobs_bwd", BWD, bad) == code


TEACHER = [(INV, dict(t_ids=None)), (INV, dict(t_ids=OK + 2)), (INV, dict(t_logits=None)),
           (INV, dict(t_logits=OK + 2)), (INV, dict(t_K=0)), (INV, dict(t_K=257)),
           (INV, dict(t_scale=0.0)), (INV, dict(t_scale=NAN)), (INV, dict(t_scale=2.0 ** 17)),
           (INV, dict(t_weight=INF)), (INV, dict(t_dtype=2)), (INV, dict(w_ce=NAN)),
           (INV, dict(ids=None)), (INV, dict(dlogits=OK + 30 * STEP)), (INV, dict(dlogits=OK + 31 * STEP + 316)),
           (INV, dict(dlogits="dloss")), (INV, dict(dlogits=None)), (INV, dict(ld_d=9)),
           (INV, dict(dlogits=OK, ld_d=12)), (INV, dict(stats=None)), (INV, dict(x=None))]


@pytest.mark.parametrize("code,bad", ROWS + TEACHER + [
    (INV, dict(loss=None)), (INV, dict(loss="stats")), (INV, dict(loss="dloss")),
    (INV, dict(stats=OK + 30 * STEP + 316)), (INV, dict(loss="dlogits")), (INV, dict(loss=OK)),
    # the gradient in the logits' place: the loss may not be there too
    (INV, dict(dlogits=OK, loss=OK + 64)), (INV, dict(dlogits=OK, stats=OK + 64))])
def test_token_loss_fwd_refuses(lib, code, bad):
    assert _call(lib, "tsp_token_loss_fwd", LOSS, bad) == code


@pytest.mark.parametrize("code,bad", ROWS + TEACHER + [(INV, dict(dlogits="stats"))])
def test_token_loss_bwd_refuses(lib, code, bad):
    assert _call(lib, "tsp_token_loss_bwd", LOSS_BWD, bad) == code


def test_binding_refuses():
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    cpu = "must live on the GPU"
    with pytest.raises(ValueError, match=cpu):
        tsp.logprobs_fwd(x, ids)
    with pytest.raises(ValueError, match=cpu):
        tsp.token_loss_fwd(x, ids)
    for bad, what in ((x.half(), "bfloat16 or float32"), (x[0], "must be"), (x.t(), "dense")):
        with pytest.raises(ValueError, match=what):
            tsp.logprobs_fwd(bad)
    with pytest.raises(ValueError, match="expected"):
        tsp.logprobs_fwd(x, ids[:3])
    with pytest.raises(ValueError, match="ids"):
        tsp.logprobs_fwd(x, ids.float())
    with pytest.raises(ValueError, match="stats"):
        tsp.logprobs_bwd(x, ids, torch.zeros(4), dlogp=torch.zeros(4))
    with pytest.raises(ValueError, match="go together"):
        tsp.token_loss_fwd(x, ids, t_ids=torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="t_ids"):
        tsp.token_loss_fwd(x, ids, t_ids=torch.zeros(4, 2, dtype=torch.int64), t_logits=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="t_logits"):
        tsp.token_loss_bwd(x, torch.zeros(4, 2), ids, t_ids=torch.zeros(4, 2, dtype=torch.int32),
                           t_logits=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="rows apart"):
        tsp.logprobs_fwd(torch.zeros(8).expand(4, 8))
