"""The checked build over the embedding, norm-residual and AdamW calls: every
computed row and place is inside its buffer, and the results are the normal
build's bit for bit.  Each library runs in its own process."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import sys, torch
sys.path.insert(0, sys.argv[3])
from folded_tensor_sequence_zigzag_gb300 import tsp
tsp.load(sys.argv[1])
gen = torch.Generator().manual_seed(1)
out = {}
for S, D, V, d, dt in ((4096, 8, 1000, 512, torch.bfloat16), (9006, 3, 77, 250, torch.float32),
                       (70000, 1, 33000, 36, torch.bfloat16), (7, 1, 5, 1001, torch.float32)):
    ids = torch.randint(-3, V, (S,), generator=gen).cuda()
    table, dx = torch.randn(V, d, generator=gen).to(dt).cuda(), torch.randn(S, d, generator=gen).to(dt).cuda()
    out[f"x{S}"] = tsp.embed_fwd(ids, table, D=D, scale=1.5).cpu()
    out[f"g{S}"] = tsp.embed_bwd(ids, dx, V, D=D, scale=1.5).cpu()
    out[f"a{S}"] = tsp.embed_bwd(ids, dx, V, D=D, out=table.float(), accumulate=True).cpu()
for rows, n in ((300, 4096), (50, 27), (3000, 1001)):
    f, x, z = (torch.randn(rows, n, generator=gen).cuda() for _ in range(3))
    g = torch.rand(n, generator=gen).cuda()
    h, b, rf, rh = tsp.norm_residual_fwd(f, x, g, g, z, 0.5, with_rstd=True)
    r = tsp.norm_residual_bwd(x, z, f, h, g, g, rf, rh, z, 0.5)
    out.update({f"{k}{rows}": v.cpu() for k, v in dict(r, h=h, b=b).items()})
ps = [torch.randn(n, generator=gen).cuda() for n in (5, 4097, 100000)]
opt = tsp.AdamW(ps, state_bits=8)
for _ in range(2):
    opt.step([p.clone() for p in ps], lr=1e-2)
out.update({f"p{i}": p.cpu() for i, p in enumerate(ps)})
torch.cuda.synchronize()
st = tsp.device_status()
if st != tsp.TSP_OK:
    raise SystemExit(f"status {st} ({tsp.strerror(st)})")
torch.save(out, sys.argv[2])
"""


def _run(lib_path, out_path):
    r = subprocess.run([sys.executable, "-c", SCRIPT, lib_path, out_path, ROOT],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return torch.load(out_path)


def test_checked_build_runs_clean_and_matches(tmp_path):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    plain = _run(build.build(), str(tmp_path / "plain.pt"))
    checked = _run(build.build(check=True), str(tmp_path / "checked.pt"))
    assert plain.keys() == checked.keys()
    for k in plain:
        assert torch.equal(plain[k], checked[k]), k
