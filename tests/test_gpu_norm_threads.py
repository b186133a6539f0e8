"""norm_residual calls from several host threads at once, each with a width of its own:
what one call sets up for its launch does not change another's."""
import threading

import pytest
import torch

from folded_tensor_sequence_zigzag_gb300 import tsp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from folded_tensor_sequence_zigzag_gb300 import build
    build.build()
    return tsp.load()


@pytest.mark.parametrize("backward", [False, True])
def test_widths_of_one_kernel_in_several_threads(lib, backward):
    """Single rows of different widths that run on the same kernel, with 60 to 130 KB of
    shared memory a CTA (the forward's four units a thread, the backward's)."""
    bf, f32 = torch.bfloat16, torch.float32
    calls, outs, keep = [], [], []
    for i, n in enumerate((4352, 8192, 6400, 8192) if backward else (8200, 16384, 12288, 16384)):
        g = torch.Generator("cuda").manual_seed(i)
        f, x = (torch.randn(1, n, generator=g, device="cuda").to(bf) for _ in range(2))
        gain = torch.rand(n, generator=g, device="cuda").to(bf)
        h, b, rf, rh = tsp.norm_residual_fwd(f, x, gain, gain, with_rstd=True)
        stream = torch.cuda.Stream()
        if backward:
            d = torch.randn(1, n, generator=g, device="cuda")
            out = [torch.empty(1, n, device="cuda"), torch.empty(1, n, dtype=bf, device="cuda"),
                   torch.empty(n, device="cuda"), torch.empty(n, device="cuda")]
            ws = torch.empty(tsp.norm_residual_bwd_workspace_bytes(1, n), dtype=torch.uint8, device="cuda")
            ins, ends = [d, d, f, None, h, gain, gain, rf, rh, out[0], out[1], None, *out[2:]], \
                [1, n, 1.0, tsp.TSP_BF16, tsp.TSP_BF16, ws.data_ptr(), ws.numel(), stream.cuda_stream]
        else:
            out = [torch.empty_like(h), torch.empty_like(b)]
            ins, ends = [f, x, None, gain, gain, *out, None, None], \
                [1, n, 1.0, 1e-6, tsp.TSP_BF16, tsp.TSP_BF16, stream.cuda_stream]
            ws = None
        calls.append([None if t is None else t.data_ptr() for t in ins] + ends)
        outs.append(out)
        keep.append((ins, ws, stream))
    fn = lib.tsp_norm_residual_bwd if backward else lib.tsp_norm_residual_fwd
    torch.cuda.synchronize()
    want = []
    for c, out in zip(calls, outs):
        assert fn(*c) == tsp.TSP_OK
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
        for t in out:
            t.zero_()
    torch.cuda.synchronize()
    start, codes = threading.Barrier(len(calls)), [set() for _ in calls]

    def run(i):
        start.wait()
        codes[i].update(fn(*calls[i]) for _ in range(20000))   # (without the interpreter's lock)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{tsp.TSP_OK}] * len(calls)
    assert all(torch.equal(a, b) for w, o in zip(want, outs) for a, b in zip(w, o))
