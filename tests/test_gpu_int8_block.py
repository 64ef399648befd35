"""The block with 8-bit projections of examples/int8_block.py, and its calls
inside HIP graphs.

Bounds: 8-bit rows whose largest value is about 3.5 deviations have a step of
3.5/127 of one, and a rounding error of step/sqrt(12) = 0.8 % of the row's
2-norm; the block rounds its activations twice on the way to a product of three
projections of the same rows (x, z, C and dt multiply), and in bf16 (0.2 %)
at five places: below 5 % in all.  Decoding repeats the prompt path's arithmetic
but for the order of sums in the scan and the conv output's rounding: its own
8-bit roundings may flip, below 2 %.  The residual stream is an fp32 sum: 1e-6.
Central differences with step 1e-2 leave the third derivatives, of order
step^2 = 1e-4 with the cancellation of the sum: below 1 %."""
import importlib.util
import os

import pytest

from scan_check import say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("int8_block", os.path.join(ROOT, "examples", "int8_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("d_model,batch,tokens", [(64, 1, 9), (256, 2, 96), (200, 3, 41), (768, 1, 200)])
def test_block(d_model, batch, tokens):
    import torch
    ex = _example()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(d_model)
    found = ex.serve(d_model, batch, tokens, gen)
    found.update(ex.train(d_model, batch, tokens, gen))
    say(str(found))
    assert found["prompt against fp32"] < 5e-2
    assert found["decoded against the prompt path"] < 2e-2
    assert found["residual stream"] < 1e-6
    assert found["gradient against differences"] < 1e-2


def _replays(calls, refill, n=3):
    """Captures calls() and replays it n times against the eager result, with
    eager work and synchronisations between the replays."""
    import torch
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = calls()
    for k in range(n):
        refill(k)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = calls()
        junk = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        assert torch.isfinite(junk)
        for got, ref in zip(outs, want):
            assert torch.equal(got, ref), f"replay {k} differs"


@pytest.mark.parametrize("M,D,n", [(1, 2560, 5120), (8, 768, 1536), (300, 771, 515), (2100, 768, 2048)])
def test_graph(M, D, n):
    """norm -> product, quantiser -> product, gradient of the norm (bit for bit)."""
    import torch
    import selective_state_space_80_amd as mamba
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, r, w = rand(M, D).bfloat16(), rand(M, D), 1 + 0.1 * rand(D)
    wq, ws = mamba.quantize_int8(rand(n, D))
    dy, y = rand(M, D).bfloat16(), rand(1, D, M).bfloat16()

    def calls():
        h, s, kept = mamba.rms_norm_int8(x, w, residual=r)
        out = mamba.int8_matmul(h, wq, s, ws)
        q, qs = mamba.quantize_int8(y, channel_major=True)
        out2 = mamba.int8_matmul(wq, q, ws, qs, out_dtype=torch.float32)
        g = mamba.rms_norm_bwd(dy, kept, w, dresidual_out=r)
        return h, s, kept, out, q, out2, g["dx"], g["dresidual"], g["dweight"]

    def refill(k):
        x.copy_(rand(M, D).bfloat16())
        r.copy_(rand(M, D))
        y.copy_(rand(1, D, M).bfloat16())
        dy.copy_(rand(M, D).bfloat16())

    _replays(calls, refill)


def test_other_stream():
    """On a stream of the caller's, with tensors made on another."""
    import torch
    import selective_state_space_80_amd as mamba
    x, r = torch.randn(500, 1000, device="cuda"), torch.randn(500, 1000, device="cuda")
    w = torch.ones(1000, device="cuda")
    wq, ws = mamba.quantize_int8(torch.randn(333, 1000, device="cuda"))

    def calls():
        h, s, kept = mamba.rms_norm_int8(x, w, residual=r)
        g = mamba.rms_norm_bwd(x, kept, w)
        return h, s, kept, mamba.int8_matmul(h, wq, s, ws), g["dx"], g["dweight"]

    want = calls()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = calls()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
