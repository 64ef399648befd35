"""The block of examples/gated_block.py (4-bit projections around the gated recurrence),
and its calls inside HIP graphs, on other streams and on two streams at once.

Bounds: the reference rounds activations to bf16 and to 4 bits where the block does, so
what differs is the fp32 sums' order, which moves a bf16 rounding by one step (0.4 %) for
about one value in a thousand and a 4-bit rounding (a step of a fifth) for about one in ten
thousand of those: 0.2 sqrt(1e-3) below 0.7 % in each of three places even if every moved
bf16 rounding moved a 4-bit one; and the output's own rounding to bf16, 0.2 %: below 2 %.
Decoding repeats the prompt path's arithmetic but for the same orders: below 2 %.  The
residual stream is an fp32 sum: 1e-6.  Central differences with step 1e-2 leave the third
derivatives, of order step^2 = 1e-4 with the cancellation of the sum: below 1 %."""
import importlib.util
import os

import pytest

from scan_check import say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("gated_block", os.path.join(ROOT, "examples", "gated_block.py"))
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
    assert found["prompt against fp32"] < 2e-2
    assert found["decoded against the prompt path"] < 2e-2
    assert found["residual stream"] < 1e-6
    assert found["gradient against differences"] < 1e-2


def _calls(B, D, L, n, seed, io):
    """Every call on inputs of its own, a packed batch among them; (inputs to refill, calls)."""
    import torch
    import selective_state_space_80_amd as mamba
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(io)  # noqa: E731
    x, r, i, z, dout = (rand(B, D, L) for _ in range(5))
    lam, bias = torch.randn(D, generator=gen, device="cuda") - 3, torch.randn(D, generator=gen, device="cuda")
    reset = torch.rand((B, L), generator=gen, device="cuda") < 0.01
    h0, xt = torch.randn((B, D), generator=gen, device="cuda"), rand(B, D)
    w, ws = mamba.quantize_mxfp4(rand(n, D))

    def calls():
        y, last, kept = mamba.gated_scan_fwd(x, r, i, lam, r_bias=bias, i_bias=bias, z=z, h0=h0, reset=reset,
                                             return_last_state=True, return_checkpoints=True)
        g = mamba.gated_scan_bwd(x, r, i, lam, dout, r_bias=bias, i_bias=bias, z=z, h0=h0, reset=reset,
                                 dh_last=h0, checkpoints=kept)
        g2 = mamba.gated_scan_bwd(x, r, i, lam, dout, z=z, h0=h0)
        q, s = mamba.quantize_mxfp4(y, channel_major=True)
        out, out2 = mamba.mxfp4_matmul(q, w, s, ws), mamba.mxfp4_matmul(w, q, ws, s, out_dtype=torch.float32)
        state = torch.empty_like(h0)
        step = mamba.gated_state_update(h0, xt, xt, xt, lam, h_out=state)
        tq, ts = mamba.quantize_mxfp4(step)
        return [y, last, kept, q, s, out, out2, state, step, tq, ts, mamba.mxfp4_matmul(tq, w, ts, ws),
                mamba.dequantize_mxfp4(q, s, D)] + [t for d in (g, g2) for t in d.values()]

    def refill():
        for t in (x, r, i, z, dout, xt):
            t.copy_(rand(*t.shape))
        h0.normal_(generator=gen)

    return refill, calls


SHAPES = [(1, 2560, 1, 512), (2, 130, 300, 515), (1, 257, 9000, 130), (3, 771, 1001, 1536), (2, 2560, 512, 5120)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,L,n", SHAPES)
def test_graph(B, D, L, n, io):
    """Captured, replayed with new inputs, eager work between: bit for bit the eager call."""
    import torch
    say(f"graph {B} x {D} x {L} {io}")
    refill, calls = _calls(B, D, L, n, L, torch.float32 if io == "f32" else torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = calls()
    for k in range(3):
        refill()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = calls()
        junk = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        assert torch.isfinite(junk)
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"replay {k} differs"


def test_two_streams_at_once():
    """Calls of two callers on their own streams, tensors made on another, several times over."""
    import torch
    sets = [_calls(*SHAPES[3], seed=1, io=torch.bfloat16)[1], _calls(*SHAPES[2], seed=2, io=torch.float32)[1]]
    want = [calls() for calls in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        for s, calls in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(calls())
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for k, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[k % 2]))


@pytest.mark.parametrize("off", [1, 3])
def test_tensors_at_any_element(off):
    """Activations that start at any element of a larger buffer, and outputs beside guarded memory."""
    import torch
    import selective_state_space_80_amd as mamba
    for io in (torch.float32, torch.bfloat16):
        for B, D, L in ((2, 5, 30), (2, 3, 700)):
            n = B * D * L
            gen = torch.Generator(device="cuda")
            gen.manual_seed(off)
            bases = [torch.randn(n + 16, generator=gen, device="cuda").to(io) for _ in range(5)]
            at = [b[off:off + n].view(B, D, L) for b in bases]
            room = torch.full((n + 16,), 7.0, device="cuda", dtype=io)
            out = room[off:off + n].view(B, D, L)
            lam = torch.zeros(D, device="cuda")
            y, kept = mamba.gated_scan_fwd(*at[:3], lam, z=at[3], out=out, return_checkpoints=True)
            g = mamba.gated_scan_bwd(*at[:3], lam, at[4], z=at[3], checkpoints=kept)
            plain = [t.clone() for t in at]
            y1, kept1 = mamba.gated_scan_fwd(*plain[:3], lam, z=plain[3], return_checkpoints=True)
            g1 = mamba.gated_scan_bwd(*plain[:3], lam, plain[4], z=plain[3], checkpoints=kept1)
            assert torch.equal(y, y1) and all(torch.equal(g[k], g1[k]) for k in g)
            assert bool((room[:off] == 7).all()) and bool((room[off + n:] == 7).all())
