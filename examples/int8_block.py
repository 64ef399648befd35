#!/usr/bin/env python3
"""A Mamba block with 8-bit projections, end to end on the library's kernels.

One block on the residual stream (kept in fp32), with random weights:

    h, r = rms_norm_int8(x, residual)              residual added, norm, 8 bits per token
    x_, z, dt, B, C = int8_matmul(W, h)            in-projections; channel-major for the scan
    y = conv1d_selective_scan_fwd(x_, ..., z)      conv + SiLU, scan, gate
    out = int8_matmul(quantize_int8(y), W_out)     out-projection of the scan's output

serve() runs a prompt and then decodes token by token through the single-token forms of the
same calls; the decoded outputs are compared with the prompt path over the whole sequence, and
both with the same block in fp32 torch on the dequantised weights.  train() takes the norm's
gradient through a scan: rms_norm -> selective_scan_fwd, selective_scan_bwd -> rms_norm_bwd.

    python examples/int8_block.py [--d-model 256] [--tokens 96] [--batch 2]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import selective_state_space_80_amd as mamba  # noqa: E402

BF16 = torch.bfloat16
N = 16    # states
TAPS = 4  # of the conv


class Int8Block:
    """Weights quantised once, a scale per output channel."""

    def __init__(self, d_model, gen):
        dev, inner = "cuda", 2 * d_model
        rand = lambda *s, std=1.0: torch.randn(s, generator=gen, device=dev) * std  # noqa: E731
        self.d_model, self.inner = d_model, inner
        self.norm_w = 1.0 + 0.1 * rand(d_model)
        q = lambda rows, cols: mamba.quantize_int8(rand(rows, cols, std=cols ** -0.5))  # noqa: E731
        self.w_x, self.w_z, self.w_dt = q(inner, d_model), q(inner, d_model), q(inner, d_model)
        self.w_b, self.w_c = q(N, d_model), q(N, d_model)
        self.w_out = q(d_model, inner)
        self.conv_w = rand(inner, TAPS, std=0.5)
        self.dt_bias = torch.full((inner,), -3.0, device=dev)
        self.A = -torch.arange(1, N + 1, device=dev, dtype=torch.float32).repeat(inner, 1)
        self.Dskip = torch.ones(inner, device=dev)

    def prompt(self, x, residual):
        """x [B, L, d_model] bf16, residual the same shape in fp32.  Returns the block's output,
        the residual stream, and the states that decoding goes on from."""
        h, s, residual = mamba.rms_norm_int8(x, self.norm_w, residual=residual)
        # weight on the left: [inner, d_model] x [B, L, d_model] -> [B, inner, L]
        x_, z, dt = (mamba.int8_matmul(w[0], h, w[1], s) for w in (self.w_x, self.w_z, self.w_dt))
        # tokens on the left: [B, L, N]
        Bm, Cm = (mamba.int8_matmul(h, w[0], s, w[1]) for w in (self.w_b, self.w_c))
        y, state, conv_state = mamba.conv1d_selective_scan_fwd(
            x_, self.conv_w, dt, self.A, Bm, Cm, return_conv_state=True, dt_bias=self.dt_bias,
            Dskip=self.Dskip, z=z, return_last_state=True)
        q, s = mamba.quantize_int8(y, channel_major=True)
        return mamba.int8_matmul(q, self.w_out[0], s, self.w_out[1]), residual, (state, conv_state)

    def token(self, x, residual, states):
        """One token: x, residual [B, d_model]; the states are updated in place."""
        state, conv_state = states
        h, s, residual = mamba.rms_norm_int8(x, self.norm_w, residual=residual)
        x_, z, dt, Bm, Cm = (mamba.int8_matmul(h, w[0], s, w[1])
                             for w in (self.w_x, self.w_z, self.w_dt, self.w_b, self.w_c))
        y = mamba.conv1d_selective_state_update(state, conv_state, x_, self.conv_w, dt, self.A,
                                                Bm, Cm, dt_bias=self.dt_bias, Dskip=self.Dskip, z=z)
        q, s = mamba.quantize_int8(y)
        return mamba.int8_matmul(q, self.w_out[0], s, self.w_out[1]), residual


def reference(block, x, residual):
    """The same block in fp32 torch, activations not quantised."""
    w = lambda q: q[0].float() * q[1].unsqueeze(-1)  # noqa: E731
    h = x.float() + residual
    n = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-5) * block.norm_w
    x_, z, dt, Bm, Cm = (n @ w(q).t() for q in (block.w_x, block.w_z, block.w_dt, block.w_b, block.w_c))
    L = x.shape[1]
    padded = torch.nn.functional.pad(x_, (0, 0, TAPS - 1, 0))
    conv = sum(padded[:, k:k + L] * block.conv_w[:, k] for k in range(TAPS))
    u = conv * torch.sigmoid(conv)
    delta = torch.nn.functional.softplus(dt + block.dt_bias)
    state, ys = torch.zeros(x.shape[0], block.inner, N, device=x.device), []
    for t in range(L):
        decay = torch.exp(delta[:, t, :, None] * block.A)
        state = decay * state + (decay - 1) / block.A * Bm[:, t, None, :] * u[:, t, :, None]
        ys.append((state * Cm[:, t, None, :]).sum(-1) + block.Dskip * u[:, t])
    y = torch.stack(ys, 1) * z * torch.sigmoid(z)
    return y @ w(block.w_out).t(), h


def apart(a, b):
    """Relative 2-norm of the difference."""
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def serve(d_model, batch, tokens, gen):
    block = Int8Block(d_model, gen)
    x = torch.randn(batch, tokens, d_model, generator=gen, device="cuda").to(BF16)
    residual = torch.randn(batch, tokens, d_model, generator=gen, device="cuda")
    out, kept, _ = block.prompt(x, residual)
    half = tokens // 2
    _, _, states = block.prompt(x[:, :half].contiguous(), residual[:, :half].contiguous())
    decoded = []
    for t in range(half, tokens):
        y, _ = block.token(x[:, t].contiguous(), residual[:, t].contiguous(), states)
        decoded.append(y)
    want, h = reference(block, x, residual)
    return {"prompt against fp32": apart(out, want),
            "decoded against the prompt path": apart(torch.stack(decoded, 1), out[:, half:]),
            "residual stream": apart(kept, h)}


def train(d_model, batch, tokens, gen):
    """Gradients of sum(scan(norm(x + r)) * dy) + sum((x + r) * dr) by the library, against
    central differences of the library's forward pass along one random direction."""
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, r, dt = rand(batch, tokens, d_model), rand(batch, tokens, d_model), 0.25 * rand(batch, d_model, tokens)
    w, dy, dr = 1.0 + 0.1 * rand(d_model), rand(batch, d_model, tokens), rand(batch, tokens, d_model)
    A = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32).repeat(d_model, 1)
    Bm, Cm = rand(batch, tokens, N), rand(batch, tokens, N)

    def forward(x, w):
        n, h = mamba.rms_norm(x, w, residual=r)
        u = n.transpose(1, 2).contiguous()
        return u, h, mamba.selective_scan_fwd(u, dt, A, Bm, Cm)

    u, h, y = forward(x, w)
    g_scan = mamba.selective_scan_bwd(u, dt, A, Bm, Cm, dy)
    g = mamba.rms_norm_bwd(g_scan["dx"].transpose(1, 2).contiguous(), h, w, dresidual_out=dr)

    def loss(x, w):
        _, h, y = forward(x, w)
        return (y.double() * dy.double()).sum() + (h.double() * dr.double()).sum()

    vx, vw, e = rand(*x.shape), rand(d_model), 1e-2
    along = (g["dx"].double() * vx.double()).sum() + (g["dweight"].double() * vw.double()).sum()
    change = (loss(x + e * vx, w + e * vw) - loss(x - e * vx, w - e * vw)) / (2 * e)
    return {"gradient against differences": abs((along - change) / change).item()}


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--d-model", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=96)
    ap.add_argument("--batch", type=int, default=2)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    found = serve(a.d_model, a.batch, a.tokens, gen)
    found.update(train(a.d_model, a.batch, a.tokens, gen))
    for name, value in found.items():
        print(f"{name}: {value:.2e}")
    return found


if __name__ == "__main__":
    main()
