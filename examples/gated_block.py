#!/usr/bin/env python3
"""A block around the gated linear recurrence with 4-bit projections, end to end on the
library's kernels.

One block on the residual stream (kept in fp32), with random weights:

    n, r = rms_norm(x, residual)                  residual added, norm
    u, z = mxfp4_matmul(W, quantize_mxfp4(n))     in-projections, channel-major for the scan
    u = conv1d_silu(u)
    r, i = mxfp4_matmul(W, quantize_mxfp4(u))     the recurrence's gates
    y = gated_scan_fwd(u, r, i, lam, z)           recurrence and output gate
    out = mxfp4_matmul(quantize_mxfp4(y), W)      out-projection

serve() runs a prompt and then decodes token by token through the single-token forms of the
same calls; the decoded outputs are compared with the prompt path over the whole sequence, and
that with the same block in fp32 torch, on weights and activations rounded to the same 4 bits.
train() takes a training step's gradients through packed sequences: rms_norm ->
gated_scan_fwd, gated_scan_bwd -> rms_norm_bwd.

    python examples/gated_block.py [--d-model 256] [--tokens 96] [--batch 2]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import selective_state_space_80_amd as mamba  # noqa: E402

BF16 = torch.bfloat16
TAPS = 4  # of the conv


class GatedBlock:
    """Weights in 4 bits, laid out once."""

    def __init__(self, d_model, gen):
        dev, inner = "cuda", 2 * d_model
        rand = lambda *s, std=1.0: torch.randn(s, generator=gen, device=dev) * std  # noqa: E731
        self.d_model, self.inner = d_model, inner
        self.norm_w = 1.0 + 0.1 * rand(d_model)
        q = lambda rows, cols: mamba.quantize_mxfp4(rand(rows, cols, std=cols ** -0.5))  # noqa: E731
        self.w_u, self.w_z = q(inner, d_model), q(inner, d_model)
        self.w_r, self.w_i = q(inner, inner), q(inner, inner)
        self.w_out = q(d_model, inner)
        self.conv_w = rand(inner, TAPS, std=0.5)
        keep = 0.9 + 0.099 * torch.rand(inner, generator=gen, device=dev)  # a at r = 0
        self.lam = torch.log(torch.expm1(-2.0 * torch.log(keep) / 8.0))
        self.r_bias, self.i_bias = rand(inner, std=0.1), rand(inner, std=0.1)

    def gates(self):
        return {"r_bias": self.r_bias, "i_bias": self.i_bias}

    def prompt(self, x, residual):
        """x [B, L, d_model] bf16, residual the same shape in fp32.  Returns the block's output,
        the residual stream, and the states that decoding goes on from."""
        n, residual = mamba.rms_norm(x, self.norm_w, residual=residual)
        q, s = mamba.quantize_mxfp4(n)
        # weight on the left: [inner, d_model] x [B, L, d_model] -> [B, inner, L]
        u_, z = (mamba.mxfp4_matmul(w[0], q, w[1], s) for w in (self.w_u, self.w_z))
        u = mamba.conv1d_silu(u_, self.conv_w)
        q, s = mamba.quantize_mxfp4(u, channel_major=True)
        r, i = (mamba.mxfp4_matmul(w[0], q, w[1], s) for w in (self.w_r, self.w_i))
        y, state = mamba.gated_scan_fwd(u, r, i, self.lam, z=z, return_last_state=True, **self.gates())
        q, s = mamba.quantize_mxfp4(y, channel_major=True)
        conv_state = torch.nn.functional.pad(u_, (TAPS - 1, 0))[..., -(TAPS - 1):].contiguous()
        return mamba.mxfp4_matmul(q, self.w_out[0], s, self.w_out[1]), residual, (state, conv_state)

    def token(self, x, residual, states):
        """One token: x, residual [B, d_model]; the states are updated in place."""
        state, conv_state = states
        n, residual = mamba.rms_norm(x, self.norm_w, residual=residual)
        q, s = mamba.quantize_mxfp4(n)
        u, z = (mamba.mxfp4_matmul(q, w[0], s, w[1]) for w in (self.w_u, self.w_z))
        u = mamba.conv1d_update(conv_state, u, self.conv_w)
        q, s = mamba.quantize_mxfp4(u)
        r, i = (mamba.mxfp4_matmul(q, w[0], s, w[1]) for w in (self.w_r, self.w_i))
        y = mamba.gated_state_update(state, u, r, i, self.lam, z=z, **self.gates())
        q, s = mamba.quantize_mxfp4(y)
        return mamba.mxfp4_matmul(q, self.w_out[0], s, self.w_out[1]), residual


def reference(block, x, residual):
    """The same block in fp32 torch, activations rounded to bf16 and to 4 bits where the block's are."""
    def project(t, q):
        return t @ mamba.dequantize_mxfp4(*q, t.shape[-1], dtype=torch.float32).t()

    def in4(t):
        return mamba.dequantize_mxfp4(*mamba.quantize_mxfp4(t.contiguous()), t.shape[-1], dtype=torch.float32)

    h = x.float() + residual
    n = (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-5) * block.norm_w).to(BF16)
    n4 = in4(n)
    u_, z = (project(n4, q).to(BF16).float() for q in (block.w_u, block.w_z))
    L = x.shape[1]
    padded = torch.nn.functional.pad(u_, (0, 0, TAPS - 1, 0))
    conv = sum(padded[:, k:k + L] * block.conv_w[:, k] for k in range(TAPS))
    u = (conv * torch.sigmoid(conv)).to(BF16)
    u4 = in4(u)
    r, i = (project(u4, q).to(BF16).float() for q in (block.w_r, block.w_i))
    v = 8.0 * torch.nn.functional.softplus(block.lam) * torch.sigmoid(r + block.r_bias)
    a, into = torch.exp(-v), torch.sqrt(-torch.expm1(-2 * v)) * torch.sigmoid(i + block.i_bias) * u.float()
    state, ys = torch.zeros(x.shape[0], block.inner, device=x.device), []
    for t in range(L):
        state = a[:, t] * state + into[:, t]
        ys.append(state)
    y = (torch.stack(ys, 1) * z * torch.sigmoid(z)).to(BF16)
    return project(in4(y), block.w_out), h


def apart(a, b):
    """Relative 2-norm of the difference."""
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def serve(d_model, batch, tokens, gen):
    block = GatedBlock(d_model, gen)
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
    """Gradients of sum(recurrence(norm(x + res)) * dy) + sum((x + res) * dres) by the library,
    two sequences packed in each row, against central differences of the library's forward pass
    along one random direction."""
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, res, dres = rand(batch, tokens, d_model), rand(batch, tokens, d_model), rand(batch, tokens, d_model)
    r, i, z, dy = (rand(batch, d_model, tokens) for _ in range(4))
    w, lam = 1.0 + 0.1 * rand(d_model), rand(d_model) - 4.0
    reset = torch.zeros(batch, tokens, dtype=torch.bool, device="cuda")
    reset[:, [0, tokens // 3]] = True

    def forward(x, w, lam):
        n, h = mamba.rms_norm(x, w, residual=res)
        u = n.transpose(1, 2).contiguous()
        return u, h, *mamba.gated_scan_fwd(u, r, i, lam, z=z, reset=reset, return_checkpoints=True)

    u, h, y, kept = forward(x, w, lam)
    g_scan = mamba.gated_scan_bwd(u, r, i, lam, dy, z=z, reset=reset, checkpoints=kept)
    g = mamba.rms_norm_bwd(g_scan["dx"].transpose(1, 2).contiguous(), h, w, dresidual_out=dres)

    def loss(x, w, lam):
        _, h, y, _ = forward(x, w, lam)
        return (y.double() * dy.double()).sum() + (h.double() * dres.double()).sum()

    vx, vw, vl, e = rand(*x.shape), rand(d_model), rand(d_model), 1e-2
    along = sum((a.double() * b.double()).sum() for a, b in
                ((g["dx"], vx), (g["dweight"], vw), (g_scan["dlam"], vl)))
    change = (loss(x + e * vx, w + e * vw, lam + e * vl) - loss(x - e * vx, w - e * vw, lam - e * vl)) / (2 * e)
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
