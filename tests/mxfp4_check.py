"""The microscaled 4-bit format in 64 bits, from its definition."""
import math

import torch

U = 2.0 ** -24
VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
GROUP, BLOCK = 256, 32


def groups(K):
    return -(-K // GROUP)


def encode(x):
    """x [..., K] -> (codes of the elements [..., G * 256], codes of the scales [..., G * 8])."""
    x = x.detach().cpu()
    K, G = x.shape[-1], groups(x.shape[-1])
    full = torch.zeros((*x.shape[:-1], G * GROUP), dtype=torch.float64)
    full[..., :K] = x.double()
    blocks = full.unflatten(-1, (-1, BLOCK))
    bad = ~torch.isfinite(blocks).all(-1)
    top = torch.where(bad, 1.0, blocks.abs().amax(-1))
    exponent = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp_min(-127)
    y = torch.ldexp(torch.where(bad[..., None], 0.0, blocks), -exponent[..., None].double())
    # the nearest value; of two as near the one whose code is even
    apart = (y.abs()[..., None] - VALUES).abs()
    code = torch.zeros(y.shape, dtype=torch.int64)
    best = apart[..., 0]
    for c in range(1, 8):
        better = (apart[..., c] < best) | ((apart[..., c] == best) & (c % 2 == 0))
        code = torch.where(better, c, code)
        best = torch.where(better, apart[..., c], best)
    sign = torch.signbit(torch.where(bad[..., None], 0.0, blocks))
    return (code + 8 * sign).flatten(-2), torch.where(bad, 255, exponent + 127)


def pack(codes, scales):
    """The layout of the library's tensors: q [..., G * 128], scale [G, ..., 8]."""
    q = (codes[..., 0::2] | codes[..., 1::2] << 4).to(torch.uint8)
    return q, scales.unflatten(-1, (-1, 8)).movedim(-2, 0).to(torch.uint8).contiguous()


def values(q, scale):
    """q, scale as the library lays them out -> [..., G * 256] in 64 bits."""
    q, scale = q.cpu(), scale.cpu()
    codes = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
    size = VALUES[codes & 7] * torch.where(codes >= 8, -1.0, 1.0)
    s = scale.movedim(0, -2).flatten(-2).long()
    power = torch.where(s == 255, math.nan, torch.ldexp(torch.ones((), dtype=torch.float64), (s - 127).double()))
    return size * power.repeat_interleave(BLOCK, -1)


def random_operand(lead, rows, K, seed, low=-6, high=6):
    """A packed operand with zeros from K on: every element code, scales of a range of powers."""
    gen = torch.Generator().manual_seed(seed)
    G = groups(K)
    codes = torch.randint(0, 16, (*lead, rows, G * GROUP), generator=gen)
    codes[..., K:] = 0
    scales = torch.randint(127 + low, 128 + high, (*lead, rows, G * 8), generator=gen)
    return pack(codes, scales)


def product_bound(a, b, out, half_step):
    """Each scaled instruction adds 64 exact products to a sum: its result and what it
    drops inside are within 2 u of the sum of sizes so far; four instructions a group,
    a few more additions where a workgroup's waves split the inner axis; then the output
    type's rounding."""
    size = a.nan_to_num().abs() @ b.nan_to_num().abs().mT
    err = (a.shape[-1] / 64 + 12) * 2 * U * size
    return err + half_step * (out.abs() + err) + 1e-37
