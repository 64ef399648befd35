"""The 4-bit product where one operand's scales are at the ends of their range, from 2^-127 to
2^127, and the other's at the opposite end: the products are ordinary numbers, the values
themselves need not be in fp32's range.  Against 64 bits, within its sums' rounding."""
import pytest
import torch

import mxfp4_check as C
from scan_check import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 70, 600), (17, 33, 256), (300, 515, 1001), (1030, 1100, 768)])
def test_scales_at_opposite_ends(M, N, K):
    import selective_state_space_80_amd as mamba
    say(f"4-bit product, scales at opposite ends, {M} x {N} x {K}")
    gen = torch.Generator().manual_seed(M)
    a, _ = C.random_operand((), M, K, 1)
    b, _ = C.random_operand((), N, K, 2)
    G = C.groups(K)
    block = torch.randint(0, 255, (G, 1, 8), generator=gen)
    block[:, :, ::3] = torch.tensor([0, 254, 1])[torch.arange(G) % 3].view(G, 1, 1)
    near = lambda rows: torch.randint(-3, 4, (G, rows, 8), generator=gen)  # noqa: E731
    sa = (block + near(M)).clamp(0, 254).to(torch.uint8)
    sb = (254 - block + near(N)).clamp(0, 254).to(torch.uint8)
    va, vb = C.values(a, sa), C.values(b, sb)
    want = va @ vb.mT
    for dtype, half_step in ((torch.float32, C.U), (torch.bfloat16, 2.0 ** -8)):
        got = mamba.mxfp4_matmul(a.cuda(), b.cuda(), sa.cuda(), sb.cuda(), out_dtype=dtype)
        part = ((got.double().cpu() - want).abs() / C.product_bound(va, vb, want, half_step)).max().item()
        say(f"  part of the bound {part:.2f}")
        assert part <= 1.0
