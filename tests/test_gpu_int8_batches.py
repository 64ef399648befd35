"""GPU parity of the 8-bit product over very many small batches with its formula
in 64 bits (the tolerance is that of the other sizes: the sum is exact, its
conversion and two scalings round three times, 3 * 2^-24 relative)."""
import pytest

from scan_check import say

pytestmark = pytest.mark.gpu

F32_TOL = 3.01 * 2.0 ** -24


@pytest.mark.parametrize("batch,M,N,K,shared", [(4300000, 1, 1, 16, "none"), (100000, 1, 40, 64, "b"),
                                                (90000, 1, 300, 272, "b"), (70000, 3, 2, 40, "none"),
                                                (70000, 2, 5, 33, "a")])
def test_many_batches(batch, M, N, K, shared):
    import torch
    import selective_state_space_80_amd as mamba
    g = torch.Generator(device="cuda")
    g.manual_seed(batch)
    i8 = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    lead_a, lead_b = () if shared == "a" else (batch,), () if shared == "b" else (batch,)
    a, b = i8(*lead_a, M, K), i8(*lead_b, N, K)
    sa, sb = (torch.rand(t.shape[:-1], generator=g, device="cuda") + 0.01 for t in (a, b))
    say(f"product batch={batch} {M}x{N}x{K} shared={shared}")
    out = mamba.int8_matmul(a, b, sa, sb, out_dtype=torch.float32)
    want = torch.zeros((batch, M, N), dtype=torch.float64, device="cuda")
    for k in range(K):
        want += a[..., k].double().unsqueeze(-1) * b[..., k].double().unsqueeze(-2)
    want *= sa.double().unsqueeze(-1) * sb.double().unsqueeze(-2)
    assert bool(((out.double() - want).abs() <= F32_TOL * want.abs()).all())
