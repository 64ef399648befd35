"""GPU parity of the 8-bit matrix product with its formula in 64 bits.

The integer sum is exact; its conversion to fp32 and the two scalings round
three times, 3 * 2^-24 relative; a bf16 output adds half an ulp, at most
2^-8."""
import pytest

from scan_check import say

pytestmark = pytest.mark.gpu

F32_TOL = 3.01 * 2.0 ** -24
BF16_TOL = F32_TOL + 2.0 ** -8


def _operand(shape, seed, full=False):
    import torch
    g = torch.Generator().manual_seed(seed)
    low, high = (-128, 128) if full else (-127, 128)
    q = torch.randint(low, high, shape, generator=g, dtype=torch.int64).to(torch.int8)
    return q.cuda(), (torch.rand(shape[:-1], generator=g) * 0.1 + 0.001).cuda()


def _want(a, b, sa, sb):
    return (a.double() @ b.double().transpose(-1, -2)) * sa.double().unsqueeze(-1) * sb.double().unsqueeze(-2)


def _check(a, b, sa, sb, what, dtypes=("f32", "bf16")):
    import torch
    import selective_state_space_80_amd as mamba
    want = _want(a, b, sa, sb)
    for name in dtypes:
        dt, tol = (torch.float32, F32_TOL) if name == "f32" else (torch.bfloat16, BF16_TOL)
        got = mamba.int8_matmul(a, b, sa, sb, out_dtype=dt)
        assert got.shape == want.shape and got.dtype == dt
        err = (got.double() - want).abs()
        bad = ~(err <= tol * want.abs())
        assert not bad.any(), f"{what} {name}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}"
    say(f"{what} ok")


SIZES = [1, 2, 15, 16, 17, 31, 33, 64, 65, 100, 127, 128, 129, 200, 256, 257, 300]


@pytest.mark.parametrize("K", [1, 2, 15, 16, 17, 31, 48, 63, 64, 65, 100, 127, 128, 129, 144, 255, 256, 272, 333,
                               512, 520, 1001, 1024, 2560, 4112])
def test_inner_sizes(K):
    for M, N in [(1, 1), (3, 5), (1, 200), (40, 33), (130, 140), (300, 257)]:
        a, sa = _operand((M, K), K + M, full=True)
        b, sb = _operand((N, K), K + N + 1, full=True)
        _check(a, b, sa, sb, f"matmul {M}x{N}x{K}")


@pytest.mark.parametrize("M", SIZES)
def test_outer_sizes(M):
    for N in SIZES:
        for K in (64, 80, 203):
            a, sa = _operand((M, K), M + 3 * N)
            b, sb = _operand((N, K), M + 5 * N)
            _check(a, b, sa, sb, f"matmul {M}x{N}x{K}", ("bf16",))


@pytest.mark.parametrize("M,N,K", [(1, 5120, 2560), (2, 2560, 5120), (5, 1000, 768), (8, 5120, 2560), (16, 5120, 2560),
                                   (17, 1536, 768), (33, 2560, 5120), (64, 2560, 5120), (100, 5120, 2560),
                                   (256, 2560, 5120), (5120, 1, 2560), (2560, 20, 5120), (1000, 1000, 1000),
                                   (1024, 1024, 1024), (700, 2048, 768), (1, 8191, 33), (513, 4001, 640),
                                   (2048, 1536, 768), (2049, 2561, 1536), (4096, 4096, 128), (3001, 515, 1001)])
def test_projection_sizes(M, N, K):
    a, sa = _operand((M, K), M + N)
    b, sb = _operand((N, K), M + K)
    _check(a, b, sa, sb, f"matmul {M}x{N}x{K}")


@pytest.mark.parametrize("batch,M,N,K", [(2, 33, 70, 128), (8, 1, 300, 257), (3, 300, 5, 64), (5, 129, 257, 96),
                                         (2, 1536, 1000, 768), (8, 256, 512, 256), (4, 2560, 1, 512),
                                         (2, 1030, 2050, 272)])
@pytest.mark.parametrize("shared", ["none", "a", "b"])
def test_batches(batch, M, N, K, shared):
    a, sa = _operand(((batch,) if shared != "a" else ()) + (M, K), M)
    b, sb = _operand(((batch,) if shared != "b" else ()) + (N, K), N)
    _check(a, b, sa, sb, f"matmul batch={batch} shared={shared} {M}x{N}x{K}")


# Sizes that take every tile form, with ragged edges, several tiles a workgroup,
# inner sizes that end inside a step, and rows on and off 64-byte boundaries.
@pytest.mark.parametrize("batch,M,N,K", [
    (1, 5000, 5200, 1040), (1, 8200, 4100, 800), (1, 7000, 6101, 720), (1, 3000, 2900, 2096), (2, 2500, 2600, 1000),  # 256 x 256
    (1, 9000, 8100, 304), (1, 6000, 6016, 400), (1, 5000, 4200, 200), (1, 4300, 4201, 64), (1, 9000, 1024, 100), (3, 1500, 1300, 16), (1, 6000, 6080, 128),  # 128 x 128
    (1, 1100, 1100, 640), (1, 600, 5000, 1300), (1, 2000, 700, 2100), (1, 600, 4992, 144),      # the same, deep
    (1, 1000, 400, 4000), (1, 400, 1000, 4000), (1, 300, 700, 4000), (1, 700, 300, 4000),       # rings
    (1, 500, 500, 3000), (1, 700, 700, 900), (1, 900, 1000, 900), (1, 200, 2900, 3000), (1, 2500, 250, 6000),
    (1, 250, 2500, 6000), (1, 50, 7000, 1500), (1, 7000, 50, 1500), (1, 2500, 100, 6000), (1, 100, 2500, 6000),
    (1, 40, 3000, 2000), (1, 3000, 40, 2000), (1, 17, 5000, 3000), (1, 5000, 17, 3000), (1, 64, 8000, 1000)])
def test_forms(batch, M, N, K):
    lead = (batch,) if batch > 1 else ()
    a, sa = _operand(lead + (M, K), M + K)
    b, sb = _operand((N, K), N + K)
    _check(a, b, sa, sb, f"matmul batch={batch} {M}x{N}x{K}")


# Drawn sizes, some for each form that the choice makes of them: rows at 16-byte
# boundaries (256 x 256, 128 x 128, the same deep, then the rings from 64 x 64 down)
# and off them, then tiles of 128 x 64 on and off.
@pytest.mark.parametrize("M,N,K", [
    (10858, 835, 1072), (1920, 7468, 560), (7304, 559, 320), (934, 7594, 800), (450, 7985, 1424),
    (3597, 571, 144), (1988, 396, 64), (4299, 169, 1280), (847, 1602, 2720), (2617, 213, 80), (7577, 88, 1632),
    (1547, 466, 1712), (9, 8923, 272), (33, 4164, 1136), (8564, 5, 4064), (5120, 79, 64), (52, 2757, 2416),
    (158, 924, 3712), (90, 1074, 1024), (2932, 24, 2064), (7243, 2, 560), (5988, 5, 96), (520, 106, 288),
    (10, 2667, 48),
    (5815, 1817, 62), (2620, 2328, 1077), (2963, 751, 3003), (262, 6656, 4043), (110, 6404, 75),
    (3141, 258, 1844), (2631, 193, 658), (40, 8845, 138), (4360, 130, 1243), (59, 10764, 63), (2124, 157, 122),
    (246, 1178, 1752), (8759, 30, 44), (2078, 198, 110), (6702, 24, 91), (293, 514, 33), (4, 8763, 1251),
    (3078, 29, 131), (10872, 6, 100), (8026, 2, 2394), (53, 5, 113), (3, 431, 199),
    (441, 3392, 2656), (225, 6784, 32), (1535, 2540, 736), (2182, 584, 2142), (5660, 164, 125)])
def test_drawn_sizes_of_every_form(M, N, K):
    a, sa = _operand((M, K), M + K)
    b, sb = _operand((N, K), N + K)
    _check(a, b, sa, sb, f"matmul {M}x{N}x{K}")


def test_extremes():
    """The largest sums an inner size of 131071 allows stay exact."""
    import torch
    import selective_state_space_80_amd as mamba
    for M, N in [(1, 3), (17, 20), (130, 130), (600, 700)]:
        K = 131071 if M < 600 else 131056
        a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
        b = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        b[-1] = 127
        one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
        out = mamba.int8_matmul(a, b, one(M), one(N), out_dtype=torch.float32)
        assert (out[:, :-1] == float(16384 * K)).all()
        assert (out[:, -1] == float(torch.tensor(-128.0 * 127 * K, dtype=torch.float32))).all()


def test_empty_sizes():
    import torch
    import selective_state_space_80_amd as mamba
    e = lambda *s: torch.empty(s, dtype=torch.int8, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    assert mamba.int8_matmul(e(0, 64), e(5, 64), f(0), f(5)).shape == (0, 5)
    assert mamba.int8_matmul(e(5, 64), e(0, 64), f(5), f(0)).shape == (5, 0)
    for M, N in [(1, 40), (40, 50), (300, 300)]:
        out = torch.full((M, N), 7.0, device="cuda")
        mamba.int8_matmul(e(M, 0), e(N, 0), f(M), f(N), out=out, out_dtype=torch.float32)
        assert not out.any()


@pytest.mark.parametrize("M,N,K", [(1, 70, 256), (20, 90, 512), (200, 190, 256), (600, 520, 640), (1100, 1030, 1024)])
def test_unaligned_storage(M, N, K):
    """Operands and output that start at any element of their storage; nothing
    is written outside the output."""
    import torch
    import selective_state_space_80_amd as mamba
    fa, sa = _operand((M * K + 16, ), 5)
    fb, _ = _operand((N * K + 16, ), 6)
    sa, sb = torch.rand(M + 1, device="cuda")[1:], torch.rand(N + 1, device="cuda")[1:]
    for oa, ob in [(0, 3), (1, 0), (7, 9), (8, 8), (4, 0)]:
        a, b = fa[oa:oa + M * K].view(M, K), fb[ob:ob + N * K].view(N, K)
        for dt, tol in ((torch.float32, F32_TOL), (torch.bfloat16, BF16_TOL)):
            pad = torch.full((M * N + 64,), 3.0, dtype=dt, device="cuda")
            out = pad[5:5 + M * N].view(M, N)
            mamba.int8_matmul(a, b, sa, sb, out_dtype=dt, out=out)
            want = _want(a, b, sa, sb)
            assert ((out.double() - want).abs() <= tol * want.abs()).all(), (oa, ob, dt)
            assert (pad[:5] == 3).all() and (pad[5 + M * N:] == 3).all()


@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (30, 40, 100), (600, 600, 256)])
def test_special_scales(M, N, K):
    """A NaN scale makes its row NaN, a zero scale its row zero, and no other."""
    import torch
    import selective_state_space_80_amd as mamba
    a, sa = _operand((M, K), 8)
    b, sb = _operand((N, K), 9)
    sb[3], sb[7] = float("nan"), 0.0
    out = mamba.int8_matmul(a, b, sa, sb, out_dtype=torch.float32)
    assert torch.isnan(out[:, 3]).all() and (out[:, 7] == 0).all()
    assert torch.isfinite(out[:, :3]).all() and torch.isfinite(out[:, 8:]).all()


def test_offsets_past_32_bits():
    """An output of more than 2^31 elements, and an operand of more than 2^31 bytes."""
    import torch
    import selective_state_space_80_amd as mamba
    for M, N, K in [(70000, 33000, 48), (33000, 40, 70000)]:
        a, sa = _operand((1, K), 12)
        a = a.expand(M, K).contiguous()
        a[-1] = -a[-1].clamp_min(-127)
        sa = torch.linspace(0.5, 1.5, M, device="cuda")
        b, sb = _operand((N, K), 13)
        out = mamba.int8_matmul(a, b, sa, sb)
        rows = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
        want = _want(a[rows], b, sa[rows], sb)
        assert ((out[rows].double() - want).abs() <= BF16_TOL * want.abs()).all(), (M, N, K)
        del out
        torch.cuda.empty_cache()


def test_same_bits_and_other_stream():
    import torch
    import selective_state_space_80_amd as mamba
    for M, N, K in [(1, 2560, 2560), (40, 512, 5120), (256, 2560, 5120), (1000, 1000, 500)]:
        a, sa = _operand((M, K), 15)
        b, sb = _operand((N, K), 16)
        want = mamba.int8_matmul(a, b, sa, sb)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = mamba.int8_matmul(a, b, sa, sb)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got, want)


def test_refusals():
    import torch
    import selective_state_space_80_amd as mamba
    a, sa = _operand((4, 64), 1)
    b, sb = _operand((6, 64), 2)
    with pytest.raises(ValueError):
        mamba.int8_matmul(a, b[:, :32].contiguous(), sa, sb)
    with pytest.raises(ValueError):
        mamba.int8_matmul(a, b, sa[:3].contiguous(), sb)
    with pytest.raises(TypeError):
        mamba.int8_matmul(a.to(torch.uint8), b, sa, sb)
    with pytest.raises(TypeError):
        mamba.int8_matmul(a, b, sa.double(), sb)
    with pytest.raises(TypeError):
        mamba.int8_matmul(a, b, sa, sb, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mamba.int8_matmul(a.t(), b.t(), sa, sb)
    with pytest.raises(ValueError):
        mamba.int8_matmul(a.cpu(), b.cpu(), sa.cpu(), sb.cpu())
    with pytest.raises(ValueError):
        mamba.int8_matmul(a[None].expand(3, 4, 64).contiguous(), b[None].expand(2, 6, 64).contiguous(), sa, sb)
    big = torch.zeros((1, 131072), dtype=torch.int8, device="cuda")
    one = torch.ones(1, device="cuda")
    with pytest.raises(mamba.MambaError):
        mamba.int8_matmul(big, big, one, one)
