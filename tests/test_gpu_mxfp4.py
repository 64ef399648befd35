"""GPU checks of the microscaled 4-bit format against 64 bits (mxfp4_check.py): the
quantiser's and the way back's every bit, the product within its sums' rounding."""
import pytest
import torch

import mxfp4_check as C
from scan_check import say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF_STEP = {F32: C.U, BF16: 2.0 ** -8}


def _mamba():
    import selective_state_space_80_amd as mamba
    return mamba


def _check_quantised(x, **kw):
    """x on the GPU, token-major; every byte of both outputs."""
    q, scale = _mamba().quantize_mxfp4(x, **kw)
    token_major = x.transpose(1, 2) if kw.get("channel_major") else x
    want_q, want_scale = C.pack(*C.encode(token_major))
    assert torch.equal(scale.cpu(), want_scale), "scales"
    assert torch.equal(q.cpu(), want_q), "elements"
    return q, scale


def _normal(shape, io, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen) * torch.exp2(torch.randint(-20, 20, (*shape[:-1], 1), generator=gen).float())
    return x.to(io).cuda()


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("K", [1, 7, 8, 31, 32, 33, 255, 256, 257, 300, 520, 1001, 2560])
@pytest.mark.parametrize("rows", [1, 3, 8, 33])
def test_quantise_rows(io, K, rows):
    say(f"quantise {rows} x {K} {io}")
    _check_quantised(_normal((rows, K), io, K))


@pytest.mark.parametrize("io", [F32, BF16])
def test_quantise_many_rows(io):
    say(f"quantise many rows {io}")
    _check_quantised(_normal((4101, 2100), io, 1))


@pytest.mark.parametrize("io", [F32, BF16])
def test_quantise_every_border(io):
    """Blocks topped by each value from 1 to 8 in 16ths; beside it values in 32nds, ties and their
    neighbours among them, at exponents over the type's whole range."""
    say(f"quantise borders {io}")
    fine = torch.arange(0, 8, 1 / 32)
    rows = []
    for top in torch.arange(1, 8, 1 / 16):
        part = fine[fine <= top]
        part = torch.nn.functional.pad(part, (0, -len(part) % 31)).view(-1, 31)
        rows.append(torch.cat([top.expand(len(part), 1), part], 1))
    blocks = torch.cat(rows)
    blocks = torch.cat([blocks, -blocks])
    for exponent in (-148, -133, -130, -128, -127, -126, -125, -124, -120, -3, 0, 5, 100, 124):
        x = torch.ldexp(blocks.double(), torch.tensor(float(exponent), dtype=torch.float64)).float().to(io)
        assert torch.isfinite(x).all()
        _check_quantised(x.cuda())
    ulp = torch.nextafter(blocks, torch.tensor(torch.inf))
    for x in (ulp, torch.nextafter(blocks, torch.tensor(-torch.inf))):
        _check_quantised(x.to(io).cuda())


@pytest.mark.parametrize("seed", [0, 1])
def test_quantise_every_bf16(seed):
    """Every bf16 bit pattern, in blocks by size and in any order."""
    say("quantise every bf16")
    bits = torch.arange(1 << 16, dtype=torch.int32)
    order = (bits * 2 ** 16 % 65521) if seed == 0 else torch.randperm(1 << 16, generator=torch.Generator().manual_seed(1))
    x = bits.to(torch.int16).view(BF16)
    x = x[order.long() % (1 << 16)].view(-1, 1024)
    q, scale = _mamba().quantize_mxfp4(x.cuda())
    codes, scales = C.encode(x)
    want_q, want_scale = C.pack(codes, scales)
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(q.cpu(), want_q)
    _check_quantised(x.float().cuda())


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("channel_major", [False, True])
def test_quantise_special_blocks(io, channel_major):
    x = _normal((2, 70, 300), io, 3)
    x[0, 0, :32] = 0.0
    x[0, 1, 5] = torch.nan
    x[0, 2, 40] = torch.inf
    x[0, 3, 299] = -torch.inf
    x[1, 4] = torch.nan
    x[1, 5] = torch.finfo(io).max
    x[1, 6] = torch.finfo(io).tiny
    x[1, 7] = 0.0
    x[1, 8, ::2] = -0.0
    q, scale = _check_quantised(x.transpose(1, 2).contiguous() if channel_major else x, channel_major=channel_major)
    assert scale[0, 0, 1, 0] == 255 and scale[0, 0, 1, 1] != 255 and scale[0, 0, 2, 1] == 255 and scale[1, 0, 3, 1] == 255
    back = _mamba().dequantize_mxfp4(q, scale, 300, dtype=F32)
    assert torch.isnan(back[0, 1, :32]).all() and not torch.isnan(back[0, 1, 32:]).any()


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("L", [1, 2, 3, 31, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("B,K", [(1, 256), (2, 33), (3, 515)])
def test_quantise_channel_major(io, L, B, K):
    say(f"quantise channel-major {B} x {K} x {L} {io}")
    gen = torch.Generator().manual_seed(L)
    _check_quantised(torch.randn((B, K, L), generator=gen).to(io).cuda(), channel_major=True)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("channel_major", [False, True])
def test_quantise_from_any_address(io, channel_major):
    for off in (1, 2, 3, 5):
        buffer = torch.randn(3 * 37 * 290 + off, generator=torch.Generator().manual_seed(off)).to(io).cuda()
        _check_quantised(buffer[off:].view(3, 37, 290), channel_major=channel_major)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 33), (8, 256), (9, 300), (70, 1000), (1000, 2560)])
def test_dequantise(out, rows, K):
    q, scale = C.random_operand((), rows, K, K, low=-20, high=20)
    got = _mamba().dequantize_mxfp4(q.cuda(), scale.cuda(), K, dtype=out)
    assert got.dtype == out and torch.equal(got.double().cpu(), C.values(q, scale)[:, :K])


@pytest.mark.parametrize("out", [F32, BF16])
def test_dequantise_every_byte_and_scale(out):
    """Each element code with each scale code: 256 scales a row, rows of every byte."""
    q = torch.arange(256, dtype=torch.uint8).repeat(16).view(32, 128).repeat(8, 1)
    scale = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 8)[None]
    got = _mamba().dequantize_mxfp4(q.cuda(), scale.contiguous().cuda(), dtype=out)
    want = C.values(q, scale)
    limit = torch.finfo(out).max
    want = torch.where(want.abs() > limit, torch.copysign(torch.tensor(torch.inf, dtype=torch.float64), want), want)
    assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
    assert torch.equal(got.double().cpu().nan_to_num(0.0, 1e300, -1e300), want.nan_to_num(0.0, 1e300, -1e300))


def _check_product(a_lead, b_lead, M, N, K, out, seed=0, low=-6, high=6):
    say(f"product {a_lead} {M} x {b_lead} {N} x {K} {out}")
    a, sa = C.random_operand(a_lead, M, K, seed, low, high)
    b, sb = C.random_operand(b_lead, N, K, seed + 1, low, high)
    va, vb = C.values(a, sa), C.values(b, sb)
    want = va @ vb.mT
    if K == 0:
        want = torch.zeros((*(a_lead or b_lead), M, N), dtype=torch.float64)
    got = _mamba().mxfp4_matmul(a.cuda(), b.cuda(), sa.cuda(), sb.cuda(), out_dtype=out)
    assert got.dtype == out and got.shape == want.shape
    part = ((got.double().cpu() - want).abs() / C.product_bound(va, vb, want, HALF_STEP[out])).max().item()
    say(f"  part of the bound {part:.2f}")
    assert part <= 1.0


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 5120, 2560), (1, 130, 300), (2, 3, 64), (16, 16, 256), (17, 33, 257), (31, 129, 520), (33, 515, 1001),
    (64, 64, 512), (100, 2560, 768), (128, 128, 256), (129, 127, 2304), (256, 2560, 5120), (333, 515, 1001), (1000, 100, 130),
    (513, 1025, 768), (2048, 1536, 256), (1300, 1290, 1300), (3, 8192, 32), (8192, 3, 32)])
def test_product(out, M, N, K):
    _check_product((), (), M, N, K, out)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("a_lead,b_lead", [((3,), (3,)), ((), (3,)), ((3,), ())])
@pytest.mark.parametrize("M,N,K", [(1, 1, 40), (5, 300, 300), (130, 70, 256), (300, 257, 768)])
def test_product_batches(out, a_lead, b_lead, M, N, K):
    _check_product(a_lead, b_lead, M, N, K, out)


def test_product_large():
    _check_product((), (), 4097, 2051, 1280, BF16)


def test_product_range():
    """Scales far apart, products beside 2^100 and 2^-100 that meet in one sum."""
    _check_product((), (), 70, 70, 600, F32, low=-60, high=60)


def test_product_of_no_channels_or_rows():
    _check_product((), (), 5, 7, 0, F32)
    mamba = _mamba()
    empty = torch.empty(0, 128, dtype=torch.uint8, device="cuda")
    scale = torch.empty(1, 0, 8, dtype=torch.uint8, device="cuda")
    b, sb = (t.cuda() for t in C.random_operand((), 3, 256, 1))
    assert mamba.mxfp4_matmul(empty, b, scale, sb).shape == (0, 3)


def test_nan_scales_reach_their_row_only():
    for M, N, K in [(40, 50, 600), (300, 300, 1024), (1, 600, 512)]:
        a, sa = C.random_operand((), M, K, 1)
        b, sb = C.random_operand((), N, K, 2)
        sa[-1, M // 2, 7] = 255
        sb[0, 3, 0] = 255
        got = _mamba().mxfp4_matmul(a.cuda(), b.cuda(), sa.cuda(), sb.cuda(), out_dtype=F32).cpu()
        want = torch.zeros(M, N, dtype=torch.bool)
        want[M // 2] = True
        want[:, 3] = True
        assert torch.equal(torch.isnan(got), want)


def test_quantised_product_is_the_products_of_its_values():
    """The operators in a run: quantise both, multiply; against 64 bits on the dequantised values."""
    mamba = _mamba()
    x, w = _normal((2, 90, 700), BF16, 5), _normal((130, 700), F32, 6)
    (q, s), (wq, ws) = mamba.quantize_mxfp4(x), mamba.quantize_mxfp4(w)
    got = mamba.mxfp4_matmul(q, wq, s, ws, out_dtype=F32)
    vx, vw = (mamba.dequantize_mxfp4(*t, 700, dtype=F32).double().cpu() for t in ((q, s), (wq, ws)))
    want = vx @ vw.t()
    assert ((got.double().cpu() - want).abs() / C.product_bound(vx, vw, want, C.U)).max() <= 1


def test_offsets_past_32_bits():
    """Packed rows beyond 4 GiB, in the quantiser, the way back and both of the product's operands."""
    mamba = _mamba()
    rows = (1 << 25) + 37
    x = torch.zeros(rows, 256, dtype=BF16, device="cuda")
    tail = torch.randn(64, 256, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    x[-64:] = tail
    q, s = mamba.quantize_mxfp4(x)
    del x
    q1, s1 = mamba.quantize_mxfp4(tail)
    assert torch.equal(q[-64:], q1) and torch.equal(s[0, -64:], s1[0])
    assert torch.equal(mamba.dequantize_mxfp4(q, s)[-64:], mamba.dequantize_mxfp4(q1, s1))
    w, sw = mamba.quantize_mxfp4(torch.randn(24, 256, generator=torch.Generator().manual_seed(2)).cuda())
    want = mamba.mxfp4_matmul(q1, w, s1, sw)
    assert torch.equal(mamba.mxfp4_matmul(q, w, s, sw)[-64:], want)
    assert torch.equal(mamba.mxfp4_matmul(w, q, sw, s)[:, -64:], want.t())


def test_one_row_and_the_callers_own_buffers():
    mamba = _mamba()
    x = _normal((700,), F32, 8)
    q, s = mamba.quantize_mxfp4(x)
    assert q.shape == (384,) and s.shape == (3, 8)
    q2, s2 = mamba.quantize_mxfp4(x[None], out=torch.full((1, 384), 9, dtype=torch.uint8, device="cuda"),
                                  scale=torch.full((3, 1, 8), 9, dtype=torch.uint8, device="cuda"))
    assert torch.equal(q2[0], q) and torch.equal(s2[:, 0], s)
    back = mamba.dequantize_mxfp4(q, s, dtype=F32)
    assert back.shape == (768,) and not back[700:].any()
    assert torch.equal(back[:700].cpu().double(), C.values(q, s)[:700])
    out = torch.full((1, 700), 9.0, device="cuda")
    assert mamba.dequantize_mxfp4(q2, s2, 700, dtype=F32, out=out) is out and torch.equal(out[0], back[:700])
    prod = torch.full((1, 1), 9.0, device="cuda")
    assert mamba.mxfp4_matmul(q2, q2, s2, s2, out_dtype=F32, out=prod) is prod
    v = C.values(q2, s2)
    assert ((prod.cpu().double() - v @ v.t()).abs() <= C.product_bound(v, v, v @ v.t(), C.U)).all()
