"""Sizes that take every form of the 8-bit product, by loads straight into LDS
(16-byte aligned rows) and by way of registers; for the tile forms with at most
one tile a workgroup and with several, which run the loads across a tile's end,
each with inner sizes of few and of many steps that end inside one.  On the CPU
the list is held against the choice itself, so that a new fit cannot drop a path
from it; on the GPU every element is compared with the formula in 64 bits.  The
sum is exact, its conversion to fp32 and the two scalings round three times; a
bf16 output adds half a unit, at most 2^-8."""
import pytest

from scan_check import say

import selective_state_space_80_amd as mamba

F32_TOL = 3.01 * 2.0 ** -24
BF16_TOL = F32_TOL + 2.0 ** -8
TILES = range(4)    # forms that are tiles; 4..12 are rings
A, B = mamba.INT8_SHARED_A, mamba.INT8_SHARED_B

# (form, aligned, several tiles a workgroup): (batch, M, N, K, shared operand)
SIZES = {
    (0, True, False): [(1, 6027, 1298, 1392, 0), (9, 2561, 300, 1488, A)],
    (0, True, True): [(1, 727, 43372, 688, 0), (3, 4000, 2500, 1008, A)],
    (1, True, False): [(1, 12513, 288, 960, 0), (1, 654, 5832, 32, 0), (130, 140, 90, 3600, 0)],
    (1, True, True): [(1, 3605, 2973, 608, 0), (1, 3703, 2972, 16, 0), (3, 5000, 700, 912, 0), (600, 33, 70, 96, 0),
                      (270, 130, 190, 3600, A)],
    (1, False, False): [(1, 709, 5429, 843, 0), (1, 50601, 87, 6, 0), (80, 300, 200, 700, 0)],
    (1, False, True): [(1, 33257, 136, 412, 0), (1, 1210, 10022, 1, 0), (40, 1030, 300, 3000, A), (300, 200, 70, 1000, 0)],
    (2, True, False): [(1, 7959, 334, 560, 0), (1, 4278, 517, 16, 0), (1, 129, 8400, 432, 0)],
    (2, True, True): [(1, 66233, 65, 3136, 0), (1, 65788, 117, 2960, 0), (1, 71449, 72, 5568, 0)],
    (2, False, False): [(1, 27005, 94, 522, 0), (1, 1461, 1428, 8, 0), (1, 144, 8222, 437, 0)],
    (3, True, False): [(1, 5878, 229, 592, 0), (1, 6176, 186, 16, 0), (1, 8730, 65, 400, 0)],
    (3, True, True): [(1, 76707, 14, 464, 0), (1, 66053, 10, 144, 0), (2, 36043, 31, 192, B)],
    (3, False, False): [(1, 1581, 1031, 485, 0), (1, 3261, 311, 4, 0), (1, 8300, 67, 433, 0)],
    (3, False, True): [(1, 56821, 64, 3464, 0), (1, 110002, 64, 3464, 0), (1, 64021, 4, 3, 0), (1, 119088, 2, 433, 0)],
    (4, True, False): [(1, 101, 6194, 432, 0), (1, 145, 4118, 16, 0)],
    (4, False, False): [(1, 6547, 98, 398, 0)],
    (5, True, False): [(1, 8830, 33, 416, 0), (1, 8297, 33, 16, 0), (140, 140, 190, 3600, 0)],
    (5, False, False): [(1, 2745, 167, 404, 0), (1, 8584, 34, 1, 0)],
    (6, True, False): [(1, 6325, 78, 400, 0), (1, 6185, 67, 16, 0)],
    (6, False, False): [(1, 6498, 66, 397, 0), (1, 12654, 33, 1, 0)],
    (7, True, False): [(1, 4405, 33, 416, 0), (1, 33, 4163, 16, 0)],
    (7, False, False): [(1, 740, 351, 386, 0), (1, 33, 5497, 1, 0)],
    (8, True, False): [(1, 8439, 1, 400, 0), (1, 8193, 1, 16, 0)],
    (8, False, False): [(1, 4137, 65, 390, 0), (1, 8590, 17, 1, 0)],
    (9, True, False): [(1, 66, 1662, 400, 0), (1, 4109, 17, 16, 0)],
    (9, False, False): [(1, 211, 597, 401, 0), (1, 17, 4214, 1, 0)],
    (10, True, False): [(1, 674, 86, 400, 0), (1, 1, 4103, 16, 0)],
    (10, False, False): [(1, 66, 882, 395, 0), (1, 1, 4135, 1, 0)],
    (11, True, False): [(1, 4515, 1, 416, 0), (1, 4097, 1, 16, 0)],
    (11, False, False): [(1, 4457, 1, 385, 0), (1, 4146, 1, 1, 0)],
    (12, True, False): [(1, 1, 1, 400, 0), (1, 16, 33, 2064, 0)],
    (12, False, False): [(1, 1, 1, 385, 0), (1, 9, 17, 1001, 0)],
}
CASES = [(key, *size) for key, sizes in SIZES.items() for size in sizes]


def test_every_path_has_sizes():
    # 256 x 256 tiles are for aligned rows; 128 x 128 in four stages by way of
    # registers are taken for few tiles only
    never = {(0, False, False), (0, False, True), (2, False, True)}
    want = {(f, aligned, several) for f in range(13) for aligned in (True, False)
            for several in ((True, False) if f in TILES else (False,))} - never
    assert set(SIZES) == want


@pytest.mark.parametrize("key,batch,M,N,K,shared", CASES)
def test_size_takes_its_path(key, batch, M, N, K, shared):
    form, tiles, slots = mamba.int8_matmul_form(M, N, K, batch, K % 16 == 0, shared)
    assert (form, K % 16 == 0, form in TILES and tiles > slots) == key


def test_form_of_empty_and_refused_products():
    assert mamba.int8_matmul_form(0, 5, 64) == (-1, 0, 0) and mamba.int8_matmul_form(3, 5, 64, batch=0) == (-1, 0, 0)
    for bad in (dict(M=-1, N=1, K=1), dict(M=1, N=1, K=131072), dict(M=1, N=1, K=1, flags=4)):
        with pytest.raises(mamba.MambaError):
            mamba.int8_matmul_form(**bad)


@pytest.mark.gpu
@pytest.mark.parametrize("key,batch,M,N,K,shared", CASES)
def test_product(key, batch, M, N, K, shared):
    import torch
    say(f"product form={key[0]} aligned={key[1]} several={key[2]} batch={batch} {M}x{N}x{K} shared={shared}")
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)

    def operand(rows, flag):
        lead = (batch,) if batch > 1 and not shared & flag else ()
        q = torch.randint(-128, 128, (*lead, rows, K), generator=g, device="cuda", dtype=torch.int8)
        return q, torch.rand((*lead, rows), generator=g, device="cuda") * 0.1 + 0.001

    (a, sa), (b, sb) = operand(M, A), operand(N, B)
    of = lambda t, flag, i: t[i].double() if batch > 1 and not shared & flag else t.double()  # noqa: E731
    for dt, tol in ((torch.float32, F32_TOL), (torch.bfloat16, BF16_TOL)):
        # guard bands around the output
        count = batch * M * N
        room = torch.full((count + 128,), 3.0, dtype=dt, device="cuda")
        out = room[64:64 + count].view(*((batch,) if batch > 1 else ()), M, N)
        mamba.int8_matmul(a, b, sa, sb, out_dtype=dt, out=out)
        assert bool((room[:64] == 3).all()) and bool((room[64 + count:] == 3).all())
        for i in range(batch):
            want = of(a, A, i) @ of(b, B, i).t() * of(sa, A, i)[:, None] * of(sb, B, i)
            got = (out[i] if batch > 1 else out).double()
            bad = ~((got - want).abs() <= tol * want.abs())
            assert not bool(bad.any()), f"{dt} batch {i}: {int(bad.sum())} wrong, first {bad.nonzero()[0].tolist()}"
