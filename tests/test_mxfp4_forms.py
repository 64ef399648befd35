"""Sizes that take every form of the 4-bit product; for the tile forms with at most one
tile a workgroup and with several, which run the loads across a tile's end; inner sizes of
one group of 256 and of several.  On the CPU the list is held against the choice itself, so
that a new fit cannot drop a path from it; on the GPU every element is compared with 64
bits, within the bound that mxfp4_check.py derives, and the memory around the output is
looked at."""
import pytest

from scan_check import say

import mxfp4_check as C
import selective_state_space_80_amd as mamba

TILES = range(4)    # forms that are tiles; 4..12 are rings
A, B = mamba.MXFP4_SHARED_A, mamba.MXFP4_SHARED_B

# (form, several tiles a workgroup): (batch, M, N, K, shared operand)
SIZES = {
    (0, False): [(2, 473, 13500, 922, 0), (1, 2437, 5000, 1114, 0)],
    (0, True): [(40, 758, 812, 993, B), (1, 8267, 7165, 336, 0)],
    (1, False): [(1, 5, 33288, 1886, 0), (1, 112, 48965, 100, 0), (1, 3345, 1220, 26, 0)],
    (1, True): [(40, 33285, 1, 57, 0), (40, 73, 2013, 3731, A), (40, 3197, 187, 302, A), (1, 1206, 8569, 695, 0)],
    (2, False): [(40, 3, 516, 14, 0), (1, 2620, 1441, 4533, 0), (2, 5100, 255, 491, A)],
    (3, False): [(1, 23826, 10, 56, 0), (1, 701, 2216, 2490, 0), (1, 3143, 389, 2, 0)],
    (3, True): [(2, 45093, 26, 34, A), (40, 6541, 9, 847, 0), (2, 38527, 4, 3, A)],
    (4, False): [(1, 5143, 154, 1006, 0), (3, 1644, 179, 233, B), (1, 149, 4250, 147, 0)],
    (5, False): [(3, 70, 2121, 51, 0), (1, 248, 5379, 5985, 0), (1, 4544, 115, 198, 0)],
    (6, False): [(2, 7800, 37, 72, 0), (40, 321, 74, 2959, B), (2, 3497, 77, 452, 0)],
    (7, False): [(2, 10, 5258, 407, A), (40, 27, 327, 4, B), (3, 19, 6217, 11, B)],
    (8, False): [(40, 208, 9, 228, 0), (2, 4305, 11, 1357, 0), (40, 306, 7, 53, B)],
    (9, False): [(1, 229, 612, 2, 0), (1, 31, 8000, 538, 0), (1, 32, 4723, 11, 0)],
    (10, False): [(1, 2, 5442, 216, 0), (1, 1, 16412, 3744, 0), (1, 3434, 17, 67, 0)],
    (11, False): [(1, 6820, 4, 1326, 0), (2, 1074, 38, 3, A), (1, 8012, 3, 112, 0)],
    (12, False): [(2, 1, 652, 7, 0), (1, 44, 1, 3432, 0), (1, 30, 243, 1, 0)],
}
CASES = [(key, *size) for key, sizes in SIZES.items() for size in sizes]


def test_every_path_has_sizes():
    # 128 x 128 in four stages are taken for few tiles only
    assert set(SIZES) == {(f, several) for f in range(13) for several in ((False, True) if f in TILES else (False,))} - {(2, True)}


@pytest.mark.parametrize("key,batch,M,N,K,shared", CASES)
def test_size_takes_its_path(key, batch, M, N, K, shared):
    form, tiles, slots = mamba.mxfp4_matmul_form(M, N, K, batch, shared)
    assert (form, form in TILES and tiles > slots) == key


def test_form_of_empty_and_refused_products():
    for empty in (dict(M=0, N=5, K=64), dict(M=3, N=5, K=0), dict(M=3, N=5, K=64, batch=0)):
        assert mamba.mxfp4_matmul_form(**empty) == (-1, 0, 0)
    for bad in (dict(M=-1, N=1, K=1), dict(M=1, N=1, K=(1 << 23) + 1), dict(M=1, N=1, K=1, flags=4)):
        with pytest.raises(mamba.MambaError):
            mamba.mxfp4_matmul_form(**bad)


@pytest.mark.gpu
@pytest.mark.parametrize("key,batch,M,N,K,shared", CASES)
def test_product(key, batch, M, N, K, shared):
    import torch
    say(f"4-bit product form={key[0]} several={key[1]} batch={batch} {M}x{N}x{K} shared={shared}")
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    groups, table = C.groups(K), torch.cat([C.VALUES, -C.VALUES]).cuda()

    def operand(rows, flag):
        lead = (batch,) if batch > 1 and not shared & flag else ()
        q = torch.randint(0, 256, (*lead, rows, groups * 128), generator=g, device="cuda", dtype=torch.uint8)
        q[..., -(-K // 2):] = 0
        if K % 2:
            q[..., K // 2] &= 15
        return q, torch.randint(121, 134, (groups, *lead, rows, 8), generator=g, device="cuda", dtype=torch.uint8)

    def values(q, s, i):
        q, s = (q[i], s[:, i]) if q.dim() == 3 else (q, s)
        codes = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
        power = torch.exp2(s.movedim(0, -2).flatten(-2).double() - 127)
        return table[codes] * power.repeat_interleave(32, -1)

    (a, sa), (b, sb) = operand(M, A), operand(N, B)
    for dt, half_step in ((torch.float32, C.U), (torch.bfloat16, 2.0 ** -8)):
        # guard bands around the output
        count = batch * M * N
        room = torch.full((count + 128,), 3.0, dtype=dt, device="cuda")
        out = room[64:64 + count].view(*((batch,) if batch > 1 else ()), M, N)
        mamba.mxfp4_matmul(a, b, sa, sb, out_dtype=dt, out=out)
        assert bool((room[:64] == 3).all()) and bool((room[64 + count:] == 3).all())
        for i in range(batch):
            va, vb = values(a, sa, i), values(b, sb, i)
            want = va @ vb.t()
            bad = (out[i] if batch > 1 else out).double().sub(want).abs() > C.product_bound(va, vb, want, half_step)
            assert not bool(bad.any()), f"{dt} batch {i}: {int(bad.sum())} wrong, first {bad.nonzero()[0].tolist()}"
