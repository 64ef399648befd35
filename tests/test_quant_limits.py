"""CPU checks of the sizes that the norm, the quantiser and the 8-bit product
take: what is refused is what no launch can hold, and nothing else.  An accepted
size goes on to the check for NULL, which stops every call here."""
import ctypes

import pytest

import selective_state_space_80_amd as mamba

F32, BF16 = mamba.MAMBA_F32, mamba.MAMBA_BF16
OK, ENULL, ESHAPE = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    return mamba.load_library()


def _p(k):
    return ctypes.c_void_p(k << 40)  # never dereferenced


# Four rows a workgroup of 256 threads: 2^24 workgroups would have 2^32 threads,
# one more than a launch takes.
@pytest.mark.parametrize("M,D,want", [
    ((1 << 26) - 3, 512, ESHAPE), ((1 << 26) - 1, 4096, ESHAPE), ((1 << 26) - 4, 512, ENULL),
    ((1 << 26) - 4, 4096, ENULL), ((1 << 22) - 1, 4097, ENULL), (1 << 22, 4097, ESHAPE)])
def test_rows(lib, M, D, want):
    assert lib.mamba_rms_norm(None, None, _p(3), _p(4), None, M, D, 1e-5, BF16, F32, None) == want
    assert lib.mamba_rms_norm_int8(None, None, _p(3), _p(4), _p(5), None, M, D, 1e-5, F32, F32, None) == want
    assert lib.mamba_quantize_int8(None, _p(2), _p(3), 1, M, D, 0, BF16, None) == want


def product(lib, batch, M, N, K, flags=0):
    return lib.mamba_int8_matmul(_p(1), _p(2), _p(3), None, _p(5), batch, M, N, K, BF16, flags, None)


A, B = mamba.INT8_SHARED_A, mamba.INT8_SHARED_B


# The limit is on tiles of 128 x 64 outputs a batch, 2^30 (32-bit tile numbers);
# batches of one right operand are one batch.
@pytest.mark.parametrize("batch,M,N,K,flags,want", [
    (1 << 24, 0, 64, 64, 0, OK), (1 << 24, 64, 0, 64, 0, OK), (1 << 24, 64, 0, 0, A, OK),      # nothing to do
    (1, 1 << 27, 1 << 10, 64, 0, ENULL), (5000000, 1, 1, 64, 0, ENULL), (1 << 23, 1, 64, 64, B, ENULL),
    (1 << 23, 1, 64, 64, A, ENULL), (100000, 1, 5120, 2560, B, ENULL), (100000, 5120, 1, 2560, A, ENULL),
    (1, 1 << 36, 1, 1, 0, ENULL), (1, 1 << 38, 1, 1, 0, ESHAPE), (1, 1, 1 << 38, 1, 0, ESHAPE),
    (1 << 19, 1 << 19, 1, 1, B, ESHAPE), (1 << 19, 1 << 19, 1, 1, 0, ENULL),
    (1, 1 << 21, 1 << 20, 1, 0, ESHAPE), (100000, 5120, 1, 2560, 0, ESHAPE)])
def test_product_sizes(lib, batch, M, N, K, flags, want):
    assert product(lib, batch, M, N, K, flags) == want
