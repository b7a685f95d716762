"""Sizes of the gated delta rule whose workspace is past what its size can hold: refused, not wrapped
around.  No device is touched."""
import ctypes

import pytest

from xlstm_mlstm_matrix_amd import binding as B

OK, SHAPE = 0, 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from xlstm_mlstm_matrix_amd import build
        build.build()
    return B.lib()


def query(backward, *dims):
    n = ctypes.c_size_t(0)
    f = B.lib().mlstm_deltarule_bwd_workspace_size if backward else B.lib().mlstm_deltarule_fwd_workspace_size
    return f(*dims, ctypes.byref(n)), n.value


@pytest.mark.parametrize("heads", [524287, 524286, 524285, 524284, 500001, 467003, 262144, 70000])
def test_workspaces_of_2_to_the_64_bytes(heads):
    """Float32 gradients of heads of 256 x 512 keep 1193984 bytes a chunk of 32 tokens: at the least
    number of chunks that make 2^64 bytes, and around it, the sum in 64 bits is small."""
    per = 1193984
    for more in range(-2, 3):
        nch = min(-(-(1 << 64) // (heads * per)) + more, 1 << 25)
        for io in (0, 1):
            for back in (False, True):
                for T in (32 * nch, 32 * nch - 31):
                    assert query(back, heads, 1, 1, T, 256, 512, io)[0] == SHAPE
                    assert query(back, 1, heads, heads, T, 256, 512, io)[0] == SHAPE


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("back", [False, True])
def test_limit_is_2_to_the_40_bytes(io, back):
    """The longest sequences that pass need 2^40 bytes or little less, one chunk more is refused."""
    for heads, dk, dv in ((524287, 16, 16), (4096, 256, 512), (300, 64, 64)):
        lo, hi = 1, 1 << 25
        while lo < hi:
            mid = (lo + hi + 1) // 2
            if query(back, heads, 1, 1, 32 * mid, dk, dv, io)[0] == OK:
                lo = mid
            else:
                hi = mid - 1
        status, n = query(back, heads, 1, 1, 32 * lo, dk, dv, io)
        assert status == OK and n <= 1 << 40
        if lo < 1 << 25:
            assert query(back, heads, 1, 1, 32 * lo + 1, dk, dv, io)[0] == SHAPE
            # a sequence's bytes grow by whole blocks of two chunks
            assert n * (lo + 2) >= (1 << 40) * lo
