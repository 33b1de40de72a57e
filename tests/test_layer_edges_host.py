"""Host-side checks of the operators around the scan at the edges of what they
take (no GPU work: every call below fails validation before any launch)."""
import ctypes
import os

import pytest

import selective_state_space_mamba_amd as ms
from selective_state_space_mamba_amd import _binding as E

FAKE = 0x100000  # 16-byte aligned stand-in pointer


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ms.LIB_PATH):
        from selective_state_space_mamba_amd import build
        build.build(force=False)
    return ms.load_library()


def test_glr_alignment_of_batch_slices(lib):
    """bfloat16 rows of 8k + 4 channels are a multiple of 8 bytes, not of 16: so far may an item begin.  (The sizes
    need a workspace that is not given: the call is refused for that, and only once the pointers have passed.)"""
    def fwd(dim, dtype, off):
        d = ms.make_glr_dims(1, 1000, dim, dtype)
        p = FAKE + off
        return lib.mamba_glr_fwd(p, p, p, p, FAKE, ctypes.byref(d), p, FAKE, None, 0, None)

    def bwd(dim, dtype, off):
        d = ms.make_glr_dims(1, 1000, dim, dtype)
        p = FAKE + off
        return lib.mamba_glr_bwd(p, p, p, p, FAKE, p, FAKE, ctypes.byref(d), p, p, p, p, FAKE, FAKE, None, 0, None)

    for call in (fwd, bwd):
        assert call(68, ms.DTYPE_BF16, 8) == E.MAMBA_ERR_WORKSPACE
        assert call(68, ms.DTYPE_BF16, 4) == E.MAMBA_ERR_UNSUPPORTED
        assert call(64, ms.DTYPE_BF16, 8) == E.MAMBA_ERR_UNSUPPORTED
        assert call(68, ms.DTYPE_F32, 8) == E.MAMBA_ERR_UNSUPPORTED
        assert call(68, ms.DTYPE_F32, 16) == E.MAMBA_ERR_WORKSPACE


def test_linear_tiles_are_all_run(lib):
    """The sizes that test_gpu_linear_tiles runs reach each tile in each operand layout, whole and in shares."""
    from linear_tiles import CASES, sizes
    seen = set()
    for product, m, n, k, tile, shared in CASES:
        M, K, N = sizes(product, m, n, k)
        rows, cols, shares = ms.linear_plan(ms.make_linear_dims(M, K, N, ms.DTYPE_BF16), product)
        assert ((rows, cols), shares > 1) == (tile, shared), (product, m, n, k, rows, cols, shares)
        seen.add((product, tile, shared))
    assert len(seen) == 3 * 3 * 2


def test_linear_plan(lib):
    def plan(M, K, N, product=0, **kw):
        return ms.linear_plan(ms.make_linear_dims(M, K, N, kw.pop("dtype", ms.DTYPE_BF16), **kw), product)

    assert [plan(M, 64, 64)[:2] for M in (1, 16, 17, 32, 33, 64, 65)] == [
        (16, 16), (16, 16), (32, 16), (32, 16), (64, 16), (64, 16), (128, 128)]
    assert plan(16384, 768, 1536, dtype=ms.DTYPE_F32) == (128, 128, 1)
    for bad in (dict(product=3), dict(product=-1), dict(act=9)):
        with pytest.raises(ms.MambaError):
            plan(8, 64, 64, **bad)
    with pytest.raises(ms.MambaError):
        plan(8, 60, 64)
    assert lib.mamba_linear_plan(None, 0, None, None, None) == E.MAMBA_ERR_INVALID
