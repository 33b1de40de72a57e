"""GPU: the product with 4-bit weights over as many rows as it takes, and rows
and outputs of more than 2^31 elements: every row as in a call of its own few."""
import pytest

import selective_state_space_mamba_amd as ms

from ffutil import close, dtype_of, maker, mm, weights4
from scanutil import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch().cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N,group", [(1 << 18, 96, 8200, 32), (1 << 18, 8224, 8, 128), (4099, 1056, 264, 64)])
def test_many_rows(M, K, N, group, dtype):
    """The same 40 rows over and over.  (Both calls' tiles sum a column's products in the same order.)"""
    t = torch()
    print("[gpu case] q4 rows", M, K, N, dtype, flush=True)
    n = maker(M % 1000 + K)
    part, b = n((40, K), dtype), n((N,), std=0.2)
    q, scale, z, w = weights4(N, K, group, K, True)
    few = ms.linear_q4(part, q, scale, z, b, group=group, act=ms.ACT_SILU)
    u = mm(part, w) + b.double()
    close("few", few, u * t.sigmoid(u), dtype)
    x = t.empty(M, K, dtype=dtype_of(dtype), device="cuda:0")
    whole = M // 40 * 40
    x[:whole].view(-1, 40, K)[:] = part
    x[whole:] = part[:M - whole]
    got = ms.linear_q4(x, q, scale, z, b, group=group, act=ms.ACT_SILU)
    assert t.equal(got[:whole].view(-1, 40, N), few.expand(whole // 40, 40, N)) and t.equal(got[whole:], few[:M - whole])
    res = got.clone()
    twice = ms.linear_q4(x, q, scale, z, b, res, group=group, act=ms.ACT_SILU, out=res)
    assert twice is res and t.equal(res, (got.float() + got.float()).to(got.dtype))
