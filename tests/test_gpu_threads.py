"""GPU: the feed-forward operators called from several threads at once, each on
a stream of its own, with sizes that share cached plans and sizes that do not."""
import threading

import pytest

import selective_state_space_mamba_amd as ms

from ffutil import maker, rows8, weights4
from scanutil import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch().cuda.empty_cache()


def work(seed, M, K, N, dtype):
    """A program of every operator on its own inputs; returns a function that runs it."""
    t = torch()
    n = maker(seed)
    x, res, w, wg, wu = n((M, K), dtype), n((M, K), dtype), n((K,)), n((N, K), dtype, K ** -0.5), n((N, K), dtype, K ** -0.5)
    dout = n((M, N), dtype)
    w8, sw = rows8(n((N, K)))
    q4 = weights4(N, K, 32, seed, True)[:3]

    def run():
        h, s, rstd = ms.rms_norm_fwd(x, w, res)
        out, pre = ms.gated_linear_fwd(h, wg, wu, want_pre=True)
        g = ms.gated_linear_bwd(h, wg, wu, dout=dout, pre=pre)
        gn = ms.rms_norm_bwd(s, w, dout=g["dx"], rstd=rstd, dadded=res)
        q, scale, _ = ms.rms_norm_q8(x, w, res)
        return [out, scale, ms.linear_q8(q, scale, w8, sw), ms.linear_q4(h, *q4, group=32)] + list(g.values()) + list(gn.values())

    return run


def test_four_threads():
    t = torch()
    runs = [work(1, 300, 96, 264, "bf16"), work(2, 300, 96, 264, "bf16"), work(3, 5, 160, 72, "f32"), work(4, 1500, 64, 520, "f32")]
    want = [[v.clone() for v in r()] for r in runs]
    t.cuda.synchronize()
    bad = []

    def loop(k):
        try:
            s = t.cuda.Stream()
            with t.cuda.stream(s):
                for i in range(30):
                    got = runs[k]()
                    s.synchronize()
                    if not all(t.equal(a, b) for a, b in zip(got, want[k])):
                        bad.append((k, i))
        except Exception as e:  # noqa: BLE001
            bad.append((k, repr(e)))

    threads = [threading.Thread(target=loop, args=(k,)) for k in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad, bad
