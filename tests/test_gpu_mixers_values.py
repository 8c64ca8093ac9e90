"""Token mixers on the GPU with values that are not finite, in the masks and gates where what depends on them is narrowest."""
import pytest
import torch

from tests.test_gpu_mixers import DT, win_inputs
from tests.test_gpu_mixers_use import BAD, poisoned, same, window_all

pytestmark = pytest.mark.gpu


@DT
@pytest.mark.parametrize("window,sinks,n", [(1, 4, 1), (17, 70, 20), (3, 40, 30), (5, 1024, 300), (17, 70, 400)])
@pytest.mark.parametrize("H,HK,D,T", [(2, 1, 128, 500), (1, 1, 33, 500), (2, 2, 256, 500), (16, 8, 64, 1100)])
def test_more_first_tokens_than_the_window(dtype, window, sinks, n, H, HK, D, T):
    """A query behind the window comes before some of the first tokens then, and reaches none of those."""
    dev, _ = win_inputs(75, dtype, 1, T, H, HK, D)
    want = window_all(dev, window, sinks)
    t = torch.arange(T, device="cuda")
    sees_n = (t >= n) & ((t - n < window) | (n < sinks))
    seen = (t <= n) & ((n - t < window) | (t < sinks))
    other = t != n
    for value in BAD:
        for name in ("q", "do"):
            got = window_all(poisoned(dev, name, n, value, 1), window, sinks)
            for out in ("o", "dq"):
                same(got[out], want[out], other, name)
            for out in ("dk", "dv"):
                same(got[out], want[out], ~seen, name)
            bad = got["dv"][0, seen, -1] if name == "q" else got["dv"][0, seen, -1, 1]
            assert not bad.isfinite().any()
        for name in ("k", "v"):
            got = window_all(poisoned(dev, name, n, value, 1), window, sinks)
            for out in ("o", "dq"):
                same(got[out], want[out], ~sees_n, name)
