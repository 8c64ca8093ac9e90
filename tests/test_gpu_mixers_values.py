"""Token mixers on the GPU with values that are not finite, in the masks and gates where what depends on them is narrowest."""
import pytest
import torch

from tests.test_gpu_mixers import DT, lin_inputs, win_check, win_inputs
from tests.test_gpu_mixers_use import BAD, linear_all, poisoned, same, window_all

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


@DT
@pytest.mark.parametrize("window", [13, 14, 15, 16, 31, 33])
@pytest.mark.parametrize("D,pad", [(128, 0), (100, 6), (256, 0), (16, 0)])
def test_queries_just_behind_the_window(dtype, window, D, pad):
    """Where the sixteen keys of a tile end among the queries of its first block."""
    T, sinks = 300, 60
    dev, _ = win_inputs(89, dtype, 1, T, 2, 1, D, pad)
    want = window_all(dev, window, sinks)
    t = torch.arange(T, device="cuda")
    for n in (window, window + 1, 31, 32, 44, 45, 46, 47, 48):
        seen = (t <= n) & ((n - t < window) | (t < sinks))
        for name in ("q", "do"):
            got = window_all(poisoned(dev, name, n, float("nan"), 1), window, sinks)
            for out in ("dk", "dv"):
                same(got[out], want[out], ~seen, (name, n))
            assert not (got["dv"][0, seen, -1] if name == "q" else got["dv"][0, seen, -1, 1]).isfinite().any()


@DT
@pytest.mark.parametrize("window,sinks,cu", [(17, 1024, None), (5, 1024, [0, 600, 1500]), (14, 500, None), (100, 1000, [0, 120, 1500])])
def test_parts_that_end_before_a_first_token(dtype, window, sinks, cu):
    """First tokens beyond the first parts' queries."""
    dev, x64 = win_inputs(91, dtype, 1, 1500, 4, 2, 40)
    win_check(dev, x64, dtype, window, sinks, 0.2, cu, 1500, 40)


@DT
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("T,HV,K,V,cu", [(333, 2, 64, 96, None), (333, 1, 40, 33, None), (150, 2, 128, 128, [0, 10, 10, 131, 150]),
                                         (333, 512, 16, 16, None), (600, 256, 16, 16, None)])
def test_gates_that_are_not_finite(dtype, value, T, HV, K, V, cu):
    """A gate reaches what crosses it: its own and later outputs and gradients of q, earlier gradients of k and v. Segments of one
    chunk, of a whole sequence's (512 heads) and two of ten chunks (256 heads). The numbers beside it are those of a gate of zero: any
    other moves the chunk's sums, and with them the rounding (2^-48 of a sum held in two fp32 numbers, 2^-24 of a decay) of differences that do
    not cross it."""
    N = len(cu) - 1 if cu else 1
    dev, _ = lin_inputs(77, dtype, 1, T, HV, HV, K, V, N, True, False)
    for n in (0, 1, 17, 31, 32, 100, 130, T - 1):
        lo, hi = next((a, b) for a, b in zip(cu or [0, T], (cu or [0, T])[1:]) if a <= n < b)
        bad = dict(dev, g=dev["g"].clone())
        bad["g"][0, n, -1] = 0.0
        want = linear_all(bad, cu)
        bad["g"][0, n, -1] = value
        got = linear_all(bad, cu)
        own = torch.zeros(T, dtype=torch.bool, device="cuda")
        own[lo:hi] = True
        t = torch.arange(T, device="cuda")
        reach = dict(o=own & (t >= n), dq=own & (t >= n), dk=own & (t < n), dv=own & (t < n))
        for name, rows in reach.items():
            assert torch.equal(got[name][:, :, :-1], want[name][:, :, :-1]), (n, name)
            same(got[name], want[name], ~rows, (n, name))
            assert not got[name][0, rows, -1].isfinite().any(), (n, name)
        same(got["dg"], want["dg"], ~own, n)
        i = next(i for i in range(N) if not cu or cu[i] == lo and cu[i + 1] == hi)
        for name in ("final_state", "dh0"):
            assert not got[name][i, -1].isfinite().any(), (n, name)
            got[name][i, -1] = want[name][i, -1]
            assert torch.equal(got[name], want[name]), (n, name)
