"""Token mixers on the GPU in the forms that large calls run, against 64 bits: linear attention whose segments have many chunks, window
attention whose tiles go straight to shared memory."""
import math

import pytest
import torch

from tests import mixer_pairs
from tests import mixer_ref as ref
from tests.test_gpu_mixers import BF16, DT, F32, lin_check, lin_inputs, win_check, win_inputs
from tests.test_gpu_mixers_use import BAD, linear_all, poisoned, same

pytestmark = pytest.mark.gpu

# T, H, HV, K, V, cuts, segments of bf16 and of fp32 (whose tiles have 64 columns: more workgroups, fewer cuts). A segment has 9 to 19 chunks of
# 32 tokens where its sequence does.
MANY = {
    "whole": (330, 256, 512, 16, 16, None, 1, 1),
    "two": (600, 64, 256, 16, 48, None, 2, 2),
    "wide": (600, 64, 256, 128, 128, None, 2, 1),
    "widest": (600, 32, 128, 256, 256, None, 2, 1),
    "odd": (610, 256, 256, 33, 20, None, 2, 2),
    "odd_wide": (600, 128, 256, 100, 90, None, 2, 1),
    "packed": (1010, 128, 256, 32, 64, [0, 1, 1, 400, 1010, 1010], 7, 7),
}


def gates(kind, shape, seed):
    """Weak: a state of hundreds of tokens. Strong: resets of -200, of the type's lowest value and of -infinity among weak ones."""
    gen = torch.Generator().manual_seed(seed)
    g = torch.nn.functional.logsigmoid(torch.randn(shape, generator=gen) + (3.0 if kind == "mild" else 6.0))
    if kind == "strong":
        r = torch.rand(shape, generator=gen)
        low = torch.tensor([-200.0, -math.inf, torch.finfo(F32).min])
        g = torch.where(r < 0.03, low[(r * 100).long().clamp(max=2)], g)
    return g


@DT
@pytest.mark.parametrize("kind", ["weak", "mild", "strong"])
@pytest.mark.parametrize("form", list(MANY))
def test_linear_attention_of_many_chunks(dtype, form, kind):
    T, H, HV, K, V, cu, *segments = MANY[form]
    N = len(cu) - 1 if cu else 1
    const = form == "two" and kind == "weak"
    dev, x64 = lin_inputs(81, dtype, 1, T, H, HV, K, V, N, form != "wide", False)
    g = gates(kind, (HV,) if const else (1, T, HV), 83)
    dev["g"], x64["g"] = g.cuda(), g.to(ref.F64).clamp(min=-1e4)  # exp of anything lower is zero as well
    want = mixer_pairs.linear_all(**x64, scale=0.7, cu=cu)
    f, _ = lin_check(dev, mixer_pairs.shared(want) if const else want, dtype, cu, 0.7, T)
    assert f["states"].shape[0] == N + segments[dtype == F32]


@DT
@pytest.mark.parametrize("T,HV,K,V", [(333, 512, 16, 16), (600, 256, 64, 32), (600, 256, 33, 20)])
def test_many_chunks_that_are_not_finite(dtype, T, HV, K, V):
    """What is not finite reaches later outputs and gradients of q, earlier gradients of k and v, and only its own head's."""
    dev, _ = lin_inputs(85, dtype, 1, T, HV, HV, K, V, 1, True, False)
    want = linear_all(dev)
    for n in (3, 31, 32, 200, T - 1):
        before, after = slice(0, n), slice(n + 1, T)
        for value in BAD:
            for name in ("q", "k", "v", "do"):
                got = linear_all(poisoned(dev, name, n, value, 5))
                for out in ("o", "dq", "dk", "dv"):
                    assert torch.equal(got[out][:, :, :-1], want[out][:, :, :-1]), (name, out)
                assert torch.equal(got["final_state"][:, :-1], want["final_state"][:, :-1])
                assert torch.equal(got["dh0"][:, :-1], want["dh0"][:, :-1])
                same(got["o"], want["o"], before, name)
                same(got["dq"], want["dq"], before, name)
                same(got["dv"], want["dv"], after, name)
                same(got["dk"], want["dk"], after, name)
                if name in ("k", "v"):
                    bad = got["o"][0, n:, -1] if name == "k" else got["o"][0, n:, -1, 5]
                    assert not bad.isfinite().any()
                elif name == "q":
                    same(got["o"], want["o"], after, name)
                    assert not got["o"][0, n, -1].isfinite().any()


@DT
@pytest.mark.parametrize("H,HK,D,window,sinks,cu", [
    (8, 8, 64, 70, 3, None), (8, 8, 64, 40, 66, [0, 1, 500, 500, 1060]),      # 64 queries and keys a workgroup
    (64, 16, 64, 70, 3, [0, 1, 500, 500, 1060]), (64, 16, 64, 129, 66, None),  # 128 of both
    (64, 16, 128, 70, 3, [0, 1, 500, 500, 1060]), (64, 16, 128, 200, 66, None)])  # 128 queries, 64 keys
def test_window_attention_in_direct_tiles(dtype, H, HK, D, window, sinks, cu):
    dev, x64 = win_inputs(87, dtype, 1, 1060, H, HK, D)
    win_check(dev, x64, dtype, window, sinks, D ** -0.5, cu, 1060, D)
