"""The 64-bit form of linear attention over all pairs against the one that goes token by token (no GPU)."""
import pytest
import torch

from tests import mixer_pairs, mixer_ref as ref


@pytest.mark.parametrize("cu,state,const", [(None, True, False), ([0, 3, 3, 11, 20], True, False), (None, False, True)])
def test_pairs_and_tokens_are_the_same(cu, state, const):
    gen = torch.Generator().manual_seed(3)

    def r(*s):
        return torch.randn(*s, generator=gen, dtype=ref.F64)

    B, T, H, HV, K, V = (1, 20, 2, 70, 3, 5) if cu else (2, 10, 2, 70, 3, 5)
    N = len(cu) - 1 if cu else B
    g = -r(HV).abs() if const else -r(B, T, HV).abs()
    h0, df = (r(N, HV, K, V), r(N, HV, K, V)) if state else (None, None)
    args = (r(B, T, H, K), r(B, T, H, K), r(B, T, HV, V), g, h0, r(B, T, HV, V), df, -0.6, cu)
    want, got = ref.linear_all(*args), mixer_pairs.linear_all(*args)
    got = mixer_pairs.shared(got) if const else got
    assert want.keys() == got.keys()
    for n in want:
        for a, b in zip(want[n], got[n]):
            # sums of a few hundred terms in 64 bits
            assert a.shape == b.shape and (a - b).abs().max() <= 1e-12 * (1 + want[n][1].abs().max()), n
