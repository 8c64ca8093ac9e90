"""Token mixers on the GPU at the ends of their sizes."""
import pytest
import torch

from chunked_gated_delta_09_amd import mixers
from tests import mixer_ref as ref
from tests.test_gpu_mixers import BF16, F32, Draw

pytestmark = pytest.mark.gpu


def test_linear_step_of_a_million_heads():
    """32768 sequences of 32 heads, all but three of them padding."""
    d = Draw(79)
    B, HV, K, V, S = 32768, 32, 128, 128, 4
    g = torch.Generator(device="cuda").manual_seed(79)
    q, k = (torch.randn(B, 1, K, generator=g, device="cuda", dtype=BF16) * K ** -0.5 for _ in range(2))
    v = torch.randn(B, HV, V, generator=g, device="cuda", dtype=BF16)
    gate = -torch.rand(B, HV, generator=g, device="cuda")
    st, st64 = d(S, HV, K, V)
    held = {0: 2, 777: 0, B - 1: 3}
    slots = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    for b, s in held.items():
        slots[b] = s
    before = st.clone()
    o = mixers.linear_attention_step(q, k, v, gate, st, slots=slots, scale=1.0)
    for b, s in held.items():
        q64, k64, v64, g64 = (t[b].cpu().to(ref.F64) for t in (q, k, v, gate))
        new = torch.exp(g64)[:, None, None] * st64[s] + k64[:, :, None] * v64[:, None]
        mag = st64[s].abs() + (k64[:, :, None] * v64[:, None]).abs()
        ref.close(st[s], new, mag, F32, 0, 16, "state")
        ref.close(o[b], (q64[:, :, None] * new).sum(1), (q64.abs()[:, :, None] * mag).sum(1), BF16, 0, 64 + K, "o")
    assert torch.equal(st[1], before[1])
    o[list(held)] = 0
    assert not o.any()
