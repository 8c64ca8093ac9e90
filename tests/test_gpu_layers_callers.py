"""The layer operators on the GPU under a caller who goes on using what was passed: cuts refilled before the backward,
a scale changed in place, states that a graph has saved."""
import pytest
import torch

from chunked_gated_delta_09_amd import autograd as ag
from chunked_gated_delta_09_amd import layers
from tests.test_gpu_layers import Draw, F32, scan_inputs

pytestmark = pytest.mark.gpu


def test_cuts_refilled_before_the_backward():
    d = Draw(91)
    x, w, dy = d(1, 50, 32)[0], d(32, 4)[0], d(1, 50, 32)[0]
    v, _ = scan_inputs(93, F32, 1, 50, 32, 16, 2, 2, "softplus dt_bias gate skip state")
    dev = {k: t[0] for k, t in v.items()}

    def grads(refill):
        cu, out = [0, 20, 50], []
        leaves = [t.clone().requires_grad_() for t in (x, w)]
        y, _ = ag.short_conv(*leaves, cu_seqlens=cu)
        if refill:
            cu[1] = 47
        out += torch.autograd.grad((y * dy).sum(), leaves)
        cu = [0, 20, 50]
        leaves = {k: t.clone().requires_grad_() for k, t in dev.items()}
        y, fin = ag.selective_scan(**leaves, cu_seqlens=cu, dt_softplus=True)
        if refill:
            cu[1] = 18  # as many chunks of 16 as before
        return out + list(torch.autograd.grad((y * dy).sum() + fin.sum(), list(leaves.values())))

    for a, b in zip(grads(False), grads(True)):
        assert torch.equal(a, b)


def test_scan_without_gradients_gives_the_same():
    v, _ = scan_inputs(95, F32, 2, 40, 32, 16, 2, 2, "softplus dt_bias gate skip state")
    leaves = {k: t[0].clone().requires_grad_() for k, t in v.items()}
    y, fin = ag.selective_scan(**leaves, dt_softplus=True)
    with torch.no_grad():
        y0, fin0 = ag.selective_scan(**leaves, dt_softplus=True)
    assert y.requires_grad and not y0.requires_grad
    assert torch.equal(y, y0) and torch.equal(fin, fin0)


def test_scale_changed_in_place():
    d = Draw(97)
    q, k, vv = (d(2, 1, 32)[0] for _ in range(3))
    g, beta, st = -torch.rand(2, 1, 32, generator=d.g).cuda(), torch.rand(2, 1, generator=d.g).cuda(), d(2, 1, 32, 32)[0]
    scale = torch.tensor(0.5)
    one = layers.kda_step(q, k, vv, g, beta, st.clone(), scale=scale)
    scale.fill_(2.0)
    two = layers.kda_step(q, k, vv, g, beta, st.clone(), scale=scale)
    assert torch.equal(one * 4, two)  # powers of two: exact


def test_a_saved_state_is_too_new_after_a_step():
    d = Draw(99)
    x, w, st = d(2, 32)[0], d(32, 4)[0], d(2, 3, 32)[0]
    factor = torch.ones_like(st, requires_grad=True)
    loss = (factor * st).sum()
    y = layers.short_conv_step(x, st, w)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        st2 = d(2, 3, 32)[0]
        assert layers.short_conv_step(x, st2, w).shape == y.shape
    graph_state = st.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layers.short_conv_step(x, graph_state, w)
    want_state = graph_state.clone()
    for _ in range(3):
        graph.replay()
        want = layers.short_conv_step(x, want_state, w)
        assert torch.equal(out, want) and torch.equal(graph_state, want_state)


def test_gradient_of_a_final_state_inside_a_larger_one():
    v, d = scan_inputs(101, F32, 2, 40, 32, 16, 2, 2, "softplus dt_bias gate skip state")
    c = d(3 + 2 * 32 * 16)[0]
    got = []
    for joined in (False, True):
        leaves = {k: t[0].clone().requires_grad_() for k, t in v.items()}
        _, fin = ag.selective_scan(**leaves, dt_softplus=True)
        flat = torch.cat([c[:3], fin.reshape(-1)]) * c if joined else fin.reshape(-1) * c[3:].clone()
        got.append(torch.autograd.grad(flat.sum(), list(leaves.values()), allow_unused=True))
    for a, b in zip(*got):
        assert torch.equal(a, b)
