"""The layer operators on the GPU under a caller who goes on using what was passed: cuts refilled before the backward,
a scale changed in place, states that a graph has saved."""
import pytest
import torch

import chunked_gated_delta_09_amd as kda
from chunked_gated_delta_09_amd import autograd as ag
from chunked_gated_delta_09_amd import layers
from tests import layer_ref as ref
from tests.test_gpu_layers import BF16, F32, Draw, ops, scan_inputs

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


def shifted(t, by):
    """The values of t, contiguous, beginning `by` elements behind an aligned address."""
    if t is None or not t.numel():
        return t
    out = t.new_empty(t.numel() + by)[by:].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 16 == by * t.element_size() % 16
    return out


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("by", [1, 2, 3])
def test_tensors_that_begin_anywhere(dtype, by):
    """Widths that allow wide loads, addresses that do not: the values of aligned tensors' calls."""
    d = Draw(103)
    B, T, D, NS, W = 2, 37, 64, 16, 4
    x, dt, z, dy = (d(B, T, D, dtype=dtype)[0] for _ in range(4))
    Bm, Cm = (d(B, T, 1, NS, dtype=dtype)[0] for _ in range(2))
    w, bias, wn = d(D, W)[0], d(D)[0], d(16)[0]
    hc, h0, A = d(B, W - 1, D, dtype=dtype)[0], d(B, D, NS)[0], -torch.rand(D, NS, generator=d.g).cuda()
    q, v = d(B, 2, 32, dtype=dtype)[0], d(B, 2, 32, dtype=dtype)[0]
    g, beta, S = -torch.rand(B, 2, 32, generator=d.g).cuda(), torch.rand(B, 2, generator=d.g).cuda(), d(B, 2, 32, 32)[0]

    def run(m):
        out = []
        f = layers.short_conv(m(x), m(w), bias=m(bias), h0=m(hc), output_final_state=True)
        r = layers.short_conv_bwd(m(x), m(w), m(dy), bias=m(bias), h0=m(hc), dfinal=m(hc))
        out += [f["y"], f["final_state"], r["dx"], r["dweight"], r["dbias"], r["dh0"]]
        f = layers.selective_scan(m(x), m(dt), A, m(Bm), m(Cm), skip=m(bias), z=m(z), dt_bias=m(bias), h0=h0, dt_softplus=True,
                                  save=True)
        r = layers.selective_scan_bwd(m(x), m(dt), A, m(Bm), m(Cm), f["states"], m(dy), skip=m(bias), z=m(z), dt_bias=m(bias),
                                      dt_softplus=True)
        out += [f["y"], f["final_state"]] + [r[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias")]
        kw = dict(weight=m(wn), bias=m(wn), gate=m(z), activation="silu", center=True)
        r = layers.group_norm_bwd(m(x), 4, m(dy), **kw)
        out += [layers.group_norm(m(x), 4, **kw), r["dx"], r["dweight"], r["dbias"], r["dgate"]]
        state = m(hc).clone() if m is not shifted_by else shifted_by(hc)
        out += [layers.short_conv_step(m(x[:, 0].contiguous()), state, m(w), bias=m(bias)), state]
        st = h0.clone()
        out += [layers.selective_scan_step(m(x[:, 0].contiguous()), m(dt[:, 0].contiguous()), A, m(Bm[:, 0].contiguous()),
                                           m(Cm[:, 0].contiguous()), st, z=m(z[:, 0].contiguous()), dt_softplus=True), st]
        Sk = S.clone() if m is not shifted_by else shifted_by(S)
        out += [layers.kda_step(m(q), m(q), m(v), m(g), m(beta), Sk), Sk]
        return out

    def shifted_by(t):
        return shifted(t, by)

    for i, (a, b) in enumerate(zip(run(lambda t: t), run(shifted_by))):
        assert a.shape == b.shape
        ref.close(b, a.cpu(), a.dtype, ops(T), i)


def test_scan_states_that_begin_anywhere_are_refused():
    """Rows of 16 states are read whole: the call says so rather than reading across."""
    d = Draw(105)
    x, A, b = d(1, 8, 8)[0], -torch.ones(8, 16, device="cuda"), d(1, 8, 1, 16)[0]
    with pytest.raises(kda.KdaError, match="h0 must be 16-byte aligned"):
        layers.selective_scan(x, x, A, b, b, h0=shifted(d(1, 8, 16)[0], 1))
    with pytest.raises(kda.KdaError, match="A must be 16-byte aligned"):
        layers.selective_scan(x, x, shifted(A, 1), b, b)
    with pytest.raises(kda.KdaError, match="state must be 16-byte aligned"):
        layers.selective_scan_step(x[0], x[0], A, b[0], b[0], shifted(d(8, 8, 16)[0], 1))
    odd = [shifted(t, 1) for t in (-torch.rand(8, 13, generator=d.g).cuda(), d(1, 8, 13)[0])]  # 13 states: single loads
    c = d(1, 8, 1, 13)[0]
    f = layers.selective_scan(x, x, odd[0], c, c, h0=odd[1])
    want = layers.selective_scan(x, x, odd[0].clone(), c, c, h0=odd[1].clone())
    assert torch.equal(f["y"], want["y"]) and torch.equal(f["final_state"], want["final_state"])
