"""The autograd wrappers without a GPU: what they keep between the forward and the backward, seen at the calls that they
make of the binding (stand-ins on the CPU here)."""
import numpy as np
import pytest
import torch

from chunked_gated_delta_09_amd import autograd as ag

CUTS = [0, 2, 5]


def record(monkeypatch, module, names, results):
    """Puts stand-ins for a forward and a backward in place; returns the list of the keyword arguments they were called
    with, cuts copied as they stood."""
    calls = []

    def stand_in(result):
        def call(*args, **kw):
            cu = kw.get("cu_seqlens")
            calls.append(dict(kw, cu_seqlens=None if cu is None else [int(c) for c in cu]))
            return {k: v() for k, v in result.items()}
        return call

    for name, result in zip(names, results):
        monkeypatch.setattr(module, name, stand_in(result))
    return calls


def refill(cu, values):
    for i, v in enumerate(values):
        cu[i] = v


def zeros(*shape):
    return lambda: torch.zeros(*shape)


@pytest.mark.parametrize("kind", [list, np.array, torch.tensor], ids=["list", "numpy", "tensor"])
def test_short_conv_keeps_its_cuts(monkeypatch, kind):
    calls = record(monkeypatch, ag.layers, ("short_conv", "short_conv_bwd"),
                   (dict(y=zeros(1, 5, 3), final_state=lambda: None),
                    dict(dx=zeros(1, 5, 3), dweight=zeros(3, 4), dbias=lambda: None, dh0=lambda: None)))
    x, w, cu = torch.zeros(1, 5, 3, requires_grad=True), torch.zeros(3, 4), kind(CUTS)
    y, _ = ag.short_conv(x, w, cu_seqlens=cu)
    refill(cu, [0, 4, 5])  # the caller's buffer holds the next batch's cuts by the time of the backward
    y.sum().backward()
    assert [c["cu_seqlens"] for c in calls] == [CUTS, CUTS]


@pytest.mark.parametrize("kind", [list, np.array, torch.tensor], ids=["list", "numpy", "tensor"])
def test_selective_scan_keeps_its_cuts(monkeypatch, kind):
    none = dict(dskip=lambda: None, dz=lambda: None, ddt_bias=lambda: None, dh0=lambda: None)
    calls = record(monkeypatch, ag.layers, ("selective_scan", "selective_scan_bwd"),
                   (dict(y=zeros(1, 5, 3), final_state=lambda: None, states=zeros(3, 3, 2)),
                    dict(dx=zeros(1, 5, 3), ddt=zeros(1, 5, 3), dA=zeros(3, 2), dB=zeros(1, 5, 1, 2), dC=zeros(1, 5, 1, 2), **none)))
    x, A, B, cu = torch.zeros(1, 5, 3, requires_grad=True), torch.zeros(3, 2), torch.zeros(1, 5, 1, 2), kind(CUTS)
    y, _ = ag.selective_scan(x, x.detach(), A, B, B, cu_seqlens=cu, output_final_state=False)
    refill(cu, [0, 4, 5])
    y.sum().backward()
    assert [c["cu_seqlens"] for c in calls] == [CUTS, CUTS]


def test_group_norm_keeps_its_eps(monkeypatch):
    seen = []
    monkeypatch.setattr(ag.layers, "group_norm", lambda x, groups, eps, **kw: seen.append(float(eps)) or torch.zeros_like(x))
    monkeypatch.setattr(ag.layers, "group_norm_bwd", lambda x, groups, dy, eps, **kw: seen.append(float(eps)) or dict(
        dx=torch.zeros_like(x), dweight=None, dbias=None, dgate=None))
    eps = torch.tensor(0.5)
    y = ag.group_norm(torch.zeros(2, 4, requires_grad=True), 2, eps=eps)
    eps.fill_(2.0)
    y.sum().backward()
    assert seen == [0.5, 0.5]


@pytest.mark.parametrize("kind", [list, np.array, torch.tensor], ids=["list", "numpy", "tensor"])
def test_kda_chunk_keeps_its_cuts_and_scale(monkeypatch, kind):
    one = zeros(1, 5, 1, 2)
    calls = record(monkeypatch, ag, ("fwd_states", "chunk_bwd"),
                   (dict(o=one, final_state=lambda: None, states=one, inv=one, saved=one),
                    dict(dq=one, dk=one, dv=one, dg=one, dbeta=zeros(1, 5, 1))))
    q, beta, cu, scale = one().requires_grad_(), torch.zeros(1, 5, 1), kind(CUTS), torch.tensor(0.5)
    o, _ = ag.kda_chunk(q, one(), one(), one(), beta, cu_seqlens=cu, scale=scale, output_final_state=False)
    refill(cu, [0, 4, 5])
    scale.fill_(2.0)
    o.sum().backward()
    assert [c["cu_seqlens"] for c in calls] == [CUTS, CUTS]
    assert [float(c["scale"]) for c in calls] == [0.5, 0.5]


NONE = dict(dskip=lambda: None, dz=lambda: None, ddt_bias=lambda: None, dh0=lambda: None)
SCAN = (dict(y=zeros(1, 5, 3), final_state=lambda: None, states=zeros(3, 3, 2)),
        dict(dx=zeros(1, 5, 3), ddt=zeros(1, 5, 3), dA=zeros(3, 2), dB=zeros(1, 5, 1, 2), dC=zeros(1, 5, 1, 2), **NONE))


def test_selective_scan_saves_states_for_a_backward_only(monkeypatch):
    """Without gradients there is no backward to keep the chunks' states for."""
    calls = record(monkeypatch, ag.layers, ("selective_scan", "selective_scan_bwd"), SCAN)
    x, A, B = torch.zeros(1, 5, 3), torch.zeros(3, 2), torch.zeros(1, 5, 1, 2)
    leaf = A.clone().requires_grad_()
    ag.selective_scan(x, x, A, B, B)
    with torch.no_grad():
        ag.selective_scan(x, x, leaf, B, B)
    with torch.inference_mode():
        ag.selective_scan(x, x, leaf, B, B)
    ag.selective_scan(x, x, leaf, B, B)[0].sum().backward()
    ag.selective_scan(x, x, A, B, B, h0=torch.zeros(1, 3, 2, requires_grad=True))
    assert [c["save"] for c in calls if "save" in c] == [False, False, False, True, True]


@pytest.mark.parametrize("given", [False, True], ids=["made", "given"])
@pytest.mark.parametrize("op", ["short_conv", "selective_scan"])
def test_one_device_copy_of_the_cuts(monkeypatch, op, given):
    """The backward takes the copy that the forward took, the caller's or the one made for it."""
    conv = (dict(y=zeros(1, 5, 3), final_state=lambda: None),
            dict(dx=zeros(1, 5, 3), dweight=zeros(3, 4), dbias=lambda: None, dh0=lambda: None))
    calls = record(monkeypatch, ag.layers, (op, op + "_bwd"), conv if op == "short_conv" else SCAN)
    x, A, B = torch.zeros(1, 5, 3, requires_grad=True), torch.zeros(3, 2), torch.zeros(1, 5, 1, 2)
    cu_dev = torch.tensor(CUTS, dtype=torch.int32) if given else None
    args = (x, torch.zeros(3, 4)) if op == "short_conv" else (x, x.detach(), A, B, B)
    getattr(ag, op)(*args, cu_seqlens=CUTS, cu_seqlens_dev=cu_dev)[0].sum().backward()
    fwd, bwd = (c["cu_seqlens_dev"] for c in calls)
    assert fwd.dtype == torch.int32 and fwd.tolist() == CUTS
    assert fwd.data_ptr() == bwd.data_ptr() == (cu_dev if given else fwd).data_ptr()


def test_selective_scan_backward_aligns_the_final_states_gradient(monkeypatch):
    """torch hands a backward views: behind a concatenation the gradient of the final state begins where the parts before
    it end, while the library reads its rows 16 bytes at a time."""
    seen = []
    x, A, B = torch.zeros(1, 5, 3, requires_grad=True), torch.zeros(3, 8), torch.zeros(1, 5, 1, 8)
    monkeypatch.setattr(ag.layers, "selective_scan", lambda *a, **kw: dict(
        y=torch.zeros(1, 5, 3), final_state=torch.zeros(1, 3, 8), states=torch.zeros(1, 3, 8)))
    monkeypatch.setattr(ag.layers, "selective_scan_bwd", lambda *a, dfinal, **kw: seen.append(dfinal) or {
        k: v() for k, v in SCAN[1].items()} | dict(dA=None, dB=None, dC=None))
    _, fin = ag.selective_scan(x, x.detach(), A, B, B)
    torch.cat([torch.zeros(3), fin.reshape(-1)]).mul(torch.arange(27.0)).sum().backward()
    (dfinal,) = seen
    assert dfinal.is_contiguous() and dfinal.data_ptr() % 16 == 0
    assert torch.equal(dfinal.reshape(-1), torch.arange(3.0, 27.0))


def test_selective_scan_refuses_forward_mode(monkeypatch):
    """It has no forward-mode derivative: dual numbers raise rather than lose their tangents."""
    record(monkeypatch, ag.layers, ("selective_scan", "selective_scan_bwd"), SCAN)
    x, A, B = torch.zeros(1, 5, 3), torch.zeros(3, 2), torch.zeros(1, 5, 1, 2)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises((NotImplementedError, RuntimeError), match="jvp"):
            ag.selective_scan(dual, x, A, B, B)
