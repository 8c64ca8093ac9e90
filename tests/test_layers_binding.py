"""The binding of the layer operators without a GPU: what it keeps from one call for the next, and what it refuses."""
import pytest
import torch

from chunked_gated_delta_09_amd import layers


class OnGpu(torch.Tensor):
    """A host tensor that passes for one on GPU 0: checks pass it, and the tests below launch nothing."""

    def get_device(self):
        return 0


def on_gpu(*shape):
    return torch.zeros(*shape).as_subclass(OnGpu)


@pytest.fixture
def launched(monkeypatch):
    """The calls that would have been launched: (name, arguments)."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            return name

    monkeypatch.setattr(layers, "_lib", Lib)
    monkeypatch.setattr(layers, "_launch", lambda dev, name, *args: calls.append((name, args)))
    return calls


def step_call(name, state, **kw):
    """One token step of two sequences on `state`."""
    x = on_gpu(2, 8)
    if name == "short_conv_step":
        return layers.short_conv_step(x, state, on_gpu(8, 4), **kw)
    if name == "selective_scan_step":
        return layers.selective_scan_step(x, x, on_gpu(8, 4), on_gpu(2, 1, 4), on_gpu(2, 1, 4), state, **kw)
    return layers.kda_step(on_gpu(2, 2, 16), on_gpu(2, 2, 16), on_gpu(2, 4, 8), on_gpu(2, 4, 16), on_gpu(2, 4), state, **kw)


STATES = {"short_conv_step": (3, 3, 8), "selective_scan_step": (3, 8, 4), "kda_step": (3, 4, 16, 8)}


def test_kda_step_reads_scale_anew(launched):
    """A scale held in a tensor and changed in place: the next call has the new value."""
    state, scale = on_gpu(*STATES["kda_step"]), torch.tensor(0.5)
    step_call("kda_step", state, scale=scale)
    scale.fill_(2.0)
    step_call("kda_step", state, scale=scale)
    step_call("kda_step", state, scale=2)
    step_call("kda_step", state)
    assert [args[0]._obj.scale for _, args in launched] == [0.5, 2.0, 2.0, 0.25]


@pytest.mark.parametrize("name", list(STATES))
def test_steps_tell_autograd_that_the_state_changed(launched, name):
    """A state that a graph has saved: its backward refuses, as behind an in-place operation of torch."""
    state = on_gpu(*STATES[name])
    w = torch.ones(state.shape, requires_grad=True)
    loss = (w * state).sum()
    step_call(name, state)
    assert [n for n, _ in launched] == ["kda_" + name.replace("selective_scan", "sscan").replace("kda_", "")]
    assert state._version == 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        step_call(name, on_gpu(*STATES[name]))  # a tensor without a version
