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


class Sized:
    """Stands in for a GPU tensor too large for this machine: its description, and no memory."""

    is_cuda, device, requires_grad = True, "cuda:0", False

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    def new_empty(self, shape, dtype=None):
        return Sized(*shape, dtype=dtype or self.dtype)


WRAPPED = 2 ** 32 + 16  # an int32 field that takes it without a look holds 16


@pytest.mark.parametrize("what,call", [
    ("T", lambda: layers.short_conv(Sized(1, WRAPPED, 8), on_gpu(8, 4))),
    ("T", lambda: layers.short_conv_bwd(Sized(1, WRAPPED, 8), on_gpu(8, 4), Sized(1, WRAPPED, 8))),
    ("B", lambda: layers.short_conv(Sized(WRAPPED, 1, 8), on_gpu(8, 4))),
    ("T", lambda: layers.selective_scan(*[Sized(1, WRAPPED, 8)] * 2, on_gpu(8, 4), *[Sized(1, WRAPPED, 1, 4)] * 2)),
    ("C", lambda: layers.group_norm(Sized(1, WRAPPED), 1)),
    ("G", lambda: layers.group_norm(Sized(1, WRAPPED), WRAPPED)),
    ("S", lambda: step_call("short_conv_step", Sized(WRAPPED, 3, 8, dtype=torch.float32))),
    ("S", lambda: step_call("selective_scan_step", Sized(WRAPPED, 8, 4, dtype=torch.float32))),
    ("S", lambda: step_call("kda_step", Sized(WRAPPED, 4, 16, 8, dtype=torch.float32))),
    ("B", lambda: layers.kda_step(*[Sized(WRAPPED, 1, 1)] * 3, Sized(WRAPPED, 1, 1, dtype=torch.float32),
                                  Sized(WRAPPED, 1, dtype=torch.float32), on_gpu(1, 1, 1, 1))),
    (str(WRAPPED), lambda: layers.short_conv(Sized(1, WRAPPED, 8), on_gpu(8, 4), cu_seqlens=[0, 16],
                                             cu_seqlens_dev=torch.zeros(2, dtype=torch.int32).as_subclass(OnGpu))),
    ("cu_seqlens", lambda: layers.short_conv(on_gpu(1, 16, 8), on_gpu(8, 4), cu_seqlens=[0, WRAPPED],
                                             cu_seqlens_dev=torch.zeros(2, dtype=torch.int32).as_subclass(OnGpu)))])
def test_sizes_that_do_not_fit_32_bits_are_refused(launched, monkeypatch, what, call):
    monkeypatch.setattr(torch, "empty_like", lambda t: t.new_empty(t.shape))
    with pytest.raises(ValueError, match=rf"{what}\b.*32 bits"):
        call()
    assert not launched
