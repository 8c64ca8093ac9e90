"""The binding of the layer operators without a GPU: what it keeps from one call for the next, and what it refuses."""
import torch

from chunked_gated_delta_09_amd import layers


def test_kda_step_reads_scale_anew(monkeypatch):
    """A scale held in a tensor and changed in place: the next call has the new value, and no tensor is kept."""
    seen = []

    class Lib:
        kda_step = None

    class T(torch.Tensor):
        """A host tensor that passes for one on GPU 0."""

        def get_device(self):
            return 0

    def on_gpu(*shape):
        return torch.zeros(*shape).as_subclass(T)

    monkeypatch.setattr(layers, "_lib", lambda: Lib)
    monkeypatch.setattr(layers, "_launch", lambda dev, fn, d, *a: seen.append(d._obj.scale))
    q, v, g, beta, state = on_gpu(2, 2, 16), on_gpu(2, 4, 8), on_gpu(2, 4, 16), on_gpu(2, 4), on_gpu(3, 4, 16, 8)
    scale = torch.tensor(0.5)
    layers.kda_step(q, q, v, g, beta, state, scale=scale)
    scale.fill_(2.0)
    layers.kda_step(q, q, v, g, beta, state, scale=scale)
    layers.kda_step(q, q, v, g, beta, state, scale=2)
    layers.kda_step(q, q, v, g, beta, state)
    assert seen == [0.5, 2.0, 2.0, 0.25]
