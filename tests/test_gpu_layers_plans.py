"""The layer operators on the GPU at sizes where a plan changes: groups of channels that do not divide a workgroup,
scans cut into segments of several chunks."""
import pytest
import torch

from chunked_gated_delta_09_amd import layers
from tests import layer_ref as ref
from tests.test_gpu_layers import BF16, F32, Draw, grads, ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,G,C", [(1, 1023, 8), (3, 1023, 8), (2, 257, 5), (1, 4097, 16), (7, 33, 24), (1200, 255, 2),
                                   (900, 3, 40)])
@pytest.mark.parametrize("opts", ["weight bias", "weight bias shared"])
def test_group_norm_groups_that_do_not_divide(dtype, R, G, C, opts):
    """Odd numbers of groups: the last workgroup has lanes without an item, rows are taken side by side."""
    d = Draw(71)
    n = C if "shared" in opts else G * C
    x, x64 = d(R, G * C, dtype=dtype, mean=0.3)
    w, w64 = d(n, std=0.3, mean=1.0)
    b, b64 = d(n, std=0.3)
    dy, dy64 = d(R, G * C, dtype=dtype, leaf=False)
    kw = dict(weight=w, bias=b, activation="silu", center=True, eps=1e-3)
    y64 = ref.norm(x64, G, w64, b64, None, "silu", True, 1e-3)
    gr = dict(zip(("dx", "dweight", "dbias"), grads((y64,), (dy64,), [x64, w64, b64])))
    ref.close(layers.group_norm(x, G, **kw), y64, dtype, 64, "y")
    r = layers.group_norm_bwd(x, G, dy, **kw)
    for k, v in gr.items():
        ref.close(r[k], v, dtype if k == "dx" else F32, 64 if k == "dx" else ops(R * G), k)
