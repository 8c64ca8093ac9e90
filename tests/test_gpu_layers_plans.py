"""The layer operators on the GPU at sizes where a plan changes: groups of channels that do not divide a workgroup,
scans cut into segments of several chunks."""
import pytest
import torch

from chunked_gated_delta_09_amd import layers
from tests import layer_ref as ref
from tests.test_gpu_layers import BF16, F32, SEQS, Draw, grads, ops
from tests.test_layers_plan import CUT, scan_plan

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


OUT = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", skip="dskip", z="dz", dt_bias="ddt_bias", h0="dh0")


@pytest.mark.parametrize("cu", [None, [0, 300, 300, 301, 700]], ids=["dense", "packed"])
def test_selective_scan_growth_of_nothing(cu):
    """A factor of e^6 a token on states that stay zero, because nothing comes in before a sequence's last two tokens,
    and on gradients that stay zero behind its first two. Over a segment of 16 tokens the factor is past fp32; what
    it carries is zero all the same."""
    T, D, NS = 700, 8, 8
    d = Draw(73)
    first, last = torch.zeros(1, T, 1), torch.zeros(1, T, 1)
    cuts = ref.cuts_of(1, T, cu)
    for lo, hi in zip(cuts[:-1], cuts[1:]):
        first[0, lo:min(lo + 2, hi)] = 1.0
        last[0, max(hi - 2, lo):hi] = 1.0
    g = d.g
    host = dict(x=torch.randn(1, T, D, generator=g) * last, dt=torch.full((1, T, D), -6.0), A=torch.full((D, NS), -1.0),
                B=torch.randn(1, T, 1, NS, generator=g), C=torch.randn(1, T, 1, NS, generator=g))
    dy = torch.randn(1, T, D, generator=g) * first
    dev = {k: v.cuda() for k, v in host.items()}
    leaf = {k: v.to(ref.F64).requires_grad_() for k, v in host.items()}
    y64, f64 = ref.scan(*leaf.values(), None, None, None, None, False, cu)
    gr = dict(zip(leaf, grads((y64,), (dy.to(ref.F64),), list(leaf.values()))))
    f = layers.selective_scan(**dev, cu_seqlens=cu, save=True)
    r = layers.selective_scan_bwd(**dev, states=f["states"], dy=dy.cuda(), cu_seqlens=cu)
    ref.close(f["y"], y64, F32, ops(2), "y")
    ref.close(f["final_state"], f64, F32, ops(2), "final_state")
    for k, v in gr.items():
        ref.close(r[OUT[k]], v, F32, ops(2), k)


def check_scan(v, dy, df, dtype, cu, softplus):
    """The scan and its backward against 64 bits; v: each input on the GPU and as a 64-bit leaf."""
    dev = {k: t[0] for k, t in v.items()}
    names = [k for k in v if v[k][1] is not None]
    y64, f64 = ref.scan(*(v[k][1] for k in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "h0")), softplus, cu)
    gr = dict(zip(names, grads((y64, f64), (dy[1], df[1]), [v[k][1] for k in names])))
    f = layers.selective_scan(**dev, cu_seqlens=cu, dt_softplus=softplus, save=True)
    dev.pop("h0")
    r = layers.selective_scan_bwd(**dev, states=f["states"], dy=dy[0], dfinal=df[0], cu_seqlens=cu, dt_softplus=softplus,
                                  output_dh0=True)
    B, T = dy[0].shape[:2]
    cuts = ref.cuts_of(B, T, cu)
    longest = max(hi - lo for lo, hi in zip(cuts[:-1], cuts[1:]))
    ref.close(f["y"], y64, dtype, ops(longest), "y")
    ref.close(f["final_state"], f64, F32, ops(longest), "final_state")
    for k in names:
        whole = k in ("A", "skip", "dt_bias")
        ref.close(r[OUT[k]], gr[k], F32 if whole or k == "h0" else dtype, ops(B * T if whole else longest), k)


@pytest.mark.parametrize("name,dtype", [(n, F32) for n in CUT] + [("quarters", BF16), ("packed_quarters", BF16)])
def test_selective_scan_segments(name, dtype):
    """Segments of several chunks, and local ones of a half and a quarter of them, with a remainder at the end and
    states that live through all of it: about half of a state is left after a segment."""
    lens, packed, D, NS, G, fwd, bwd = CUT[name]
    assert (scan_plan(lens, D, NS, G, False)[:2], scan_plan(lens, D, NS, G, True)[:2]) == (fwd, bwd)
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)] if packed else None
    B, T, N = (1, cu[-1], len(lens)) if packed else (len(lens), lens[0], len(lens))
    d = Draw(79)
    A = -torch.rand(D, NS, generator=d.g) * 3 / bwd[0]
    v = dict(x=d(B, T, D, dtype=dtype), dt=d(B, T, D, dtype=dtype, std=0.5), A=(A.cuda(), A.to(ref.F64).requires_grad_()),
             B=d(B, T, G, NS, dtype=dtype), C=d(B, T, G, NS, dtype=dtype), skip=d(D), z=d(B, T, D, dtype=dtype),
             dt_bias=d(D, std=0.5, mean=-1.0), h0=d(N, D, NS))
    check_scan(v, d(B, T, D, dtype=dtype, leaf=False), d(N, D, NS, leaf=False), dtype, cu, True)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("seqs", list(SEQS))
def test_selective_scan_one_state_and_a_bias(dtype, seqs):
    """One state a channel, four groups, a bias of the steps without softplus; all steps above zero."""
    B, T, cu = SEQS[seqs]
    D, NS, G, N = 132, 1, 4, len(cu) - 1 if cu else B
    d = Draw(83)
    A = -torch.rand(D, NS, generator=d.g) - 0.1
    dt = (torch.rand(B, T, D, generator=d.g) * 0.3 + 0.2).to(dtype)
    bias = torch.rand(D, generator=d.g) * 0.2 - 0.1
    none = (None, None)
    v = dict(x=d(B, T, D, dtype=dtype), dt=(dt.cuda(), dt.to(ref.F64).requires_grad_()),
             A=(A.cuda(), A.to(ref.F64).requires_grad_()), B=d(B, T, G, NS, dtype=dtype), C=d(B, T, G, NS, dtype=dtype),
             skip=none, z=none, dt_bias=(bias.cuda(), bias.to(ref.F64).requires_grad_()), h0=d(N, D, NS))
    check_scan(v, d(B, T, D, dtype=dtype, leaf=False), d(N, D, NS, leaf=False), dtype, cu, False)


def test_selective_scan_growth_of_little():
    """16 tokens, one segment, that multiply a state of 1e-36 by e^96: the factor is past fp32, the product is not."""
    T, D, NS = 200, 8, 8
    d = Draw(89)
    assert scan_plan([T], D, NS, 1, False)[:2] == (16, 16)
    dt = torch.zeros(1, T, D)
    dt[:, 16:32] = -6.0
    host = dict(x=torch.zeros(1, T, D), dt=dt, A=torch.full((D, NS), -1.0), B=torch.randn(1, T, 1, NS, generator=d.g),
                C=torch.randn(1, T, 1, NS, generator=d.g))
    h0 = torch.randn(1, D, NS, generator=d.g) * 1e-36
    f = layers.selective_scan(**{k: v.cuda() for k, v in host.items()}, h0=h0.cuda())
    y64, f64 = ref.scan(*(v.to(ref.F64) for v in host.values()), None, None, None, h0.to(ref.F64), False, None)
    ref.close(f["y"], y64, F32, ops(T), "y")
    ref.close(f["final_state"], f64, F32, ops(T), "final_state")
