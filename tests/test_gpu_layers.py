"""Layer operators on the GPU against their 64-bit forms: values and gradients over types, sizes,
packings, strides and states; token steps against whole sequences; a layer's run of them together;
streams, graphs and repeated calls."""
import pytest
import torch

import chunked_gated_delta_09_amd as kda
from chunked_gated_delta_09_amd import autograd as ag
from chunked_gated_delta_09_amd import layers
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


class Draw:
    """Seeded values, rounded to their type, with the 64-bit leaf that holds the same ones."""

    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def __call__(self, *shape, dtype=F32, std=1.0, mean=0.0, leaf=True):
        v = (torch.randn(*shape, generator=self.g) * std + mean).to(dtype)
        return v.cuda(), v.to(ref.F64).requires_grad_(leaf)


def grads(outs, seeds, leaves):
    """Gradients of sum<seed, out> for each leaf, zero where it takes no part."""
    total = sum((o * s.detach()).sum() for o, s in zip(outs, seeds) if s is not None)
    got = torch.autograd.grad(total, leaves, allow_unused=True)
    return [torch.zeros_like(v) if g is None else g for v, g in zip(leaves, got)]


def ops(T):
    return 64 + 4 * T


SEQS = {  # B, T, cuts
    "one_token": (1, 1, None), "dense": (2, 37, None), "tile_edge": (3, 16, None),
    "packed": (1, 70, [0, 1, 1, 4, 21, 53, 69, 70, 70]), "long": (1, 300, None),
}


# ---- short convolution


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("seqs", list(SEQS))
@pytest.mark.parametrize("D,W,opts", [(64, 4, "bias act state"), (5, 3, "act state"), (264, 2, "bias state"), (130, 4, ""),
                                      (1, 2, "bias act"), (36, 3, "bias act state sliced")])
def test_short_conv(dtype, seqs, D, W, opts):
    B, T, cu = SEQS[seqs]
    N = len(cu) - 1 if cu else B
    d = Draw(7)
    wide = "sliced" in opts
    x, x64 = d(B, T, D + (12 if wide else 0), dtype=dtype)
    xs, xs64 = (x[..., 4:4 + D], x64[..., 4:4 + D]) if wide else (x, x64)
    w, w64 = d(D, W, std=0.5)
    b, b64 = d(D) if "bias" in opts else (None, None)
    h, h64 = d(N, W - 1, D, dtype=dtype) if "state" in opts else (None, None)
    dy, dy64 = d(B, T, D, dtype=dtype, leaf=False)
    df, df64 = d(N, W - 1, D, dtype=dtype, leaf=False) if "state" in opts else (None, None)
    act = "silu" if "act" in opts else None
    y64, f64 = ref.conv(xs64, w64, b64, h64, act, cu)
    leaves = [v for v in (x64, w64, b64, h64) if v is not None]
    gr = dict(zip([n for n, v in zip(("dx", "dweight", "dbias", "dh0"), (x64, w64, b64, h64)) if v is not None],
                  grads((y64, f64), (dy64, df64), leaves)))
    f = layers.short_conv(xs, w, bias=b, h0=h, cu_seqlens=cu, activation=act, output_final_state=True)
    r = layers.short_conv_bwd(xs, w, dy, bias=b, h0=h, dfinal=df, cu_seqlens=cu, activation=act)
    ref.close(f["y"], y64, dtype, 64, "y")
    assert torch.equal(f["final_state"].cpu().to(ref.F64), f64.detach())  # copies
    gr["dx"] = gr["dx"][..., 4:4 + D] if wide else gr["dx"]
    for k, v in gr.items():
        ref.close(r[k], v, F32 if k in ("dweight", "dbias") else dtype, ops(B * T) if k in ("dweight", "dbias") else 64, k)
    assert (r["dbias"] is None) == (b is None) and (r["dh0"] is None) == (h is None)


# ---- selective scan


def scan_inputs(seed, dtype, B, T, D, NS, G, N, opts, steps=False):
    d = Draw(seed)
    lead = (B,) if steps else (B, T)
    v = {}
    v["x"], v["dt"] = d(*lead, D, dtype=dtype), d(*lead, D, dtype=dtype, std=0.5)
    if "softplus" not in opts:
        v["dt"] = tuple(t.detach().abs() * 0.2 for t in d(*lead, D, dtype=F32, std=0.5))
        v["dt"] = (v["dt"][0].to(dtype), v["dt"][0].to(dtype).cpu().to(ref.F64).requires_grad_())
    A = -torch.exp(torch.randn(D, NS, generator=d.g) * 0.5)
    v["A"] = (A.cuda(), A.to(ref.F64).requires_grad_())
    v["B"], v["C"] = d(*lead, G, NS, dtype=dtype), d(*lead, G, NS, dtype=dtype)
    v["skip"] = d(D) if "skip" in opts else (None, None)
    v["z"] = d(*lead, D, dtype=dtype) if "gate" in opts else (None, None)
    v["dt_bias"] = d(D, std=0.5, mean=-1.0) if "dt_bias" in opts else (None, None)
    v["h0"] = d(N, D, NS, std=0.5) if "state" in opts else (None, None)
    return v, d


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("seqs", list(SEQS))
@pytest.mark.parametrize("D,NS,G,opts", [
    (64, 16, 1, "softplus dt_bias gate skip state"), (6, 8, 2, "softplus gate"), (70, 13, 1, "skip state"),
    (40, 64, 2, "softplus dt_bias skip"), (33, 32, 1, "softplus gate skip state"), (132, 1, 4, "dt_bias state"),
    (20, 50, 1, "softplus gate dt_bias"), (260, 5, 1, "softplus skip gate state")])
def test_selective_scan(dtype, seqs, D, NS, G, opts):
    B, T, cu = SEQS[seqs]
    N = len(cu) - 1 if cu else B
    v, d = scan_inputs(11, dtype, B, T, D, NS, G, N, opts)
    dy, dy64 = d(B, T, D, dtype=dtype, leaf=False)
    df, df64 = d(N, D, NS, leaf=False) if "state" in opts else (None, None)
    sp = "softplus" in opts
    dev = {k: t[0] for k, t in v.items()}
    y64, f64 = ref.scan(*(v[k][1] for k in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "h0")), sp, cu)
    names = [k for k in v if v[k][1] is not None]
    gr = dict(zip(names, grads((y64, f64), (dy64, df64), [v[k][1] for k in names])))
    largest = max(float(t.detach().abs().max()) for t in [y64, f64, *gr.values()])
    if largest > torch.finfo(F32).max:
        # steps below zero (a bias without softplus) make the states grow by exp(|dt A|) a token
        pytest.skip(f"the 64-bit result {largest:.1e} is outside fp32's range")
    f = layers.selective_scan(**dev, cu_seqlens=cu, dt_softplus=sp, save=True)
    h0 = dev.pop("h0")
    r = layers.selective_scan_bwd(**dev, states=f["states"], dy=dy, dfinal=df, cu_seqlens=cu, dt_softplus=sp,
                                  output_dh0=h0 is not None)
    longest = max(b - a for a, b in zip(ref.cuts_of(B, T, cu)[:-1], ref.cuts_of(B, T, cu)[1:]))
    ref.close(f["y"], y64, dtype, ops(longest), "y")
    ref.close(f["final_state"], f64, F32, ops(longest), "final_state")
    out = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", skip="dskip", z="dz", dt_bias="ddt_bias", h0="dh0")
    for k in names:
        whole = k in ("A", "skip", "dt_bias")
        ref.close(r[out[k]], gr[k], F32 if whole or k == "h0" else dtype, ops(B * T if whole else longest), out[k])
    assert all((r[out[k]] is None) == (v[k][1] is None) for k in ("skip", "z", "dt_bias", "h0"))


@pytest.mark.parametrize("cu", [None, [0, 5, 5, 905, 1000], [0] * 10 + list(range(60)) + [959, 960, 1000]],
                         ids=["dense", "packed", "packed_tables"])
def test_selective_scan_cut_sequences(cu):
    """Few channels and long sequences: the scan is cut along the tokens. Up to 64 packed sequences are
    counted by each wave, more (the last case) by tables."""
    B, T, D, NS = 1, 1000, 64, 16
    N = len(cu) - 1 if cu else 1
    opts = "softplus dt_bias gate skip state"
    v, d = scan_inputs(5, F32, B, T, D, NS, 1, N, opts)
    v["A"] = (v["A"][0] * 0.05, (v["A"][0] * 0.05).cpu().to(ref.F64).requires_grad_())  # states that outlive a segment
    dy, dy64 = d(B, T, D, leaf=False)
    df, df64 = d(N, D, NS, leaf=False)
    dev = {k: t[0] for k, t in v.items()}
    y64, f64 = ref.scan(*(v[k][1] for k in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "h0")), True, cu)
    gr = dict(zip(v, grads((y64, f64), (dy64, df64), [t[1] for t in v.values()])))
    f = layers.selective_scan(**dev, cu_seqlens=cu, dt_softplus=True, save=True)
    dev.pop("h0")
    r = layers.selective_scan_bwd(**dev, states=f["states"], dy=dy, dfinal=df, cu_seqlens=cu, dt_softplus=True, output_dh0=True)
    ref.close(f["y"], y64, F32, ops(T), "y")
    ref.close(f["final_state"], f64, F32, ops(T), "final_state")
    out = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", skip="dskip", z="dz", dt_bias="ddt_bias", h0="dh0")
    for k in v:
        ref.close(r[out[k]], gr[k], F32, ops(T), out[k])


def test_selective_scan_column_slices():
    """x, dt, z, B and C as columns of one projection give what separate tensors give, bit for bit."""
    B, T, D, NS = 2, 40, 48, 8
    d = Draw(3)
    proj, _ = d(B, T, 3 * D + 2 * NS, dtype=BF16)
    A, skip = -torch.rand(D, NS, generator=d.g).cuda(), torch.ones(D, device="cuda")
    x, dt, z = (proj[..., i * D:(i + 1) * D] for i in range(3))
    Bm = proj[..., 3 * D:3 * D + NS].unsqueeze(2)
    Cm = proj[..., 3 * D + NS:].unsqueeze(2)
    dy, _ = d(B, T, D, dtype=BF16)
    a = layers.selective_scan(x, dt, A, Bm, Cm, skip=skip, z=z, dt_softplus=True, save=True)
    c = [t.contiguous() for t in (x, dt, z, Bm, Cm)]
    b = layers.selective_scan(c[0], c[1], A, c[3], c[4], skip=skip, z=c[2], dt_softplus=True, save=True)
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["final_state"], b["final_state"])
    ga = layers.selective_scan_bwd(x, dt, A, Bm, Cm, a["states"], dy, skip=skip, z=z, dt_softplus=True)
    gb = layers.selective_scan_bwd(c[0], c[1], A, c[3], c[4], b["states"], dy, skip=skip, z=c[2], dt_softplus=True)
    for k in ("dx", "ddt", "dA", "dB", "dC", "dskip", "dz"):
        assert torch.equal(ga[k], gb[k]), k


def test_selective_scan_extremes():
    """Decays to zero (dt A = -1000), none (dt = 0), and raw steps far below zero stay finite and right."""
    B, T, D, NS = 1, 20, 8, 8
    v, d = scan_inputs(2, F32, B, T, D, NS, 1, 1, "softplus skip gate state")
    raw = torch.tensor([1000.0, -1000.0, -30.0, 0.0, 80.0, -90.0, 5.0, -5.0]).expand(1, T, D).contiguous()
    v["dt"] = (raw.cuda(), raw.to(ref.F64).requires_grad_())
    dy, dy64 = d(B, T, D, leaf=False)
    dev = {k: t[0] for k, t in v.items()}
    y64, f64 = ref.scan(*(v[k][1] for k in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "h0")), True, None)
    names = [k for k in v if v[k][1] is not None]
    gr = dict(zip(names, grads((y64,), (dy64,), [v[k][1] for k in names])))
    f = layers.selective_scan(**dev, dt_softplus=True, save=True)
    dev.pop("h0")
    r = layers.selective_scan_bwd(**dev, states=f["states"], dy=dy, dt_softplus=True, output_dh0=True)
    ref.close(f["y"], y64, F32, ops(T), "y")
    out = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", skip="dskip", z="dz", h0="dh0")
    for k in names:
        ref.close(r[out[k]], gr[k], F32, ops(T), out[k])


# ---- group norm


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,G,C", [(1, 1, 1), (5, 3, 7), (33, 16, 128), (9, 1, 1000), (300, 5, 64), (4, 2, 2052), (3, 1, 8192),
                                   (2, 1, 5001), (70, 1, 24)])
@pytest.mark.parametrize("opts", ["gate sigmoid weight shared", "silu center weight bias", "gate silu center weight bias shared",
                                  "none", "sigmoid bias"])
def test_group_norm(dtype, R, G, C, opts):
    d = Draw(13)
    act = next((a for a in ("silu", "sigmoid") if a in opts.split()), None)
    n = C if "shared" in opts else G * C
    x, x64 = d(R, G * C, dtype=dtype, mean=0.3)
    w, w64 = d(n, std=0.3, mean=1.0) if "weight" in opts else (None, None)
    b, b64 = d(n, std=0.3) if "bias" in opts else (None, None)
    z, z64 = d(R, G * C, dtype=dtype) if "gate" in opts else (None, None)
    dy, dy64 = d(R, G * C, dtype=dtype, leaf=False)
    kw = dict(weight=w, bias=b, gate=z, activation=act, center="center" in opts, eps=1e-3)
    y64 = ref.norm(x64, G, w64, b64, z64, act, "center" in opts, 1e-3)
    names, leaves = zip(*[(k, v) for k, v in (("dx", x64), ("dweight", w64), ("dbias", b64), ("dgate", z64)) if v is not None])
    gr = dict(zip(names, grads((y64,), (dy64,), leaves)))
    ref.close(layers.group_norm(x, G, **kw), y64, dtype, 64, "y")
    r = layers.group_norm_bwd(x, G, dy, **kw)
    for k, v in gr.items():
        ref.close(r[k], v, F32 if k in ("dweight", "dbias") else dtype, ops(R * G) if k in ("dweight", "dbias") else 64, k)


def test_group_norm_rows_and_slices():
    d = Draw(4)
    wide, _ = d(2, 9, 200, dtype=BF16)
    x, z = wide[..., 8:72], wide[..., 100:164]
    w, _ = d(32, mean=1.0)
    dy, _ = d(2, 9, 64, dtype=BF16)
    kw = dict(weight=w, activation="silu")
    a, b = layers.group_norm(x, 2, gate=z, **kw), layers.group_norm(x.contiguous(), 2, gate=z.contiguous(), **kw)
    assert torch.equal(a, b)
    ga, gb = layers.group_norm_bwd(x, 2, dy, gate=z, **kw), layers.group_norm_bwd(x.contiguous(), 2, dy, gate=z.contiguous(), **kw)
    for k in ("dx", "dweight", "dgate"):
        assert torch.equal(ga[k], gb[k]), k
    empty = layers.group_norm_bwd(x[:0].contiguous(), 2, dy[:0].contiguous(), **kw)
    assert empty["dx"].shape == (0, 9, 64) and not empty["dweight"].any()


# ---- token steps


SLOTS = [3, -1, 0, 7, 3, 5, -9]   # a padding row, one behind the last row, a repeated one


def check_rows(y, state, before, used):
    """Rows of a step with SLOTS: zero for padding, NaN for what is refused; other states as they were."""
    assert not y[1].any() and not y[6].any()
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    rest = [i for i in range(before.shape[0]) if i not in used]
    assert torch.equal(state[rest], before[rest])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,W", [(64, 4), (5, 2), (1030, 3)])
def test_conv_step_slots(dtype, D, W):
    d = Draw(9)
    x, x64 = d(7, D, dtype=dtype)
    st, st64 = d(6, W - 1, D, dtype=dtype)
    w, w64 = d(D, W)
    b, b64 = d(D)
    before = st.clone()
    y = layers.short_conv_step(x, st, w, bias=b, slots=torch.tensor(SLOTS, dtype=torch.int32, device="cuda"))
    check_rows(y, st, before, (3, 0, 5))
    for row, slot in ((0, 3), (2, 0), (5, 5)):
        y64, f64 = ref.conv(x64[row].view(1, 1, D), w64, b64, st64[slot][None], "silu", None)
        ref.close(y[row], y64.reshape(D), dtype, 64)
        assert torch.equal(st[slot].cpu().to(ref.F64), f64[0].detach())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,NS,G", [(64, 16, 1), (6, 8, 2), (70, 13, 1), (40, 64, 4)])
def test_scan_step_slots(dtype, D, NS, G):
    v, d = scan_inputs(21, dtype, 7, 1, D, NS, G, 7, "softplus dt_bias gate skip", steps=True)
    v.pop("h0")
    st, st64 = d(6, D, NS)
    before = st.clone()
    y = layers.selective_scan_step(**{k: t[0] for k, t in v.items()}, state=st, dt_softplus=True,
                                   slots=torch.tensor(SLOTS, dtype=torch.int32, device="cuda"))
    check_rows(y, st, before, (3, 0, 5))
    for row, slot in ((0, 3), (2, 0), (5, 5)):
        one = {k: t[1] if k in ("A", "skip", "dt_bias") else t[1][row][None, None] for k, t in v.items()}
        y64, f64 = ref.scan(*(one[k] for k in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias")), st64[slot][None], True, None)
        ref.close(y[row], y64.reshape(D), dtype, 64)
        ref.close(st[slot], f64[0], F32, 64)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,HV,K,V", [(2, 4, 128, 128), (1, 1, 16, 16), (3, 3, 100, 37), (1, 2, 256, 256), (2, 2, 1, 3)])
@pytest.mark.parametrize("logits", [False, True], ids=["beta", "logits"])
def test_kda_step_slots(dtype, H, HV, K, V, logits):
    d = Draw(31)
    q, q64 = d(7, H, K, dtype=dtype, std=K ** -0.5)
    k, k64 = d(7, H, K, dtype=dtype, std=K ** -0.5)
    vv, v64 = d(7, HV, V, dtype=dtype)
    g = -torch.rand(7, HV, K, generator=d.g) * 2
    raw, raw64 = d(7, HV)
    beta, b64 = (raw, torch.sigmoid(raw64)) if logits else (torch.sigmoid(raw), torch.sigmoid(raw).cpu().to(ref.F64))
    st, st64 = d(6, HV, K, V)
    before = st.clone()
    o = layers.kda_step(q, k, vv, g.cuda(), beta, st, scale=0.3, beta_logits=logits,
                        slots=torch.tensor(SLOTS, dtype=torch.int32, device="cuda"))
    check_rows(o, st, before, (3, 0, 5))
    for row, slot in ((0, 3), (2, 0), (5, 5)):
        o64, s64 = ref.kda_token(q64[row][None], k64[row][None], v64[row][None], g[row][None].to(ref.F64), b64[row][None],
                                 st64[slot][None], 0.3)
        ref.close(o[row], o64[0], dtype, 64 + 4 * K)
        ref.close(st[slot], s64[0], F32, 64 + 4 * K)


def test_steps_without_slots_and_last_rows():
    """No slots: row b of the state; rows behind the batch stay as they were."""
    d = Draw(8)
    x, _ = d(3, 32)
    st, _ = d(5, 2, 32)
    w, _ = d(32, 3)
    other, before = st.clone(), st.clone()
    y = layers.short_conv_step(x, st, w)
    y2 = layers.short_conv_step(x, other, w, slots=torch.arange(3, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, y2) and torch.equal(st, other) and torch.equal(st[3:], before[3:])
    with pytest.raises(kda.KdaError, match="a row for each"):
        layers.short_conv_step(x, st[:2].contiguous(), w)


# ---- together, as a layer runs them


def test_kda_layer_prompt_and_tokens():
    """Convolution of q, k, v -> KDA -> gated head norm: a prompt through the chunk kernels with its last
    tokens then served one by one gives what the whole sequence gives, within bf16 (the chunk
    kernels' own parity bound, 2e-2 relative)."""
    B, T, cut, H, K = 2, 90, 80, 2, 128
    D = H * K
    d = Draw(17)
    proj = [d(B, T, D, dtype=BF16)[0] for _ in range(4)]
    w = [d(D, 4, std=0.5)[0] for _ in range(3)]
    g = torch.nn.functional.logsigmoid(torch.randn(B, T, H, K, generator=d.g) + 3).cuda()
    beta = torch.sigmoid(torch.randn(B, T, H, generator=d.g)).cuda()
    wn, _ = d(K, mean=1.0, std=0.1)

    def unit(t):
        return torch.nn.functional.normalize(t.float().reshape(*t.shape[:-1], H, K), dim=-1).to(BF16)

    def prompt(n):
        c = [layers.short_conv(p[:, :n].contiguous(), wi, output_final_state=True) for p, wi in zip(proj, w)]
        q, k, v = unit(c[0]["y"]), unit(c[1]["y"]), c[2]["y"].reshape(B, n, H, K)
        f = kda.fwd_states(q, k, v, g[:, :n].contiguous(), beta[:, :n].contiguous(), output_o=True)
        y = layers.group_norm(f["o"].reshape(B, n, D), H, weight=wn, gate=proj[3][:, :n].contiguous(), activation="sigmoid")
        return y, f["final_state"], [r["final_state"] for r in c]

    whole, state, _ = prompt(T)
    _, S, conv = prompt(cut)
    for t in range(cut, T):
        c = [layers.short_conv_step(p[:, t], s, wi) for p, s, wi in zip(proj, conv, w)]
        o = layers.kda_step(unit(c[0]), unit(c[1]), c[2].reshape(B, H, K), g[:, t].contiguous(), beta[:, t].contiguous(), S)
        y = layers.group_norm(o.reshape(B, D), H, weight=wn, gate=proj[3][:, t], activation="sigmoid")
        off = (y.float() - whole[:, t].float()).norm() / whole[:, t].float().norm()
        assert off < 2e-2, (t, float(off))
    assert (S - state).norm() / state.norm() < 2e-2


def test_scan_layer_prompt_and_tokens():
    """Convolution -> selective scan -> centred norm, fp32: packed prompts, then tokens from their states."""
    D, NS, W = 40, 16, 4
    d = Draw(19)
    cu, T = [0, 30, 33, 60], 60
    xin, x64 = d(1, T, D)
    extra, e64 = d(3, 2, D)           # two more tokens for each sequence
    w, w64 = d(D, W, std=0.5)
    A = -torch.rand(D, NS, generator=d.g) - 0.1
    dt, dt64 = d(1, T, D, std=0.5)
    dte, dte64 = d(3, 2, D, std=0.5)
    Bm, B64 = d(1, T, 1, NS)
    Be, Be64 = d(3, 2, 1, NS)
    wn, wn64 = d(D)
    c = layers.short_conv(xin, w, cu_seqlens=cu, output_final_state=True)
    s = layers.selective_scan(c["y"], dt, A.cuda(), Bm, Bm, cu_seqlens=cu, dt_softplus=True)
    y = layers.group_norm(s["y"], 1, weight=wn, center=True)
    conv, state = c["final_state"], s["final_state"]
    last = []
    for i in range(2):
        ci = layers.short_conv_step(extra[:, i], conv, w)
        si = layers.selective_scan_step(ci, dte[:, i], A.cuda(), Be[:, i], Be[:, i], state, dt_softplus=True)
        last.append(layers.group_norm(si, 1, weight=wn, center=True))
    for n, (lo, hi) in enumerate(zip(cu[:-1], cu[1:])):
        def run(a, b):
            return torch.cat([a[0, lo:hi], b[n]])[None]
        x = ref.conv(run(x64, e64), w64, None, None, "silu", None)[0]
        b = run(B64, Be64)
        o, _ = ref.scan(x, run(dt64, dte64), A.to(ref.F64), b, b, None, None, None, None, True, None)
        o = ref.norm(o, 1, wn64, None, None, None, True, 1e-5)[0]
        # the norm divides by the spread of 40 channels; 16 roundings more a token for the convolution before
        ref.close(y[0, lo:hi], o[:hi - lo], F32, 64 + 20 * 32, "prompt")
        ref.close(torch.stack([t[n] for t in last]), o[hi - lo:], F32, 64 + 20 * 32, "tokens")


def test_autograd_matches_the_pairs():
    d = Draw(23)
    cu = [0, 20, 50]
    x, _ = d(1, 50, 32, dtype=BF16)
    w, _ = d(32, 4)
    b, _ = d(32)
    h, _ = d(2, 3, 32, dtype=BF16)
    dy, _ = d(1, 50, 32, dtype=BF16)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, h)]
    y, fin = ag.short_conv(*leaves, cu_seqlens=cu, output_final_state=True)
    got = torch.autograd.grad((y * dy).sum() + fin.sum(), leaves)
    r = layers.short_conv_bwd(x, w, dy, bias=b, h0=h, dfinal=torch.ones_like(h), cu_seqlens=cu)
    for g, k in zip(got, ("dx", "dweight", "dbias", "dh0")):
        assert torch.equal(g, r[k]), k
    v, d = scan_inputs(29, F32, 1, 50, 32, 16, 2, 2, "softplus dt_bias gate skip state")
    leaves = {k: t[0].clone().requires_grad_() for k, t in v.items()}
    y, fin = ag.selective_scan(**leaves, cu_seqlens=cu, dt_softplus=True)
    dy, _ = d(1, 50, 32)
    got = torch.autograd.grad((y * dy).sum() + 2 * fin.sum(), list(leaves.values()))
    dev = {k: t[0] for k, t in v.items()}
    f = layers.selective_scan(**dev, cu_seqlens=cu, dt_softplus=True, save=True)
    dev.pop("h0")
    r = layers.selective_scan_bwd(**dev, states=f["states"], dy=dy, dfinal=torch.full_like(fin, 2.0), cu_seqlens=cu,
                                  dt_softplus=True, output_dh0=True)
    for g, k in zip(got, ("dx", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias", "dh0")):
        assert torch.equal(g, r[k]), k
    # only the final state takes part in the loss
    y, fin = ag.selective_scan(**leaves, cu_seqlens=cu, dt_softplus=True)
    (gx,) = torch.autograd.grad(fin.sum(), [leaves["x"]])
    r = layers.selective_scan_bwd(**dev, states=f["states"], dy=torch.zeros_like(dy), dfinal=torch.ones_like(fin),
                                  cu_seqlens=cu, dt_softplus=True)
    assert torch.equal(gx, r["dx"])
    leaves = [t.clone().requires_grad_() for t in (x, torch.ones(16, device="cuda"), dy.to(BF16))]
    y = ag.group_norm(leaves[0], 2, weight=leaves[1], gate=leaves[2], activation="silu")
    got = torch.autograd.grad(y.float().sum(), leaves)
    r = layers.group_norm_bwd(x, 2, torch.ones_like(x), weight=torch.ones(16, device="cuda"), gate=dy.to(BF16), activation="silu")
    for g, k in zip(got, ("dx", "dweight", "dgate")):
        assert torch.equal(g, r[k]), k


def run_all(t, pack):
    """Every operator once, on tensors made beforehand."""
    cu = dict(cu_seqlens=pack[0], cu_seqlens_dev=pack[1])
    out = []
    f = layers.short_conv(t["x"], t["w"], h0=t["hc"], output_final_state=True, **cu)
    b = layers.short_conv_bwd(t["x"], t["w"], t["dy"], h0=t["hc"], **cu)
    out += [f["y"], f["final_state"], b["dx"], b["dweight"], b["dh0"]]
    f = layers.selective_scan(t["x"], t["dt"], t["A"], t["B"], t["C"], z=t["z"], h0=t["h0"], dt_softplus=True, save=True, **cu)
    b = layers.selective_scan_bwd(t["x"], t["dt"], t["A"], t["B"], t["C"], f["states"], t["dy"], z=t["z"], dt_softplus=True,
                                  output_dh0=True, **cu)
    out += [f["y"], f["final_state"]] + [b[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dz", "dh0")]
    kw = dict(weight=t["wn"], gate=t["z"], activation="silu", center=True)
    b = layers.group_norm_bwd(t["x"], 4, t["dy"], **kw)
    out += [layers.group_norm(t["x"], 4, **kw), b["dx"], b["dweight"], b["dgate"]]
    st, ss = t["st"].clone(), t["ss"].clone()
    out += [layers.short_conv_step(t["x"][0, :8], st, t["w"]), st]
    out += [layers.selective_scan_step(t["x"][0, :8], t["dt"][0, :8], t["A"], t["B"][0, :8], t["C"][0, :8], ss), ss]
    sk = t["sk"].clone()
    out += [layers.kda_step(t["q"], t["q"], t["q"], t["gk"], t["beta"], sk), sk]
    return out


def all_inputs(seed):
    d = Draw(seed)
    T, D = 700, 64
    shapes = dict(x=(1, T, D), dt=(1, T, D), z=(1, T, D), dy=(1, T, D), B=(1, T, 1, 16), C=(1, T, 1, 16), hc=(3, 3, D),
                  st=(8, 3, D), q=(8, 2, 32))
    t = {k: d(*s, dtype=BF16)[0] for k, s in shapes.items()}
    t.update(w=d(D, 4)[0], wn=d(16)[0], h0=d(3, D, 16)[0], ss=d(8, D, 16)[0], sk=d(8, 2, 32, 32, std=0.1)[0], beta=d(8, 2, std=0.1)[0])
    t["A"] = -torch.rand(D, 16, generator=d.g).cuda()
    t["gk"] = -torch.rand(8, 2, 32, generator=d.g).cuda()
    cu = [0, 500, 500, 700]
    return t, (cu, torch.tensor(cu, dtype=torch.int32, device="cuda"))


def test_runs_twice_the_same_and_on_another_stream():
    t, pack = all_inputs(41)
    first = run_all(t, pack)
    again = run_all(t, pack)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run_all(t, pack)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for i, (a, b, c) in enumerate(zip(first, again, other)):
        assert torch.equal(a, b) and torch.equal(a, c), i


def test_graph_replays():
    """A captured run of every operator, replayed on new inputs with eager work between the replays."""
    t, pack = all_inputs(43)
    run_all(t, pack)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run_all(t, pack)
    for seed in (44, 45, 46):
        new, _ = all_inputs(seed)
        for k in t:
            t[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for i, (a, b) in enumerate(zip(got, run_all(new, pack))):
            assert torch.equal(a, b), (seed, i)


def test_two_streams_at_once():
    """Calls that overlap on two streams have workspaces of their own."""
    sets = [all_inputs(s) for s in (51, 52)]
    want = [run_all(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = run_all(*sets[i])
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)


# ---- edges


def test_no_tokens():
    """T = 0: states pass through, gradients of parameters are zero."""
    d = Draw(61)
    D, NS = 24, 16
    x = torch.empty(2, 0, D, device="cuda")
    w, h = d(D, 4)[0], d(2, 3, D)[0]
    f = layers.short_conv(x, w, h0=h, output_final_state=True)
    b = layers.short_conv_bwd(x, w, x, h0=h, dfinal=h)
    assert f["y"].shape == (2, 0, D) and torch.equal(f["final_state"], h)
    assert torch.equal(b["dh0"], h) and not b["dweight"].any()
    A, h0, bc = -torch.ones(D, NS, device="cuda"), d(2, D, NS)[0], torch.empty(2, 0, 1, NS, device="cuda")
    f = layers.selective_scan(x, x, A, bc, bc, skip=w[:, 0].contiguous(), h0=h0, save=True)
    b = layers.selective_scan_bwd(x, x, A, bc, bc, f["states"], x, skip=w[:, 0].contiguous(), dfinal=h0, output_dh0=True)
    assert torch.equal(f["final_state"], h0) and torch.equal(b["dh0"], h0)
    assert not b["dA"].any() and not b["dskip"].any()


def test_many_short_sequences():
    """More sequences than a table's workgroup has lanes, most of them empty or a token long."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 4, (1500,), generator=g)
    cu = [0] + torch.cumsum(lens, 0).tolist()
    T, D, NS, N = cu[-1], 12, 8, 1500
    v, d = scan_inputs(63, F32, 1, T, D, NS, 1, N, "softplus skip gate state")
    dy, dy64 = d(1, T, D, leaf=False)
    df, df64 = d(N, D, NS, leaf=False)
    dev = {k: t[0] for k, t in v.items()}
    y64, f64 = ref.scan(*(v[k][1] for k in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "h0")), True, cu)
    names = [k for k in v if v[k][1] is not None]
    gr = dict(zip(names, grads((y64, f64), (dy64, df64), [v[k][1] for k in names])))
    f = layers.selective_scan(**dev, cu_seqlens=cu, dt_softplus=True, save=True)
    dev.pop("h0")
    r = layers.selective_scan_bwd(**dev, states=f["states"], dy=dy, dfinal=df, cu_seqlens=cu, dt_softplus=True, output_dh0=True)
    ref.close(f["y"], y64, F32, ops(4), "y")
    ref.close(f["final_state"], f64, F32, ops(4), "final_state")
    out = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", skip="dskip", z="dz", h0="dh0")
    for k in names:
        ref.close(r[out[k]], gr[k], F32, ops(T if k in ("A", "skip") else 4), out[k])
    w, w64 = d(D, 4)
    h, h64 = d(N, 3, D)
    y64, f64 = ref.conv(v["x"][1], w64, None, h64, "silu", cu)
    gw, gh = grads((y64,), (dy64,), [w64, h64])
    f = layers.short_conv(v["x"][0], w, h0=h, cu_seqlens=cu, output_final_state=True)
    b = layers.short_conv_bwd(v["x"][0], w, dy, h0=h, cu_seqlens=cu)
    ref.close(f["y"], y64, F32, 64, "y")
    ref.close(b["dweight"], gw, F32, ops(T), "dweight")
    ref.close(b["dh0"], gh, F32, 64, "dh0")


def test_masked_neighbours_do_not_leak():
    """NaN and infinity in one sequence's inputs and states stay in that sequence."""
    cu, T, D, NS = [0, 9, 30, 41], 41, 16, 8
    v, d = scan_inputs(67, F32, 1, T, D, NS, 1, 3, "softplus gate state")
    dev = {k: t[0] for k, t in v.items()}
    w, h = d(D, 4)[0], d(3, 3, D)[0]
    dy = d(1, T, D)[0]

    def run():
        f = layers.short_conv(dev["x"], w, h0=h, cu_seqlens=cu, output_final_state=True)
        b = layers.short_conv_bwd(dev["x"], w, dy, h0=h, cu_seqlens=cu)
        s = layers.selective_scan(**dev, cu_seqlens=cu, dt_softplus=True, save=True)
        kw = {k: t for k, t in dev.items() if k != "h0"}
        g = layers.selective_scan_bwd(**kw, states=s["states"], dy=dy, cu_seqlens=cu, dt_softplus=True, output_dh0=True)
        rows = [f["y"][0], b["dx"][0], s["y"][0]] + [g[k][0] for k in ("dx", "ddt", "dz", "dB", "dC")]
        return rows, [f["final_state"], b["dh0"], s["final_state"], g["dh0"]]

    clean = run()
    for k in ("x", "dt", "z", "B", "C"):
        dev[k][0, 9:30] = float("nan") if k != "z" else float("inf")
    dy[0, 9:30] = float("nan")
    h[1], dev["h0"][1] = float("inf"), float("nan")
    dirty = run()
    keep = torch.cat([torch.arange(9), torch.arange(30, 41)]).cuda()
    for a, b in zip(clean[0], dirty[0]):
        assert torch.equal(a[keep], b[keep])
    for a, b in zip(clean[1], dirty[1]):
        assert torch.equal(a[[0, 2]], b[[0, 2]])


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last rows against a run of their own."""
    D, T = 4096, 2 ** 19 + 40
    x = torch.empty(1, T, D, dtype=BF16, device="cuda").uniform_(-1, 1, generator=torch.Generator("cuda").manual_seed(5))
    assert x.numel() > 2 ** 31
    w = torch.rand(D, 4, device="cuda") - 0.5
    tail = x[:, -200:].contiguous()
    y, small = layers.short_conv(x, w)["y"], layers.short_conv(tail, w)["y"]
    assert torch.equal(y[:, -100:], small[:, -100:])
    del y
    dx, small = layers.short_conv_bwd(x, w, x)["dx"], layers.short_conv_bwd(tail, w, tail)["dx"]
    assert torch.equal(dx[:, -100:], small[:, -100:])
    del dx
    gate = x.view(-1, 32, 128)
    y = layers.group_norm(x, 32, gate=x, activation="silu")
    assert torch.equal(y[:, -100:], layers.group_norm(tail, 32, gate=tail, activation="silu")[:, -100:])
    del y, gate
    # decays of e^-2 a token and more: 100 tokens on, nothing is left of an earlier state
    A = -torch.arange(2, 10, device="cuda", dtype=F32).expand(D, 8).contiguous()
    bc = torch.ones(1, T, 1, 8, dtype=BF16, device="cuda")
    step = torch.ones_like(x)
    y = layers.selective_scan(x, step, A, bc, bc)["y"]
    small = layers.selective_scan(tail, step[:, -200:].contiguous(), A, bc[:, -200:].contiguous(), bc[:, -200:].contiguous())["y"]
    # both within half a step of bf16 of sums of at most 8 terms that fp32 holds to 2^-20
    ref.close(y[:, -100:], small[:, -100:].cpu(), BF16, 64)
    del x, y, step
    state = torch.zeros(33000, 1, 256, 256, device="cuda")
    assert state.numel() > 2 ** 31
    state[-1] = 1.0
    q = torch.ones(1, 1, 256, device="cuda")
    o = layers.kda_step(q, q * 0, q, q * 0, torch.ones(1, 1, device="cuda"), state, scale=1.0,
                        slots=torch.tensor([32999], dtype=torch.int32, device="cuda"))
    assert torch.equal(o, torch.full_like(o, 256.0)) and not state[0].any()
