"""Cases of the layer operators: short causal convolution, selective state space scan, group norm
with an activation, and the single-token step of Kimi Delta Attention.

`run` computes a case with elementary torch operations in 32 bits (rounded once at the end), or,
where `own` is true, with the library's kernels. `exact` computes the same outputs in 64 bits from
the operators' definitions.
"""
import math

import numpy as np
import torch

own = False

LN_EPS = 1e-5


# ---------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # q, k and v of a training batch before the chunk kernels: B=4, T=4096, 32 heads of 128 channels
        dict(name="conv_train_bf16", op="conv_train", dtype="bf16", B=4, T=4096, D=4096, W=4, act=True, bias=True,
             packed=0, state=False),
        # a small fp32 run of packed sequences with carried states, as tests and fine-tuning on short texts have
        dict(name="conv_train_packed_f32", op="conv_train", dtype="f32", B=1, T=1777, D=1000, W=3, act=True, bias=False,
             packed=9, state=True),
        # one token of each of 64 served sequences
        dict(name="conv_step", op="conv_step", dtype="bf16", B=64, D=4096, W=4, act=True, bias=True, slots=256),
        # a training batch: B=2, T=2048, 16 heads of 128 channels, 16 states a channel
        dict(name="scan_train_bf16", op="scan_train", dtype="bf16", B=2, T=2048, D=2048, N=16, G=1, gate=True, packed=0,
             state=False),
        # a small fp32 run of packed sequences with carried states and two groups of B and C
        dict(name="scan_train_packed_f32", op="scan_train", dtype="f32", B=1, T=777, D=200, N=8, G=2, gate=False, packed=5,
             state=True),
        # a long prompt: B=1, T=16384
        dict(name="scan_prompt_bf16", op="scan_prompt", dtype="bf16", B=1, T=16384, D=2048, N=16, G=1, gate=True, packed=0,
             state=False),
        # one token of each of 128 served sequences
        dict(name="scan_step", op="scan_step", dtype="bf16", B=128, D=4096, N=16, G=1, gate=True, slots=256),
        # the gated head norm of a training batch: B=4, T=4096, 32 heads of 128 channels, one weight for all heads
        dict(name="norm_train_bf16", op="norm_train", dtype="bf16", R=16384, G=32, C=128, center=False, act="sigmoid",
             gate=True, shared=True, bias=False),
        # a centred norm with its activation, odd width, fp32
        dict(name="norm_train_f32", op="norm_train", dtype="f32", R=1500, G=3, C=333, center=True, act="silu", gate=False,
             shared=False, bias=True),
        # the gated head norm of eight served sequences
        dict(name="norm_token", op="norm", dtype="bf16", R=8, G=16, C=128, center=False, act="sigmoid", gate=True, shared=True,
             bias=False),
        # one sequence served alone: 16 heads
        dict(name="kda_step_1", op="kda_step", dtype="bf16", B=1, H=16, HV=16, K=128, V=128, slots=4),
        # a full batch served together: 32 value heads in groups of 4
        dict(name="kda_step_256", op="kda_step", dtype="bf16", B=256, H=8, HV=32, K=128, V=128, slots=256),
    ]


def _log(rng, lo, hi):
    """An integer from lo to hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_train", "conv_step", "scan_train", "scan_prompt", "scan_step", "norm_train", "norm", "kda_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv_train":
        D = _log(rng, 8, 4096)
        B = rng.choice([1, 1, 2, 4])
        T = _log(rng, 2, max(2, min(16384, 30_000_000 // (B * D))))
        packed = rng.randint(2, 9) if B == 1 and T > 40 and rng.random() < 0.5 else 0
        return dict(op=op, dtype=dtype, B=B, T=T, D=D, W=rng.choice([2, 3, 4, 4]), act=rng.random() < 0.8,
                    bias=rng.random() < 0.5, packed=packed, state=rng.random() < 0.5)
    if op == "conv_step":
        B = _log(rng, 1, 256)
        return dict(op=op, dtype=dtype, B=B, D=_log(rng, 8, 8192), W=rng.choice([2, 3, 4, 4]), act=rng.random() < 0.8,
                    bias=rng.random() < 0.5, slots=B + rng.randint(0, 64))
    if op in ("scan_train", "scan_prompt"):
        N = rng.choice([4, 8, 16, 16, 16, 13, 32, 64])
        G = rng.choice([1, 1, 2, 4])
        D = G * _log(rng, max(1, 8 // G), 4096 // G)
        B = rng.choice([1, 1, 2, 4])
        most = (6_000_000 if op == "scan_train" else 24_000_000) * 16 // N
        T = _log(rng, 2, max(2, min(4096 if op == "scan_train" else 16384, most // (B * D))))
        packed = rng.randint(2, 9) if B == 1 and T > 40 and rng.random() < 0.5 else 0
        return dict(op=op, dtype=dtype, B=B, T=T, D=D, N=N, G=G, gate=rng.random() < 0.6, packed=packed,
                    state=rng.random() < 0.5)
    if op == "scan_step":
        B = _log(rng, 1, 256)
        G = rng.choice([1, 1, 2, 4])
        return dict(op=op, dtype=dtype, B=B, D=G * _log(rng, 8, 8192 // G), N=rng.choice([4, 8, 16, 16, 13, 32, 64]), G=G,
                    gate=rng.random() < 0.6, slots=B + rng.randint(0, 64))
    if op in ("norm_train", "norm"):
        C = _log(rng, 8, 4096)
        G = _log(rng, 1, max(1, 8192 // C))
        R = _log(rng, 1, max(1, min(16384, 60_000_000 // (G * C))))
        gate = rng.random() < 0.6
        return dict(op=op, dtype=dtype, R=R, G=G, C=C, center=rng.random() < 0.5, act=rng.choice(["silu", "sigmoid"]),
                    gate=gate, shared=rng.random() < 0.5, bias=rng.random() < 0.5)
    K = rng.choice([16, 64, 128, 128, 128, 96])
    V = K if rng.random() < 0.7 else rng.choice([64, 128, 256, 80])
    H = rng.choice([1, 2, 4, 8, 16])
    HV = H * rng.choice([1, 1, 2, 4])
    B = _log(rng, 1, max(1, min(256, 130_000_000 // (HV * K * V))))
    return dict(op="kda_step", dtype=dtype, B=B, H=H, HV=HV, K=K, V=V, slots=B + rng.randint(0, 8))


# ---------------------------------------------------------------------------------------------
# inputs


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _cuts(case, seed):
    """cu_seqlens of a packed case (sequences of any length from zero on), None of a dense one."""
    if not case["packed"]:
        return None
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    inner = np.sort(r.randint(0, case["T"] + 1, case["packed"] - 1))
    return [0] + [int(c) for c in inner] + [case["T"]]


def prepare(case, seed):
    op, dt = case["op"], _dtype(case)
    gen = torch.Generator("cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=None):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype or dt)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo

    def slots():
        perm = torch.randperm(case["slots"], generator=gen, device="cuda")
        return perm[: case["B"]].to(torch.int32).contiguous()

    s = dict(case=case, op=op)
    f32 = torch.float32
    if op in ("conv_train", "scan_train", "scan_prompt"):
        s["cu"] = _cuts(case, seed)
        cu = s["cu"] or [b * case["T"] for b in range(case["B"] + 1)]
        total = case["B"] * case["T"]
        lens = np.diff(cu)
        n_seq = len(lens)
        # what a program that packs sequences keeps on the GPU beside the list of cuts: every token's sequence and place in it
        s["seq"] = torch.from_numpy(np.repeat(np.arange(n_seq), lens)).cuda()
        s["pos"] = torch.arange(total, device="cuda") - torch.from_numpy(np.repeat(cu[:-1], lens)).cuda()
        s["begin"] = torch.tensor(cu[:-1], device="cuda")
        s["end"] = torch.tensor(cu[1:], device="cuda")
        s["n_seq"] = n_seq
        s["cu_dev"] = torch.tensor(cu, dtype=torch.int32, device="cuda") if s["cu"] else None
    if op.startswith("conv"):
        D, W = case["D"], case["W"]
        shape = (case["B"], D) if op == "conv_step" else (case["B"], case["T"], D)
        s["x"] = normal(*shape)
        s["weight"] = uniform(D, W, lo=-1.0, hi=1.0) / math.sqrt(W)
        s["bias"] = uniform(D, lo=-0.5, hi=0.5) if case["bias"] else None
        if op == "conv_step":
            s["state"] = normal(case["slots"], W - 1, D)
            s["slots"] = slots()
        else:
            s["dy"] = normal(*shape)
            s["h0"] = normal(s["n_seq"], W - 1, D) if case["state"] else None
            s["dfinal"] = normal(s["n_seq"], W - 1, D) if case["state"] else None
    elif op.startswith("scan"):
        D, N, G = case["D"], case["N"], case["G"]
        lead = (case["B"],) if op == "scan_step" else (case["B"], case["T"])
        s["x"] = normal(*lead, D)
        s["dt"] = normal(*lead, D, std=0.5)
        first = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = first + torch.log(-torch.expm1(-first))  # softplus(dt_bias) = first
        s["A"] = -(torch.arange(1, N + 1, device="cuda", dtype=f32) * torch.exp(normal(D, N, std=0.1, dtype=f32)))
        s["B"] = normal(*lead, G, N)
        s["C"] = normal(*lead, G, N)
        s["skip"] = normal(D, std=0.1, mean=1.0, dtype=f32)
        s["z"] = normal(*lead, D) if case["gate"] else None
        if op == "scan_step":
            s["state"] = normal(case["slots"], D, N, std=0.3, dtype=f32)
            s["slots"] = slots()
        else:
            s["h0"] = normal(s["n_seq"], D, N, std=0.3, dtype=f32) if case["state"] else None
            s["dfinal"] = normal(s["n_seq"], D, N, std=0.3, dtype=f32) if case["state"] else None
            s["dy"] = normal(*lead, D) if op == "scan_train" else None
    elif op.startswith("norm"):
        R, G, C = case["R"], case["G"], case["C"]
        s["x"] = normal(R, G * C, mean=0.2)
        s["weight"] = normal(C if case["shared"] else G * C, std=0.1, mean=1.0, dtype=f32)
        s["bias"] = normal(C if case["shared"] else G * C, std=0.1, dtype=f32) if case["bias"] else None
        s["gate"] = normal(R, G * C) if case["gate"] else None
        s["dy"] = normal(R, G * C) if op == "norm_train" else None
    else:
        B, H, HV, K, V = (case[k] for k in ("B", "H", "HV", "K", "V"))
        q, k = normal(B, H, K, dtype=f32), normal(B, H, K, dtype=f32)
        s["q"] = (q / q.norm(dim=-1, keepdim=True)).to(dt)
        s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
        s["v"] = normal(B, HV, V)
        s["g"] = torch.nn.functional.logsigmoid(normal(B, HV, K, mean=3.0, dtype=f32))
        s["beta"] = torch.sigmoid(normal(B, HV, dtype=f32))
        s["state"] = normal(case["slots"], HV, K, V, std=0.1, dtype=f32)
        s["slots"] = slots()
        s["scale"] = 1.0 / math.sqrt(K)
    return s


# ---------------------------------------------------------------------------------------------
# plain forms (32 bits)


def _sig(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _act(x, name):
    return x if name is None else _sig(x) if name == "sigmoid" else x * _sig(x)


def _dact(x, name):
    """The activation's derivative."""
    sg = _sig(x)
    return sg * (1.0 - sg) if name == "sigmoid" else sg * (1.0 + x * (1.0 - sg))


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))


def _taps(s, x, h0, W):
    """[total, W, D]: for each token the W inputs that its output sees."""
    total, D = x.shape
    at = torch.arange(total, device=x.device)
    cols = []
    for j in range(W):
        back = W - 1 - j
        inside = s["pos"] >= back
        rows = x[(at - back).clamp(min=0)]
        # token t sees row (W-1) + pos - back of [h0 | tokens]
        early = h0[s["seq"], (s["pos"] + j).clamp(max=W - 2)] if h0 is not None else torch.zeros_like(rows)
        cols.append(torch.where(inside[:, None], rows, early))
    return torch.stack(cols, 1)


def _conv_train(s):
    c, dt = s["case"], s["x"].dtype
    D, W = c["D"], c["W"]
    x, dy = s["x"].reshape(-1, D).float(), s["dy"].reshape(-1, D).float()
    h0 = s["h0"].float() if s["h0"] is not None else None
    taps = _taps(s, x, h0, W)
    u = (taps * s["weight"].t()[None]).sum(1)
    if s["bias"] is not None:
        u = u + s["bias"]
    y = _act(u, "silu" if c["act"] else None)
    du = dy * _dact(u, "silu") if c["act"] else dy
    out = dict(y=y.to(dt).reshape(s["x"].shape), dweight=(du[:, None] * taps).sum(0).t().contiguous())
    if s["bias"] is not None:
        out["dbias"] = du.sum(0)
    # the gradient of every row of [h0 | tokens]: tap j of token t is row pos + j
    n = s["n_seq"]
    hist = x.new_zeros(x.shape[0] + n * (W - 1), D)
    row0 = s["begin"] + torch.arange(n, device=x.device) * (W - 1)  # where a sequence's history begins
    at = row0[s["seq"]] + s["pos"]
    for j in range(W):
        hist[at + j] += du * s["weight"][:, j]
    if s["dfinal"] is not None:
        last = (row0 + (s["end"] - s["begin"]))[:, None] + torch.arange(W - 1, device=x.device)
        hist[last] += s["dfinal"].float()
    out["dx"] = hist[at + (W - 1)].to(dt).reshape(s["x"].shape)
    if h0 is not None:
        lead = row0[:, None] + torch.arange(W - 1, device=x.device)
        full = x.new_zeros(x.shape[0] + n * (W - 1), D)
        full[at + (W - 1)] = x
        full[lead] = h0
        last = (row0 + (s["end"] - s["begin"]))[:, None] + torch.arange(W - 1, device=x.device)
        out["final_state"] = full[last].to(dt)
        out["dh0"] = hist[lead].to(dt)
    return out


def _conv_step(s):
    c, dt = s["case"], s["x"].dtype
    at = s["slots"].long()
    win = torch.cat([s["state"][at], s["x"][:, None]], 1)
    u = (win.float() * s["weight"].t()[None]).sum(1)
    if s["bias"] is not None:
        u = u + s["bias"]
    s["state"][at] = win[:, 1:]
    return dict(y=_act(u, "silu" if c["act"] else None).to(dt), state=s["state"])


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 0, by doubling."""
    step = 1
    while step < a.shape[0]:
        b = torch.cat([b[:step], torch.addcmul(b[step:], a[step:], b[:-step])])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _scan_seq(s):
    """The selective scan over whole sequences, with its gradients in a training case."""
    c, dt_ = s["case"], s["x"].dtype
    D, N, G = c["D"], c["N"], c["G"]
    total, n = c["B"] * c["T"], s["n_seq"]
    x = s["x"].reshape(total, D).float()
    raw = s["dt"].reshape(total, D).float() + s["dt_bias"]
    dt = _softplus(raw)
    Bm, Cm = (s[k].reshape(total, G, N).float().repeat_interleave(D // G, 1) for k in ("B", "C"))  # [total, D, N]
    some = s["end"] > s["begin"]
    # the first token of each sequence that has one (an empty one's place is a dummy row behind the last)
    heads = torch.where(some, s["begin"], torch.full_like(s["begin"], total))
    tails = torch.where(some, s["end"] - 1, torch.full_like(s["end"], total))
    a = torch.exp(dt[:, :, None] * s["A"])
    h0 = s["h0"] if s["h0"] is not None else x.new_zeros(n, D, N)
    first = x.new_zeros(total + 1, dtype=torch.bool)
    first[heads] = True
    before = x.new_zeros(total + 1, D, N)  # the state before a sequence's first token, zero elsewhere
    before[heads] = h0
    first, before = first[:total], before[:total]
    cut = torch.where(first[:, None, None], torch.zeros_like(a), a)
    h = _scan(cut, torch.addcmul((dt * x)[:, :, None] * Bm, a, before))
    pre = (h * Cm).sum(-1) + s["skip"] * x
    z = s["z"].reshape(total, D).float() if s["z"] is not None else None
    y = pre * _act(z, "silu") if z is not None else pre
    last = torch.cat([h, h.new_zeros(1, D, N)])[tails]
    out = dict(y=y.to(dt_).reshape(s["x"].shape), final_state=torch.where(some[:, None, None], last, h0))
    if c["op"] == "scan_prompt":
        return out
    dy = s["dy"].reshape(total, D).float()
    if z is not None:
        out["dz"] = (dy * pre * _dact(z, "silu")).to(dt_).reshape(s["x"].shape)
        dy = dy * _act(z, "silu")
    dfinal = s["dfinal"] if s["dfinal"] is not None else x.new_zeros(n, D, N)
    after = x.new_zeros(total + 1, D, N)
    after[tails] = dfinal
    # r_t = C_t dy_t + a_{t+1} r_{t+1}
    nxt = torch.cat([cut[1:], torch.zeros_like(cut[:1])])
    r = _scan(nxt.flip(0), (dy[:, :, None] * Cm + after[:total]).flip(0)).flip(0)
    prev = torch.where(first[:, None, None], before, torch.cat([torch.zeros_like(h[:1]), h[:-1]]))
    q = a * r
    p = q * prev
    rb = (r * Bm).sum(-1)
    ddt = (x * rb + (p * s["A"]).sum(-1)) * _sig(raw)
    out["dx"] = (dt * rb + s["skip"] * dy).to(dt_).reshape(s["x"].shape)
    out["ddt"] = ddt.to(dt_).reshape(s["x"].shape)
    out["ddt_bias"] = ddt.sum(0)
    out["dA"] = (dt[:, :, None] * p).sum(0)
    out["dskip"] = (dy * x).sum(0)
    out["dB"] = (r * (dt * x)[:, :, None]).reshape(total, G, D // G, N).sum(2).to(dt_).reshape(s["B"].shape)
    out["dC"] = (h * dy[:, :, None]).reshape(total, G, D // G, N).sum(2).to(dt_).reshape(s["C"].shape)
    if s["h0"] is not None:
        out["dh0"] = torch.where(some[:, None, None], torch.cat([q, q.new_zeros(1, D, N)])[heads], dfinal)
    return out


def _scan_step(s):
    c, dt_ = s["case"], s["x"].dtype
    at = s["slots"].long()
    x = s["x"].float()
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    Bm, Cm = (s[k].float().repeat_interleave(c["D"] // c["G"], 1) for k in ("B", "C"))
    h = torch.exp(dt[:, :, None] * s["A"]) * s["state"][at] + (dt * x)[:, :, None] * Bm
    y = (h * Cm).sum(-1) + s["skip"] * x
    if s["z"] is not None:
        y = y * _act(s["z"].float(), "silu")
    s["state"][at] = h
    return dict(y=y.to(dt_), state=s["state"])


def _norm(s):
    c, dt_ = s["case"], s["x"].dtype
    shape = (c["R"], c["G"], c["C"])
    x = s["x"].reshape(shape).float()
    w = s["weight"].reshape(-1, c["C"])
    mean = x.mean(-1, keepdim=True) if c["center"] else 0.0
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + LN_EPS)
    n = (x - mean) * rstd
    u = n * w
    if s["bias"] is not None:
        u = u + s["bias"].reshape(-1, c["C"])
    gate = s["gate"].reshape(shape).float() if s["gate"] is not None else None
    y = u * _act(gate, c["act"]) if gate is not None else _act(u, c["act"])
    out = dict(y=y.to(dt_).reshape(s["x"].shape))
    if c["op"] == "norm":
        return out
    dy = s["dy"].reshape(shape).float()
    if gate is not None:
        out["dgate"] = (dy * u * _dact(gate, c["act"])).to(dt_).reshape(s["x"].shape)
        du = dy * _act(gate, c["act"])
    else:
        du = dy * _dact(u, c["act"])
    over = (0, 1) if c["shared"] else (0,)
    out["dweight"] = (du * n).sum(over).reshape(-1)
    if s["bias"] is not None:
        out["dbias"] = du.sum(over).reshape(-1)
    dn = du * w
    corr = (dn * n).mean(-1, keepdim=True)
    dx = dn - n * corr
    if c["center"]:
        dx = dx - dn.mean(-1, keepdim=True)
    out["dx"] = (dx * rstd).to(dt_).reshape(s["x"].shape)
    return out


def _kda_step(s):
    c = s["case"]
    at = s["slots"].long()
    rep = c["HV"] // c["H"]
    q, k = (s[n].float().repeat_interleave(rep, 1) for n in ("q", "k"))
    S = torch.exp(s["g"])[..., None] * s["state"][at]
    u = s["beta"][..., None] * (s["v"].float() - (k[..., None] * S).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["state"][at] = S
    return dict(o=((q[..., None] * S).sum(-2) * s["scale"]).to(s["v"].dtype), state=s["state"])


def _plain(s):
    op = s["op"]
    if op == "conv_train":
        return _conv_train(s)
    if op == "conv_step":
        return _conv_step(s)
    if op in ("scan_train", "scan_prompt"):
        return _scan_seq(s)
    if op == "scan_step":
        return _scan_step(s)
    return _kda_step(s) if op == "kda_step" else _norm(s)


# ---------------------------------------------------------------------------------------------
# the library's calls


def _library(s):
    from chunked_gated_delta_09_amd import layers
    c, op = s["case"], s["op"]
    packed = dict(cu_seqlens=s.get("cu"), cu_seqlens_dev=s.get("cu_dev"))
    if op == "conv_train":
        act = "silu" if c["act"] else None
        f = layers.short_conv(s["x"], s["weight"], bias=s["bias"], h0=s["h0"], **packed, activation=act,
                              output_final_state=s["h0"] is not None)
        b = layers.short_conv_bwd(s["x"], s["weight"], s["dy"], bias=s["bias"], h0=s["h0"], dfinal=s["dfinal"],
                                  **packed, activation=act)
        out = dict(y=f["y"], dweight=b["dweight"], dx=b["dx"])
        if s["bias"] is not None:
            out["dbias"] = b["dbias"]
        if s["h0"] is not None:
            out["final_state"], out["dh0"] = f["final_state"], b["dh0"]
        return out
    if op == "conv_step":
        y = layers.short_conv_step(s["x"], s["state"], s["weight"], bias=s["bias"], slots=s["slots"],
                                   activation="silu" if c["act"] else None)
        return dict(y=y, state=s["state"])
    if op in ("scan_train", "scan_prompt"):
        train = op == "scan_train"
        f = layers.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"],
                                  h0=s["h0"], **packed, dt_softplus=True, save=train)
        out = dict(y=f["y"], final_state=f["final_state"])
        if train:
            b = layers.selective_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], f["states"], s["dy"], skip=s["skip"],
                                          z=s["z"], dt_bias=s["dt_bias"], dfinal=s["dfinal"], **packed,
                                          dt_softplus=True, output_dh0=s["h0"] is not None)
            names = ["dx", "ddt", "ddt_bias", "dA", "dskip", "dB", "dC"]
            names += ["dz"] if s["z"] is not None else []
            names += ["dh0"] if s["h0"] is not None else []
            out.update((k, b[k]) for k in names)
        return out
    if op == "scan_step":
        y = layers.selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], slots=s["slots"],
                                       skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True)
        return dict(y=y, state=s["state"])
    if op == "kda_step":
        o = layers.kda_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"], scale=s["scale"])
        return dict(o=o, state=s["state"])
    kw = dict(weight=s["weight"], bias=s["bias"], gate=s["gate"], activation=c["act"], center=c["center"], eps=LN_EPS)
    out = dict(y=layers.group_norm(s["x"], c["G"], **kw))
    if op == "norm_train":
        b = layers.group_norm_bwd(s["x"], c["G"], s["dy"], **kw)
        out.update(dx=b["dx"], dweight=b["dweight"])
        if s["bias"] is not None:
            out["dbias"] = b["dbias"]
        if s["gate"] is not None:
            out["dgate"] = b["dgate"]
    return out


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    c, es = case, 4 if case["dtype"] == "f32" else 2
    op = c["op"]
    if op == "conv_train":
        e = c["B"] * c["T"] * c["D"]
        n = (c["packed"] or c["B"]) * (c["W"] - 1) * c["D"] if c["state"] else 0
        return dict(bytes=e * es * 4 + 4 * n * es + c["D"] * c["W"] * 8, flops=e * (6 * c["W"] + (14 if c["act"] else 0)))
    if op == "conv_step":
        e = c["B"] * c["D"]
        return dict(bytes=e * es * (2 + 2 * (c["W"] - 1)) + c["D"] * c["W"] * 4, flops=e * (2 * c["W"] + 5))
    if op in ("scan_train", "scan_prompt"):
        t, D, N = c["B"] * c["T"], c["D"], c["N"]
        n_seq = c["packed"] or c["B"]
        st = n_seq * D * N * 4
        ed = t * D * es
        bc = 2 * t * c["G"] * N * es
        par = D * N * 4 + 2 * D * 4
        gate = 1 if c["gate"] else 0
        if op == "scan_prompt":
            return dict(bytes=ed * (3 + gate) + bc + par + st * (2 if c["state"] else 1), flops=t * D * (N * 6 + 10))
        # x, dt, z, dy and B, C in; y, dx, ddt, dz and dB, dC out
        return dict(bytes=ed * (6 + 2 * gate) + 2 * bc + 2 * par + st * (4 if c["state"] else 1), flops=t * D * (N * 20 + 30))
    if op == "scan_step":
        e = c["B"] * c["D"]
        return dict(bytes=e * (c["N"] * 8 + es * (3 + (1 if c["gate"] else 0))) + 2 * c["B"] * c["G"] * c["N"] * es
                    + c["D"] * c["N"] * 4, flops=e * (6 * c["N"] + 10))
    if op == "kda_step":
        st = c["B"] * c["HV"] * c["K"] * c["V"]
        return dict(bytes=st * 8 + c["B"] * (2 * c["H"] * c["K"] * es + 2 * c["HV"] * c["V"] * es + c["HV"] * (c["K"] + 1) * 4),
                    flops=st * 7)
    e = c["R"] * c["G"] * c["C"]
    gate = 1 if c["gate"] else 0
    par = (c["C"] if c["shared"] else c["G"] * c["C"]) * 4
    if op == "norm":
        return dict(bytes=e * es * (2 + gate) + par, flops=e * 10)
    return dict(bytes=e * es * (4 + 2 * gate) + 2 * par, flops=e * 30)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _silu64(v):
    return v * torch.sigmoid(v)


def _exact_conv_seq(c, x, w, b, h0, dy, dfinal):
    """One sequence. x, dy [L, D]; h0, dfinal [W-1, D]: the history is [h0 | x]."""
    W, L = c["W"], x.shape[0]
    hist = torch.cat([h0, x])
    u = sum(hist[j:j + L] * w[:, j] for j in range(W)) + b
    sg = torch.sigmoid(u)
    y, du = (u * sg, dy * (sg + u * sg * (1 - sg))) if c["act"] else (u, dy)
    dhist = torch.zeros_like(hist)
    for j in range(W):
        dhist[j:j + L] += du * w[:, j]
    dhist[L:] += dfinal
    dw = torch.stack([(du * hist[j:j + L]).sum(0) for j in range(W)], 1)
    return y, dhist[W - 1:], dhist[:W - 1], hist[L:], dw, du.sum(0)


def _exact_scan_seq(c, x, raw, A, Bm, Cm, skip, z, h0, dy, dfinal):
    """One batch of sequences of one length, token by token. x, raw, z, dy [n, L, D]; Bm, Cm [n, L, G, N]."""
    n, L, D = x.shape
    G = c["G"]
    dt = torch.nn.functional.softplus(raw, threshold=700.0)
    train = dy is not None
    wide = (lambda v: v[:, :, None, :].expand(n, G, D // G, c["N"]).reshape(n, D, c["N"]))
    h, ys, hs = h0, [], [h0] if train else None
    for t in range(L):
        h = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * x[:, t])[..., None] * wide(Bm[:, t])
        ys.append((h * wide(Cm[:, t])).sum(-1) + skip * x[:, t])
        if train:
            hs.append(h)
    pre = torch.stack(ys, 1) if L else torch.zeros_like(x)
    sz = torch.sigmoid(z) if z is not None else None
    out = dict(y=pre * z * sz if z is not None else pre, final_state=h)
    if not train:
        return out
    if z is not None:
        out["dz"] = dy * pre * (sz + z * sz * (1 - sz))
        dy = dy * z * sz
    dx, ddt, dB, dC = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(Bm), torch.zeros_like(Cm)
    dA, dh = torch.zeros_like(A), dfinal
    for t in range(L - 1, -1, -1):
        dh = dh + dy[:, t, :, None] * wide(Cm[:, t])
        dC[:, t] = (hs[t + 1] * dy[:, t, :, None]).reshape(n, G, D // G, c["N"]).sum(2)
        dB[:, t] = (dh * (dt[:, t] * x[:, t])[..., None]).reshape(n, G, D // G, c["N"]).sum(2)
        into = (dh * wide(Bm[:, t])).sum(-1)
        a = torch.exp(dt[:, t, :, None] * A)
        lam = dh * a * hs[t]
        dx[:, t] = dt[:, t] * into + skip * dy[:, t]
        ddt[:, t] = x[:, t] * into + (lam * A).sum(-1)
        dA += (lam * dt[:, t, :, None]).sum(0)
        dh = dh * a
    ddt = ddt * torch.sigmoid(raw)
    out.update(dx=dx, ddt=ddt, dB=dB, dC=dC, dA=dA, dh0=dh, ddt_bias=ddt.sum((0, 1)), dskip=(dy * x).sum((0, 1)))
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    op = c["op"]
    if op == "conv_train":
        D, W = c["D"], c["W"]
        cu = s["cu"] or [b * c["T"] for b in range(c["B"] + 1)]
        x, dy = s["x"].reshape(-1, D), s["dy"].reshape(-1, D)
        zero = x.new_zeros(W - 1, D)
        b = s["bias"] if s["bias"] is not None else x.new_zeros(D)
        parts = [_exact_conv_seq(c, x[lo:hi], s["weight"], b, s["h0"][i] if c["state"] else zero, dy[lo:hi],
                                 s["dfinal"][i] if c["state"] else zero) for i, (lo, hi) in enumerate(zip(cu[:-1], cu[1:]))]
        out = dict(y=torch.cat([p[0] for p in parts]).reshape(s["x"].shape),
                   dx=torch.cat([p[1] for p in parts]).reshape(s["x"].shape), dweight=sum(p[4] for p in parts))
        if c["bias"]:
            out["dbias"] = sum(p[5] for p in parts)
        if c["state"]:
            out["dh0"], out["final_state"] = torch.stack([p[2] for p in parts]), torch.stack([p[3] for p in parts])
        return out
    if op == "conv_step":
        at, W = s["slots"].long(), c["W"]
        old = s["state"][at]
        u = s["x"] * s["weight"][:, W - 1] + (s["bias"] if s["bias"] is not None else 0.0)
        for j in range(W - 1):
            u = u + old[:, j] * s["weight"][:, j]
        state = s["state"].clone()
        state[at, : W - 2] = old[:, 1:]
        state[at, W - 2] = s["x"]
        return dict(y=_silu64(u) if c["act"] else u, state=state)
    if op in ("scan_train", "scan_prompt"):
        D, N = c["D"], c["N"]
        raw = s["dt"] + s["dt_bias"]
        zero = raw.new_zeros(1, D, N)
        train = op == "scan_train"
        if s["cu"] is None:
            z0 = zero.expand(c["B"], D, N)
            o = _exact_scan_seq(c, s["x"], raw, s["A"], s["B"], s["C"], s["skip"], s["z"], s["h0"] if c["state"] else z0,
                                s["dy"], s["dfinal"] if c["state"] else z0)
        else:
            pick = (lambda v, lo, hi: None if v is None else v[:, lo:hi])
            parts = [_exact_scan_seq(c, *(pick(v, lo, hi) for v in (s["x"], raw)), s["A"],
                                     *(pick(v, lo, hi) for v in (s["B"], s["C"])), s["skip"], pick(s["z"], lo, hi),
                                     s["h0"][i:i + 1] if c["state"] else zero, pick(s["dy"], lo, hi),
                                     s["dfinal"][i:i + 1] if c["state"] else zero)
                     for i, (lo, hi) in enumerate(zip(s["cu"][:-1], s["cu"][1:]))]
            o = {}
            for k in parts[0]:
                v = [p[k] for p in parts]
                o[k] = sum(v) if k in ("dA", "ddt_bias", "dskip") else torch.cat(v, 0 if k in ("final_state", "dh0") else 1)
        if train and not c["state"]:
            del o["dh0"]
        return o
    if op == "scan_step":
        at = s["slots"].long()
        dt = torch.nn.functional.softplus(s["dt"] + s["dt_bias"], threshold=700.0)
        grp = torch.arange(c["D"], device=at.device) // (c["D"] // c["G"])
        h = torch.exp(dt[..., None] * s["A"]) * s["state"][at] + s["B"][:, grp] * (dt * s["x"])[..., None]
        y = (h * s["C"][:, grp]).sum(-1) + s["skip"] * s["x"]
        state = s["state"].clone()
        state[at] = h
        return dict(y=y * _silu64(s["z"]) if s["z"] is not None else y, state=state)
    if op == "kda_step":
        at, grp = s["slots"].long(), torch.arange(c["HV"], device=s["slots"].device) // (c["HV"] // c["H"])
        q, k = s["q"][:, grp], s["k"][:, grp]
        S = s["state"][at] * torch.exp(s["g"])[..., None]
        read = torch.matmul(k[:, :, None, :], S)[:, :, 0]
        S = S + torch.matmul(k[..., None], (s["beta"][..., None] * (s["v"] - read))[:, :, None, :])
        state = s["state"].clone()
        state[at] = S
        return dict(o=torch.matmul(q[:, :, None, :], S)[:, :, 0] * s["scale"], state=state)
    act = torch.sigmoid if c["act"] == "sigmoid" else _silu64
    leaf = [s["x"], s["weight"]] + [s[k] for k in ("bias", "gate") if s[k] is not None]
    names = ["dx", "dweight"] + ["d" + k for k in ("bias", "gate") if s[k] is not None]
    leaf = [v.requires_grad_(op == "norm_train") for v in leaf]
    x = s["x"].reshape(c["R"], c["G"], c["C"])
    x = x - x.mean(-1, keepdim=True) if c["center"] else x
    u = x / torch.sqrt((x * x).mean(-1, keepdim=True) + LN_EPS) * s["weight"].reshape(-1, c["C"])
    if s["bias"] is not None:
        u = u + s["bias"].reshape(-1, c["C"])
    u = u.reshape(s["x"].shape)
    y = u * act(s["gate"]) if s["gate"] is not None else act(u)
    out = dict(y=y.detach())
    if op == "norm_train":
        out.update(zip(names, torch.autograd.grad(y, leaf, s["dy"])))
    return out
