"""Plain 64-bit forms of the layer operators on the CPU, token by token from their definitions, and
the tolerances of the tests that use them."""
import torch

F64 = torch.float64
ACT = {None: lambda v: v, "silu": lambda v: v * torch.sigmoid(v), "sigmoid": torch.sigmoid}


def half_step(dtype):
    """The largest relative error of rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def close(got, ref, dtype, ops, what=""):
    """Every value within the rounding of its type, plus `ops` fp32 roundings (each at most 2^-24)
    of terms as large as the tensor's largest value. `ops` is 64 for the constant work of an
    operator (activations: a few hardware functions of one unit in the last place each; trees of
    sums) and 4 for each token that a state or a sum over tokens passes through."""
    got, ref = got.detach().cpu().to(F64), ref.detach().to(F64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), what
    if not ref.numel():
        return
    bound = half_step(dtype) * ref.abs() + ops * 2.0 ** -24 * ref.abs().max()
    if dtype != torch.float32:
        bound = bound * (1 + 2.0 ** -8)  # the rounded value's own step may be the next larger one
    off = (got - ref).abs()
    worst = (off / bound.clamp(min=1e-300)).max().item()
    assert (off <= bound).all(), f"{what}: {worst:.3g} times the bound"


def cuts_of(B, T, cu):
    return list(cu) if cu is not None else [b * T for b in range(B + 1)]


def conv(x, w, bias, h0, act, cu):
    """x [B,T,D] -> y, final_state."""
    B, T, D = x.shape
    W = w.shape[1]
    ys, fin = [], []
    flat = x.reshape(B * T, D)
    cuts = cuts_of(B, T, cu)
    for n, (lo, hi) in enumerate(zip(cuts[:-1], cuts[1:])):
        lead = h0[n] if h0 is not None else torch.zeros(W - 1, D, dtype=F64)
        hist = torch.cat([lead, flat[lo:hi]])
        for t in range(hi - lo):
            u = (hist[t:t + W] * w.t()).sum(0)
            ys.append(ACT[act](u + bias if bias is not None else u))
        fin.append(hist[hi - lo:])
    y = torch.stack(ys).reshape(B, T, D) if ys else torch.zeros(B, T, D, dtype=F64)
    return y, torch.stack(fin)


def scan(x, dt, A, Bm, Cm, skip, z, dt_bias, h0, softplus, cu):
    """-> y [B,T,D], final_state [N,D,NS]."""
    B, T, D = x.shape
    G, NS = Bm.shape[2:]
    raw = dt + dt_bias if dt_bias is not None else dt
    # logaddexp: its derivative is the sigmoid at 0 too, where |raw| and max(raw, 0) have none
    step = (torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw).reshape(B * T, D)
    xf, bf, cf = x.reshape(B * T, D), Bm.reshape(B * T, G, NS), Cm.reshape(B * T, G, NS)
    cuts, ys, fin = cuts_of(B, T, cu), [], []
    for n, (lo, hi) in enumerate(zip(cuts[:-1], cuts[1:])):
        h = h0[n] if h0 is not None else torch.zeros(D, NS, dtype=F64)
        for t in range(lo, hi):
            b, c = (v[t].repeat_interleave(D // G, 0) for v in (bf, cf))
            h = torch.exp(step[t, :, None] * A) * h + (step[t] * xf[t])[:, None] * b
            y = (h * c).sum(1)
            ys.append(y + skip * xf[t] if skip is not None else y)
        fin.append(h)
    y = torch.stack(ys).reshape(B, T, D) if ys else torch.zeros(B, T, D, dtype=F64)
    return (y * ACT["silu"](z) if z is not None else y), torch.stack(fin)


def norm(x, groups, w, bias, gate, act, center, eps):
    shape = x.shape
    C = shape[-1] // groups
    v = x.reshape(-1, groups, C)
    if center:
        v = v - v.mean(-1, keepdim=True)
    u = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    if w is not None:
        u = u * w.reshape(-1, C)
    if bias is not None:
        u = u + bias.reshape(-1, C)
    u = u.reshape(shape)
    return u * ACT[act](gate) if gate is not None else ACT[act](u)


def kda_token(q, k, v, g, beta, S, scale):
    """One token: q, k [B,H,K], v [B,HV,V], g [B,HV,K], beta [B,HV], S [B,HV,K,V] -> o, S."""
    rep = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    S = torch.exp(g)[..., None] * S
    u = beta[..., None] * (v - (k[..., None] * S).sum(2))
    S = S + k[..., None] * u[:, :, None]
    return scale * (q[..., None] * S).sum(2), S
