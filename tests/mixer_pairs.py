"""Linear attention in 64 bits on the CPU over all pairs of a sequence's tokens, for long sequences of many heads: the values and
magnitudes of ``mixer_ref.linear_all``, which goes token by token."""
import torch

from tests import mixer_ref as ref

HEADS = 64  # at a time


def decay(x):
    """e^x, zero where fp32 holds no normal number: e^-200, a reset, is 1e-87 and its products are zero in fp32, while the bounds are
    relative to sums as small as itself. (A product of decays is at least 2^-126 only if each of them is, so it
    does not matter how the kernels form it; between e^-87 and e^-200 the tests have no total.)"""
    y = torch.exp(x)
    return y * (y >= 2.0 ** -126)


def _heads(q, k, v, g, h0, do, df, scale):
    """One sequence: q, k [h, L, K]; v, do [h, L, V]; g [h, L]; h0, df [h, K, V]."""
    L = q.shape[1]
    G = g.cumsum(1)
    low = torch.ones(L, L, dtype=torch.bool).tril()
    pair = decay((G[:, :, None] - G[:, None, :]).masked_fill(~low, -float("inf")))
    start, rest, whole = decay(G)[..., None], decay(G[:, -1:] - G)[..., None], decay(G[:, -1])[:, None, None]
    A, B = scale * (q @ k.mT), do @ v.mT
    out = dict(o=(A * pair) @ v + scale * start * (q @ h0), final_state=whole * h0 + (rest * k).mT @ v,
               dq=(scale * B * pair) @ k + scale * start * (do @ h0.mT), dk=(scale * B * pair).mT @ q + rest * (v @ df.mT),
               dv=(A * pair).mT @ do + rest * (k @ df), dh0=scale * (start * q).mT @ do + whole * df)
    # every path is counted for the decays between its two ends: pairs, first state to output, key to final state, state to state
    M = A * B * pair * ~torch.eye(L, dtype=torch.bool)
    first = scale * start[..., 0] * ((q @ h0) * do).sum(2)
    last = rest[..., 0] * ((k @ df) * v).sum(2)
    dg = (M.sum(2) - M.sum(1) + first).flip(1).cumsum(1).flip(1) + last.cumsum(1) - last
    out["dg"] = dg + whole[..., 0] * (h0 * df).sum((1, 2))[:, None]
    return out


def linear_all(q, k, v, g, h0, do, dfinal, scale, cu):
    B, T, H, K = q.shape
    HV, V = v.shape[2:]
    rep, cuts = HV // H, ref.cuts_of(B, T, cu)
    N = len(cuts) - 1
    g = g if g.dim() == 3 else g.expand(B, T, HV)
    out = {}
    for mag in (False, True):
        f = (lambda t: t.abs()) if mag else (lambda t: t)
        def rows(t, heads):
            return f(t).reshape(B * T, -1, t.shape[-1])[:, heads].transpose(0, 1)
        first, left = (torch.zeros(N, HV, K, V, dtype=ref.F64) if t is None else f(t) for t in (h0, dfinal))
        res = dict(o=torch.zeros(B * T, HV, V), dq=torch.zeros(B * T, HV, K), dk=torch.zeros(B * T, HV, K),
                   dv=torch.zeros(B * T, HV, V), dg=torch.zeros(B * T, HV))
        res = {n: t.to(ref.F64) for n, t in res.items()}
        res["final_state"], res["dh0"] = first.clone(), left.clone()
        for a in range(0, HV, HEADS):
            hv = torch.arange(a, min(a + HEADS, HV))
            x = [rows(q, hv // rep), rows(k, hv // rep), rows(v, hv), g.reshape(B * T, HV)[:, hv].T, rows(do, hv)]
            for n, (lo, hi) in enumerate(zip(cuts[:-1], cuts[1:])):
                if hi == lo:
                    continue
                qs, ks, vs, gs, ds = (t[:, lo:hi] for t in x)
                r = _heads(qs, ks, vs, gs, first[n, hv], ds, left[n, hv], abs(scale) if mag else scale)
                for name in ("o", "dq", "dk", "dv"):
                    res[name][lo:hi, hv] = r[name].transpose(0, 1)
                dg = r["dg"]
                if mag:
                    # suffix sums of q.dq and k.dk, whose terms cancel
                    dg = dg + ((qs * r["dq"]).sum(2) + (ks * r["dk"]).sum(2)).flip(1).cumsum(1).flip(1)
                res["dg"][lo:hi, hv] = dg.T
                res["final_state"][n, hv], res["dh0"][n, hv] = r["final_state"], r["dh0"]
        for name in ("dq", "dk"):
            res[name] = res[name].reshape(B, T, H, rep, K).sum(3)
        for name in ("o", "dv"):
            res[name] = res[name].reshape(B, T, HV, V)
        res["dg"] = res["dg"].reshape(B, T, HV)
        out[mag] = res
    return {n: (out[False][n], out[True][n]) for n in out[False] if n != "dh0" or h0 is not None}


def shared(want):
    """The same for one decay a head."""
    return dict(want, dg=tuple(t.sum((0, 1)) for t in want["dg"]))
