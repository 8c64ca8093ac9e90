"""Training entry point: the chunked KDA forward (output o and final state) with its backward
wired into torch autograd.

Forward: `kda_fwd_states` (per-chunk states S_in, WY/UT inverses, o, S_T). Backward:
`kda_chunk_bwd` on the saved states and inverses with dO and the gradient of S_T. With
``save_operands`` (the default) the pair is `kda_fwd_states_save` / `kda_chunk_bwd_saved`: the
forward also keeps the backward's chunk operands (kr, -w^T, Q'^T, e^gam), so the backward
skips their recomputation (FLA chunk_bwd page: the disable_recompute switch). Both run
entirely in the HIP library; this module only marshals tensors (FLA chunk_bwd page:
`chunk_kda_bwd` takes the forward's saved inverses and states and returns dq, dk, dv,
dbeta, dg, dh0; FlashKDA backward page: the chunk kernel's inputs are the forward
workspace and dO).

`short_conv`, `selective_scan` and `group_norm` are the operators of ``layers`` in the same form.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import chunk_bwd, fwd_states, layers


def _kept(cu_seqlens):
    """The cuts as they are now: the backward may run after the caller has refilled their list or buffer."""
    if cu_seqlens is None:
        return None
    return tuple(int(c) for c in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens))


class KdaChunkFunction(torch.autograd.Function):
    """o, S_T = KDA(q, k, v, g, beta, h0) with gradients for q, k, v, g, beta and h0.

    g is the per-channel log decay (fp32, natural log), beta the write strength (fp32). The
    gradient of S_T reaches the backward in the input precision (bf16 for bf16 inputs), the
    precision in which the library takes dS_final."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, h0, cu_seqlens, C, scale, output_final_state, beta_logits, save_operands):
        cu_seqlens, scale = _kept(cu_seqlens), None if scale is None else float(scale)
        fw = fwd_states(q, k, v, g, beta, h0=h0, cu_seqlens=cu_seqlens, C=C, scale=scale, output_o=True,
                        output_final_state=output_final_state, beta_logits=beta_logits, save=save_operands)
        ctx.save_for_backward(q, k, v, g, beta, fw["states"], fw["inv"], fw["saved"])
        ctx.cu_seqlens, ctx.C, ctx.scale, ctx.beta_logits = cu_seqlens, C, scale, beta_logits
        ctx.h0_dtype = None if h0 is None else h0.dtype
        return fw["o"], fw["final_state"]

    @staticmethod
    def backward(ctx, do, dfinal):
        q, k, v, g, beta, states, inv, saved = ctx.saved_tensors
        dS = None if dfinal is None else dfinal.to(q.dtype).contiguous()
        r = chunk_bwd(q, k, v, g, beta, states, inv, do.to(q.dtype).contiguous(), dS_final=dS,
                      cu_seqlens=ctx.cu_seqlens, C=ctx.C, scale=ctx.scale, output_dh0=ctx.h0_dtype is not None,
                      beta_logits=ctx.beta_logits, saved=saved)
        dh0 = None if ctx.h0_dtype is None else r["dh0"].to(ctx.h0_dtype)
        return r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"], dh0, None, None, None, None, None, None


def kda_chunk(q, k, v, g, beta, h0=None, cu_seqlens=None, C=64, scale=None, output_final_state=True,
              beta_logits=False, save_operands=True):
    """Differentiable chunked KDA. Shapes: q, k [B,T,H,K]; v [B,T,HV,V]; g [B,T,HV,K] fp32;
    beta [B,T,HV] fp32 (write strengths, or their logits with ``beta_logits``); h0
    [N,HV,K,V] or None; packed sequences via cu_seqlens (host list, B = 1).
    ``save_operands``: keep the backward's chunk operands from the forward (saved-operand
    mode) rather than recomputing them in the backward. Returns (o [B,T,HV,V], S_T
    [N,HV,K,V] fp32 or None)."""
    return KdaChunkFunction.apply(q, k, v, g, beta, h0, cu_seqlens, C, scale, output_final_state, beta_logits,
                                  save_operands)


def _kept_both(cu_seqlens, cu_seqlens_dev, device):
    """The cuts as _kept has them, and one copy of them on the GPU for the forward and the backward."""
    cu_seqlens = _kept(cu_seqlens)
    if cu_seqlens is not None and cu_seqlens_dev is None:
        cu_seqlens_dev = torch.tensor(cu_seqlens, dtype=torch.int32, device=device)
    return cu_seqlens, cu_seqlens_dev


class ShortConvFunction(torch.autograd.Function):
    """y, final_state = short_conv(x, weight, bias, h0) with gradients for all four."""

    @staticmethod
    def forward(ctx, x, weight, bias, h0, cu_seqlens, cu_seqlens_dev, activation, output_final_state):
        cu_seqlens, cu_seqlens_dev = _kept_both(cu_seqlens, cu_seqlens_dev, x.device)
        f = layers.short_conv(x, weight, bias=bias, h0=h0, cu_seqlens=cu_seqlens, cu_seqlens_dev=cu_seqlens_dev,
                              activation=activation, output_final_state=output_final_state)
        ctx.save_for_backward(x, weight, bias, h0, cu_seqlens_dev)
        ctx.cu_seqlens, ctx.activation = cu_seqlens, activation
        ctx.set_materialize_grads(False)
        return f["y"], f["final_state"]

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal):
        x, weight, bias, h0, cu_dev = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.contiguous()
        r = layers.short_conv_bwd(x, weight, dy, bias=bias, h0=h0, dfinal=None if dfinal is None else dfinal.contiguous(),
                                  cu_seqlens=ctx.cu_seqlens, cu_seqlens_dev=cu_dev, activation=ctx.activation)
        return r["dx"], r["dweight"], r["dbias"], r["dh0"], None, None, None, None


def short_conv(x, weight, bias=None, h0=None, cu_seqlens=None, cu_seqlens_dev=None, activation="silu",
               output_final_state=False):
    """Differentiable ``layers.short_conv``. Returns (y, final_state or None)."""
    return ShortConvFunction.apply(x, weight, bias, h0, cu_seqlens, cu_seqlens_dev, activation, output_final_state)


def _rows16(t):
    """A gradient of states as the library reads it: contiguous, and 16-byte aligned, which a view of a larger gradient
    may not be."""
    if t is None:
        return None
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


class SelectiveScanFunction(torch.autograd.Function):
    """y, final_state = selective_scan(x, dt, A, B, C, skip, z, dt_bias, h0) with gradients for all nine."""

    @staticmethod
    def forward(ctx, x, dt, A, B, C, skip, z, dt_bias, h0, cu_seqlens, cu_seqlens_dev, dt_softplus, output_final_state,
                save=True):
        cu_seqlens, cu_seqlens_dev = _kept_both(cu_seqlens, cu_seqlens_dev, x.device)
        f = layers.selective_scan(x, dt, A, B, C, skip=skip, z=z, dt_bias=dt_bias, h0=h0, cu_seqlens=cu_seqlens,
                                  cu_seqlens_dev=cu_seqlens_dev, dt_softplus=dt_softplus,
                                  output_final_state=output_final_state, save=save)
        ctx.save_for_backward(x, dt, A, B, C, skip, z, dt_bias, cu_seqlens_dev, f["states"])
        ctx.cu_seqlens, ctx.dt_softplus, ctx.has_h0 = cu_seqlens, dt_softplus, h0 is not None
        ctx.set_materialize_grads(False)
        return f["y"], f["final_state"]

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal):
        x, dt, A, B, C, skip, z, dt_bias, cu_dev, states = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.contiguous()
        r = layers.selective_scan_bwd(x, dt, A, B, C, states, dy, skip=skip, z=z, dt_bias=dt_bias,
                                      dfinal=_rows16(dfinal), cu_seqlens=ctx.cu_seqlens,
                                      cu_seqlens_dev=cu_dev, dt_softplus=ctx.dt_softplus, output_dh0=ctx.has_h0)
        return (r["dx"], r["ddt"], r["dA"], r["dB"], r["dC"], r["dskip"], r["dz"], r["ddt_bias"], r["dh0"], None, None,
                None, None, None)


def selective_scan(x, dt, A, B, C, skip=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, cu_seqlens_dev=None,
                   dt_softplus=False, output_final_state=True):
    """Differentiable ``layers.selective_scan``. Returns (y, final_state or None). The states of the chunks are
    kept (and written) where a backward can follow."""
    save = torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                           for t in (x, dt, A, B, C, skip, z, dt_bias, h0))
    return SelectiveScanFunction.apply(x, dt, A, B, C, skip, z, dt_bias, h0, cu_seqlens, cu_seqlens_dev, dt_softplus,
                                       output_final_state, save)


class GroupNormFunction(torch.autograd.Function):
    """y = group_norm(x, weight, bias, gate) with gradients for all four. The statistics are formed again
    in the backward, which reads x in any case."""

    @staticmethod
    def forward(ctx, x, weight, bias, gate, groups, activation, center, eps):
        ctx.save_for_backward(x, weight, bias, gate)
        ctx.args = dict(activation=activation, center=center, eps=float(eps))
        ctx.groups = groups
        return layers.group_norm(x, groups, weight=weight, bias=bias, gate=gate, **ctx.args)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, gate = ctx.saved_tensors
        r = layers.group_norm_bwd(x, ctx.groups, dy.contiguous(), weight=weight, bias=bias, gate=gate, **ctx.args)
        return r["dx"], r["dweight"], r["dbias"], r["dgate"], None, None, None, None


def group_norm(x, groups, weight=None, bias=None, gate=None, activation=None, center=False, eps=1e-5):
    """Differentiable ``layers.group_norm``."""
    return GroupNormFunction.apply(x, weight, bias, gate, groups, activation, center, eps)
