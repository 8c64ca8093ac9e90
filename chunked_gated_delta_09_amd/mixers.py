"""Token mixers with a state of bounded size per sequence, beside KDA's recurrence: linear attention with a decay for each
head, and softmax attention with a sliding window and a few first tokens that stay visible. Forward and backward over
whole sequences, and single tokens (``*_step``) on a state that is updated in place.

Argument marshalling over the C ABI in ``include/kda_mixers.h``; every step of the computation is a HIP kernel of the
library. What ``layers`` says of tensors, packed sequences, token steps and slots holds here: ``q``, ``k`` and ``v`` may be
column slices of a wider contiguous tensor, other tensors are contiguous. Nothing here is recorded by autograd
(``autograd`` has the differentiable forms).
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import KdaError, load
from .layers import (_DT, _bytes, _cuts, _fit, _gpu, _i32, _i64, _f32, _I32_MAX, _launch, _like, _need, _new, _new_if, _pi32,
                     _plan, _plan_of, _rows, _vp, _written, _ws)

__all__ = ["linear_attention", "linear_attention_bwd", "linear_attention_step", "window_attention", "window_attention_bwd",
           "window_attention_step"]

F32 = torch.float32


class _Dims(ctypes.Structure):
    @staticmethod
    def library():
        return _lib()


class _LinDims(_Dims):
    _fields_ = [("B", _i32), ("T", _i32), ("H", _i32), ("HV", _i32), ("K", _i32), ("V", _i32), ("N", _i32),
                ("cu_seqlens_dev", _vp), ("cu_seqlens_host", _pi32), ("q_row", _i64), ("k_row", _i64), ("v_row", _i64),
                ("g_const", _i32), ("scale", _f32), ("dtype", _i32)]


class _WinDims(_Dims):
    _fields_ = [("B", _i32), ("T", _i32), ("H", _i32), ("HK", _i32), ("D", _i32), ("N", _i32), ("cu_seqlens_dev", _vp),
                ("cu_seqlens_host", _pi32), ("q_row", _i64), ("k_row", _i64), ("v_row", _i64), ("window", _i32),
                ("sinks", _i32), ("scale", _f32), ("dtype", _i32)]


_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = load()
        sz, st = ctypes.c_size_t, ctypes.c_int
        for name, res, args in [
            ("kda_lattn_num_states", _i64, [_vp]),
            ("kda_lattn_fwd_workspace_bytes", sz, [_vp]),
            ("kda_lattn_bwd_workspace_bytes", sz, [_vp]),
            ("kda_lattn_fwd", st, [_vp] * 10 + [sz, _vp]),
            ("kda_lattn_bwd", st, [_vp] * 14 + [sz, _vp]),
            ("kda_lattn_step", st, [_vp] * 6 + [_i32] + [_vp] * 3),
            ("kda_wattn_bwd_workspace_bytes", sz, [_vp]),
            ("kda_wattn_step_workspace_bytes", sz, [_vp]),
            ("kda_wattn_fwd", st, [_vp] * 9),
            ("kda_wattn_bwd", st, [_vp] * 11 + [sz, _vp]),
            ("kda_wattn_step", st, [_vp] * 6 + [_i32] + [_vp] * 4 + [sz, _vp]),
        ]:
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _ready = lib
    return _ready


def _refused():
    return KdaError(-1, load().kda_last_error().decode())


# ---- linear attention


def _lin(q, k, v, g, scale, lead, cuts):
    dev = _gpu(q, "q")
    if q.dim() != lead + 2 or v.dim() != lead + 2:
        raise ValueError("q must be %s and v %s" % (("[B, T, H, K]", "[B, T, HV, V]") if lead == 2 else
                                                    ("[B, H, K]", "[B, HV, V]")))
    dt, shape, (H, K), (HV, V) = q.dtype, tuple(q.shape[:lead]), q.shape[lead:], v.shape[lead:]
    N, cu_dev, cu_host, keep = _cuts(*cuts, shape[0], dev)
    pq, rq = _rows(q, "q", dt, q.shape, dev, lead)
    pk, rk = _rows(k, "k", dt, q.shape, dev, lead)
    pv, rv = _rows(v, "v", dt, shape + (HV, V), dev, lead)
    const = g.dim() == 1
    pg = _need(g, "g", F32, (HV,) if const else shape + (HV,), dev)
    scale = 1.0 / math.sqrt(K) if scale is None else float(scale)
    plan = _plan_of(_LinDims, cu_dev, cu_host, (shape[0], shape[1] if lead == 2 else 1, H, HV, K, V, N),
                    (rq, rk, rv, int(const), scale, _DT[dt]))
    return plan, dev, (N, HV, K, V), (rq, rk, rv), (pq, pk, pv, pg), keep


def linear_attention(q, k, v, g, h0=None, cu_seqlens=None, cu_seqlens_dev=None, scale=None, output_final_state=True,
                     save=False):
    """S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t. q, k [B,T,H,K]; v [B,T,HV,V] (value head h has q/k head
    h // (HV // H); K and V up to 256); g [B,T,HV] fp32, the natural logarithm of the decays, or [HV], one for all tokens;
    h0 [N,HV,K,V] fp32; scale: 1/sqrt(K) by default. Returns dict(o [B,T,HV,V], final_state [N,HV,K,V] fp32 or None,
    states or None). ``save``: keep the states (fp32) that ``linear_attention_bwd`` starts from."""
    plan, dev, (N, HV, K, V), (_, _, rv), ptrs, keep = _lin(q, k, v, g, scale, 2, (cu_seqlens, cu_seqlens_dev))
    ph0 = _need(h0, "h0", F32, (N, HV, K, V), dev)
    count = plan.size("kda_lattn_num_states") if save else 0
    if count < 0:
        raise _refused()
    need = plan.size("kda_lattn_fwd_workspace_bytes")
    o, po = _like(v, rv)
    final, pf = _new_if(output_final_state, q, (N, HV, K, V), F32)
    states, ps = _new_if(save, q, (count, HV, K, V), F32)
    ws, pws = _ws(q, need)
    _launch(dev, _lib().kda_lattn_fwd, plan.ref, *ptrs, ph0, po, pf, ps, pws, need)
    del keep
    return dict(o=o, final_state=final, states=states)


def linear_attention_bwd(q, k, v, g, states, do, dfinal=None, cu_seqlens=None, cu_seqlens_dev=None, scale=None,
                         output_dh0=False):
    """Gradients of sum<do, o> + <dfinal, final_state>, from the ``states`` of ``linear_attention(..., save=True)`` on the
    same arguments. Returns dict(dq, dk [B,T,H,K], dv [B,T,HV,V], dg as g, dh0 [N,HV,K,V] fp32 or None)."""
    plan, dev, (N, HV, K, V), (rq, rk, rv), ptrs, keep = _lin(q, k, v, g, scale, 2, (cu_seqlens, cu_seqlens_dev))
    count = plan.size("kda_lattn_num_states")
    if count < 0:
        raise _refused()
    ps = _need(states, "states", F32, (count, HV, K, V), dev)
    pdo = _need(do, "do", q.dtype, v.shape, dev)
    pdf = _need(dfinal, "dfinal", F32, (N, HV, K, V), dev)
    need = _bytes(plan.size("kda_lattn_bwd_workspace_bytes"))
    (dq, pdq), (dk, pdk), (dv, pdv), (dg, pdg) = _like(q, rq), _like(k, rk), _like(v, rv), _like(g)
    dh0, pdh0 = _new_if(output_dh0, q, (N, HV, K, V), F32)
    ws, pws = _ws(q, need)
    _launch(dev, _lib().kda_lattn_bwd, plan.ref, *ptrs, ps, pdo, pdf, pdq, pdk, pdv, pdg, pdh0, pws, need)
    del keep
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dh0=dh0)


def linear_attention_step(q, k, v, g, state, slots=None, scale=None):
    """One token of each sequence: q, k [B,H,K], v [B,HV,V], g [B,HV] or [HV] fp32, state [S,HV,K,V] fp32 updated in place
    (``linear_attention``'s final_state is one). Returns o [B,HV,V]."""
    plan, dev, (B, HV, K, V), (_, _, rv), ptrs, _ = _lin(q, k, v, g, scale, 1, (None, None))
    if state.dim() != 4:
        raise ValueError("state must be [S, HV, K, V]")
    S = state.shape[0]
    pst = _need(state, "state", F32, (S, HV, K, V), dev)
    psl = _need(slots, "slots", torch.int32, (B,), dev)
    o, po = _like(v, rv)
    _launch(dev, _lib().kda_lattn_step, plan.ref, *ptrs, psl, S if S <= _I32_MAX else _fit("S", S), pst, po)
    _written((state,))
    return o


# ---- window attention


def _win(q, k, v, window, sinks, scale, lead, cuts):
    dev = _gpu(q, "q")
    if q.dim() != lead + 2 or k.dim() != lead + 2:
        raise ValueError("q must be %s and k %s" % (("[B, T, H, D]", "[B, T, HK, D]") if lead == 2 else
                                                    ("[B, H, D]", "[B, HK, D]")))
    dt, shape, (H, D), HK = q.dtype, tuple(q.shape[:lead]), q.shape[lead:], k.shape[lead]
    N, cu_dev, cu_host, keep = _cuts(*cuts, shape[0], dev)
    pq, rq = _rows(q, "q", dt, q.shape, dev, lead)
    pk, rk = _rows(k, "k", dt, shape + (HK, D), dev, lead)
    pv, rv = _rows(v, "v", dt, shape + (HK, D), dev, lead)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    window, sinks = _fit("window", int(window)), _fit("sinks", int(sinks))
    plan = _plan_of(_WinDims, cu_dev, cu_host, (shape[0], shape[1] if lead == 2 else 1, H, HK, D, N),
                    (rq, rk, rv, window, sinks, scale, _DT[dt]))
    return plan, dev, (N, H, HK, D), (rq, rk, rv), (pq, pk, pv), keep


def window_attention(q, k, v, window, sinks=0, cu_seqlens=None, cu_seqlens_dev=None, scale=None, save=False,
                     output_cache=False):
    """Softmax attention where token i of a sequence sees the tokens j <= i with i - j < window, and the first ``sinks``
    tokens: q [B,T,H,D] (D up to 256); k, v [B,T,HK,D], query head h with key head h // (H // HK); scale: 1/sqrt(D) by
    default. Returns dict(o [B,T,H,D], lse or None, k_cache, v_cache or None). ``save``: keep lse [B,T,H] fp32 for
    ``window_attention_bwd``. ``output_cache``: the caches [N,sinks+window,HK,D] with which ``window_attention_step``
    goes on behind each sequence's last token."""
    plan, dev, (N, H, HK, D), (rq, _, _), ptrs, keep = _win(q, k, v, window, sinks, scale, 2, (cu_seqlens, cu_seqlens_dev))
    o, po = _like(q, rq)
    lse, pl = _new_if(save, q, q.shape[:3], F32)
    rows = max(0, int(window) + int(sinks))  # the library refuses the sizes for which this is not the cache's
    (kc, pkc), (vc, pvc) = (_new_if(output_cache, q, (N, rows, HK, D)) for _ in range(2))
    _launch(dev, _lib().kda_wattn_fwd, plan.ref, *ptrs, po, pl, pkc, pvc)
    del keep
    return dict(o=o, lse=lse, k_cache=kc, v_cache=vc)


def window_attention_bwd(q, k, v, o, lse, do, window, sinks=0, cu_seqlens=None, cu_seqlens_dev=None, scale=None):
    """Gradients of sum<do, o>, from the o and lse of ``window_attention(..., save=True)`` on the same arguments. Returns
    dict(dq [B,T,H,D], dk, dv [B,T,HK,D])."""
    plan, dev, (N, H, HK, D), (rq, rk, rv), ptrs, keep = _win(q, k, v, window, sinks, scale, 2,
                                                             (cu_seqlens, cu_seqlens_dev))
    po = _need(o, "o", q.dtype, q.shape, dev)
    pl = _need(lse, "lse", F32, q.shape[:3], dev)
    pdo = _need(do, "do", q.dtype, q.shape, dev)
    need = plan.size("kda_wattn_bwd_workspace_bytes")
    (dq, pdq), (dk, pdk), (dv, pdv) = _like(q, rq), _like(k, rk), _like(v, rv)
    ws, pws = _ws(q, need)
    _launch(dev, _lib().kda_wattn_bwd, plan.ref, *ptrs, po, pl, pdo, pdq, pdk, pdv, pws, need)
    del keep
    return dict(dq=dq, dk=dk, dv=dv)


def window_attention_step(q, k, v, k_cache, v_cache, pos, sinks=0, slots=None, scale=None):
    """One token of each sequence: q [B,H,D], k, v [B,HK,D]; k_cache, v_cache [S,sinks+window,HK,D], updated in place (token
    p of a sequence is in row p where p < sinks, else in row sinks + (p - sinks) % window); pos int32 [B] on the GPU:
    the tokens that each sequence has had before. Returns o [B,H,D]; the row of a negative pos is NaN."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [S, sinks + window, HK, D]")
    S, rows = k_cache.shape[:2]
    plan, dev, (B, H, HK, D), (rq, _, _), ptrs, _ = _win(q, k, v, rows - int(sinks), sinks, scale, 1, (None, None))
    pkc = _need(k_cache, "k_cache", q.dtype, (S, rows, HK, D), dev)
    pvc = _need(v_cache, "v_cache", q.dtype, (S, rows, HK, D), dev)
    ppos = _need(pos, "pos", torch.int32, (B,), dev)
    psl = _need(slots, "slots", torch.int32, (B,), dev)
    need = plan.sizes.get("step")
    if need is None:
        need = _lib().kda_wattn_step_workspace_bytes(plan.ref)
        if need == ctypes.c_size_t(-1).value:
            raise _refused()
        plan.sizes["step"] = need
    o, po = _like(q, rq)
    ws, pws = _ws(q, need)
    _launch(dev, _lib().kda_wattn_step, plan.ref, *ptrs, ppos, psl, S if S <= _I32_MAX else _fit("S", S), pkc, pvc, po, pws,
            need)
    _written((k_cache, v_cache))
    return o
