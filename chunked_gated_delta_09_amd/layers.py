"""Operators around the KDA chunk recurrence in a layer: short causal convolution, selective state
space scan, norm per group of channels with an activation, and the single-token forms a served
model runs (``*_step``, with KDA's own as ``kda_step``).

Argument marshalling over the C ABI in ``include/kda_layers.h``; every step of the computation is a
HIP kernel of the library. Tensors are on one GPU, whose current stream the call is enqueued on.
They are contiguous, except that ``x``, ``dt``, ``z``, ``B``, ``C`` and ``gate`` may be column slices
of a wider contiguous tensor (``proj[..., a:b]``).

Packed sequences: ``cu_seqlens`` is the host list of cuts, with batch size 1; a caller that has a
device copy (int32) passes it as ``cu_seqlens_dev``, otherwise the call makes one (which copies
from the host, so it cannot be captured into a graph).

Token steps update the state in place. ``slots`` (int32 [B] on the GPU) names the state row of each
batch row; None: row b. A negative slot marks a padding row (no state is touched, its output is
zero); a slot behind the state's last row, or one that an earlier batch row has as well, is refused
on the GPU: no state is touched for that row and its output is NaN.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import KdaError, _check, load, make_dims

__all__ = ["short_conv", "short_conv_bwd", "short_conv_step", "selective_scan", "selective_scan_bwd",
           "selective_scan_step", "group_norm", "group_norm_bwd", "kda_step", "SCAN_CHUNK"]

SCAN_CHUNK = 16
_ACT = {None: 0, "silu": 1, "sigmoid": 2}
_DT = {torch.float32: 0, torch.bfloat16: 1}

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
_pi32 = ctypes.POINTER(_i32)


class _ConvDims(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("D", _i32), ("W", _i32), ("N", _i32), ("cu_seqlens_dev", _vp),
                ("cu_seqlens_host", _pi32), ("x_row", _i64), ("act", _i32), ("dtype", _i32)]


class _ScanDims(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("D", _i32), ("NS", _i32), ("G", _i32), ("N", _i32), ("cu_seqlens_dev", _vp),
                ("cu_seqlens_host", _pi32), ("x_row", _i64), ("dt_row", _i64), ("z_row", _i64), ("b_row", _i64),
                ("c_row", _i64), ("softplus", _i32), ("dtype", _i32)]


class _NormDims(ctypes.Structure):
    _fields_ = [("R", _i64), ("G", _i32), ("C", _i32), ("center", _i32), ("act", _i32), ("shared", _i32), ("eps", _f32),
                ("x_row", _i64), ("gate_row", _i64), ("dtype", _i32)]


_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = load()
        sz, st = ctypes.c_size_t, ctypes.c_int
        for name, res, args in [
            ("kda_short_conv_fwd", st, [_vp] * 8),
            ("kda_short_conv_bwd_workspace_bytes", sz, [_vp]),
            ("kda_short_conv_bwd", st, [_vp] * 12 + [sz, _vp]),
            ("kda_short_conv_step", st, [_vp] * 5 + [_i32] + [_vp] * 3),
            ("kda_sscan_num_chunks", _i64, [_vp]),
            ("kda_sscan_fwd_workspace_bytes", sz, [_vp]),
            ("kda_sscan_bwd_workspace_bytes", sz, [_vp]),
            ("kda_sscan_fwd", st, [_vp] * 14 + [sz, _vp]),
            ("kda_sscan_bwd", st, [_vp] * 22 + [sz, _vp]),
            ("kda_sscan_step", st, [_vp] * 10 + [_i32] + [_vp] * 3),
            ("kda_group_norm_fwd", st, [_vp] * 7),
            ("kda_group_norm_bwd_workspace_bytes", sz, [_vp]),
            ("kda_group_norm_bwd", st, [_vp] * 11 + [sz, _vp]),
            ("kda_step", st, [_vp] * 7 + [_i32] + [_vp] * 3),
        ]:
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _ready = lib
    return _ready


def _on(dev):
    """The library launches on the current device: make it the tensors' for the call."""
    if dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


def _p(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, shape, dev):
    """A contiguous tensor of this type and shape on `dev` (None passes)."""
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name, dtype, shape, dev, lead):
    """As _need for a tensor that may be a column slice: the first `lead` dimensions are its rows.
    Returns the elements between two rows."""
    if t is None:
        return 0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return 0
    width, row = 1, None
    for i in range(t.dim() - 1, lead - 1, -1):
        if t.shape[i] != 1 and t.stride(i) != width:
            raise ValueError(f"{name} must be contiguous or a column slice of a contiguous tensor")
        width *= t.shape[i]
    count = 1  # rows of the dimensions behind the current one
    for i in range(lead - 1, -1, -1):
        if t.shape[i] != 1:
            if row is None:
                if t.stride(i) % count or t.stride(i) // count < width:
                    raise ValueError(f"{name} must be contiguous or a column slice of a contiguous tensor")
                row = t.stride(i) // count
            elif t.stride(i) != row * count:
                raise ValueError(f"{name} must be contiguous or a column slice of a contiguous tensor")
        count *= t.shape[i]
    return row or 0


def _gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype not in _DT:
        raise ValueError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    return t.device


def _act(activation, allowed):
    if activation not in allowed:
        raise ValueError(f"activation must be one of {allowed}, got {activation!r}")
    return _ACT[activation]


def _cuts(cu_seqlens, cu_seqlens_dev, B, dev):
    """(sequences, device cuts or None, host array or None)."""
    if cu_seqlens is None:
        if cu_seqlens_dev is not None:
            raise ValueError("cu_seqlens_dev needs the host list cu_seqlens beside it")
        return B, None, None
    if B != 1:
        raise ValueError("packed sequences need batch size 1")
    cu = [int(c) for c in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
    if len(cu) < 2:
        raise ValueError("cu_seqlens needs at least two entries")
    if cu_seqlens_dev is None:
        cu_seqlens_dev = torch.tensor(cu, dtype=torch.int32, device=dev)
    _need(cu_seqlens_dev, "cu_seqlens_dev", torch.int32, (len(cu),), dev)
    return len(cu) - 1, cu_seqlens_dev, (_i32 * len(cu))(*cu)


def _bytes(n):
    if n == 0:
        raise KdaError(-1, load().kda_last_error().decode())
    return n


def _ws(n, dev):
    return torch.empty(n, dtype=torch.uint8, device=dev) if n else None


def _slots(slots, B, dev):
    _need(slots, "slots", torch.int32, (B,), dev)


# ---- short convolution


def _conv(x, weight, bias, h0, cu_seqlens, cu_seqlens_dev, activation):
    dev = _gpu(x, "x")
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [B, T, D] and weight [D, W]")
    B, T, D = x.shape
    W = weight.shape[1]
    N, cu_dev, cu_host = _cuts(cu_seqlens, cu_seqlens_dev, B, dev)
    row = _rows(x, "x", x.dtype, (B, T, D), dev, 2)
    _need(weight, "weight", torch.float32, (D, W), dev)
    _need(bias, "bias", torch.float32, (D,), dev)
    _need(h0, "h0", x.dtype, (N, W - 1, D), dev)
    d = _ConvDims(B, T, D, W, N, _p(cu_dev), cu_host, row, _act(activation, (None, "silu")), _DT[x.dtype])
    return d, dev, (B, T, D, W, N), (cu_dev, cu_host)


def short_conv(x, weight, bias=None, h0=None, cu_seqlens=None, cu_seqlens_dev=None, activation="silu",
               output_final_state=False):
    """Causal convolution over the tokens, one filter per channel: u_t = bias + sum_j weight[:, j]
    x_{t-(W-1)+j}, y = u or silu(u). x [B,T,D]; weight [D,W] fp32 (W = 2, 3, 4; the last tap sees the
    current token); bias [D] fp32; h0 [N,W-1,D]: the rows before each sequence's first. Returns
    dict(y [B,T,D], final_state [N,W-1,D] or None: the last W-1 rows of [h0 | x])."""
    d, dev, (B, T, D, W, N), keep = _conv(x, weight, bias, h0, cu_seqlens, cu_seqlens_dev, activation)
    with _on(dev):
        y = torch.empty(B, T, D, dtype=x.dtype, device=dev)
        final = torch.empty(N, W - 1, D, dtype=x.dtype, device=dev) if output_final_state else None
        _check(_lib().kda_short_conv_fwd(ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(h0), _p(y), _p(final),
                                         _stream(dev)))
    del keep
    return dict(y=y, final_state=final)


def short_conv_bwd(x, weight, dy, bias=None, h0=None, dfinal=None, cu_seqlens=None, cu_seqlens_dev=None,
                   activation="silu"):
    """Gradients of sum<dy, y> + <dfinal, final_state>. Returns dict(dx [B,T,D], dweight [D,W] fp32,
    dbias [D] fp32 or None, dh0 [N,W-1,D] or None)."""
    d, dev, (B, T, D, W, N), keep = _conv(x, weight, bias, h0, cu_seqlens, cu_seqlens_dev, activation)
    _need(dy, "dy", x.dtype, (B, T, D), dev)
    _need(dfinal, "dfinal", x.dtype, (N, W - 1, D), dev)
    lib = _lib()
    need = lib.kda_short_conv_bwd_workspace_bytes(ctypes.byref(d))
    with _on(dev):
        dx = torch.empty(B, T, D, dtype=x.dtype, device=dev)
        dw = torch.empty_like(weight)
        db = torch.empty_like(bias) if bias is not None else None
        dh0 = torch.empty_like(h0) if h0 is not None else None
        ws = _ws(need, dev)
        _check(lib.kda_short_conv_bwd(ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(h0), _p(dy), _p(dfinal), _p(dx),
                                      _p(dw), _p(db), _p(dh0), _p(ws), need, _stream(dev)))
    del keep
    return dict(dx=dx, dweight=dw, dbias=db, dh0=dh0)


def short_conv_step(x, state, weight, bias=None, slots=None, activation="silu"):
    """One token of each sequence: x [B,D], state [S,W-1,D] of x's type, updated in place. Returns y
    [B,D]."""
    dev = _gpu(x, "x")
    if x.dim() != 2 or weight.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be [B, D], weight [D, W] and state [S, W-1, D]")
    B, D = x.shape
    W = weight.shape[1]
    row = _rows(x, "x", x.dtype, (B, D), dev, 1)
    _need(weight, "weight", torch.float32, (D, W), dev)
    _need(bias, "bias", torch.float32, (D,), dev)
    _need(state, "state", x.dtype, (state.shape[0], W - 1, D), dev)
    _slots(slots, B, dev)
    d = _ConvDims(B, 1, D, W, B, None, None, row, _act(activation, (None, "silu")), _DT[x.dtype])
    with _on(dev):
        y = torch.empty(B, D, dtype=x.dtype, device=dev)
        _check(_lib().kda_short_conv_step(ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(slots), state.shape[0],
                                          _p(state), _p(y), _stream(dev)))
    return y


# ---- selective scan


def _scan(x, dt, A, B, C, skip, z, dt_bias, softplus, lead, cuts):
    dev = _gpu(x, "x")
    if x.dim() != lead + 1 or A.dim() != 2 or B.dim() != lead + 2:
        raise ValueError("x must be %s, A [D, NS] and B, C %s" % (("[B, T, D]", "[B, T, G, NS]") if lead == 2 else
                                                                   ("[B, D]", "[B, G, NS]")))
    rows, D, NS, G = tuple(x.shape[:-1]), x.shape[-1], A.shape[1], B.shape[-2]
    N, cu_dev, cu_host = _cuts(*cuts, rows[0], dev)
    dt_ = x.dtype
    strides = [_rows(x, "x", dt_, rows + (D,), dev, lead), _rows(dt, "dt", dt_, rows + (D,), dev, lead),
               _rows(z, "z", dt_, rows + (D,), dev, lead), _rows(B, "B", dt_, rows + (G, NS), dev, lead),
               _rows(C, "C", dt_, rows + (G, NS), dev, lead)]
    _need(A, "A", torch.float32, (D, NS), dev)
    _need(skip, "skip", torch.float32, (D,), dev)
    _need(dt_bias, "dt_bias", torch.float32, (D,), dev)
    d = _ScanDims(rows[0], rows[1] if lead == 2 else 1, D, NS, G, N, _p(cu_dev), cu_host, *strides, int(bool(softplus)),
                  _DT[dt_])
    return d, dev, (rows, D, NS, G, N), (cu_dev, cu_host)


def selective_scan(x, dt, A, B, C, skip=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, cu_seqlens_dev=None,
                   dt_softplus=False, output_final_state=True, save=False):
    """h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t, y_t = <C_t, h_t> + skip x_t, times silu(z_t) with z; dt_t is
    dt + dt_bias, or its softplus with ``dt_softplus``. x, dt, z [B,T,D]; A [D,NS] fp32 (NS <= 64); B, C
    [B,T,G,NS], shared by the D/G channels of a group; skip, dt_bias [D] fp32; h0 [N,D,NS] fp32.
    Returns dict(y [B,T,D], final_state [N,D,NS] fp32 or None, states or None). ``save``: keep the state
    entering every SCAN_CHUNK tokens (fp32 [chunks,D,NS]) for ``selective_scan_bwd``."""
    d, dev, (rows, D, NS, G, N), keep = _scan(x, dt, A, B, C, skip, z, dt_bias, dt_softplus, 2,
                                              (cu_seqlens, cu_seqlens_dev))
    _need(h0, "h0", torch.float32, (N, D, NS), dev)
    lib = _lib()
    chunks = lib.kda_sscan_num_chunks(ctypes.byref(d))
    if chunks < 0:
        raise KdaError(-1, lib.kda_last_error().decode())
    need = lib.kda_sscan_fwd_workspace_bytes(ctypes.byref(d))
    with _on(dev):
        y = torch.empty(*rows, D, dtype=x.dtype, device=dev)
        final = torch.empty(N, D, NS, dtype=torch.float32, device=dev) if output_final_state else None
        states = torch.empty(chunks, D, NS, dtype=torch.float32, device=dev) if save else None
        ws = _ws(need, dev)
        _check(lib.kda_sscan_fwd(ctypes.byref(d), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(skip), _p(z), _p(dt_bias),
                                 _p(h0), _p(y), _p(final), _p(states), _p(ws), need, _stream(dev)))
    del keep
    return dict(y=y, final_state=final, states=states)


def selective_scan_bwd(x, dt, A, B, C, states, dy, skip=None, z=None, dt_bias=None, dfinal=None, cu_seqlens=None,
                       cu_seqlens_dev=None, dt_softplus=False, output_dh0=False):
    """Gradients of sum<dy, y> + <dfinal, final_state>, from the ``states`` of
    ``selective_scan(..., save=True)`` on the same arguments. Returns dict(dx, ddt [B,T,D], dA [D,NS]
    fp32, dB, dC [B,T,G,NS], dskip [D] fp32 or None, dz [B,T,D] or None, ddt_bias [D] fp32 or None, dh0
    [N,D,NS] fp32 or None)."""
    d, dev, (rows, D, NS, G, N), keep = _scan(x, dt, A, B, C, skip, z, dt_bias, dt_softplus, 2,
                                              (cu_seqlens, cu_seqlens_dev))
    lib = _lib()
    chunks = lib.kda_sscan_num_chunks(ctypes.byref(d))
    if chunks < 0:
        raise KdaError(-1, lib.kda_last_error().decode())
    _need(states, "states", torch.float32, (chunks, D, NS), dev)
    _need(dy, "dy", x.dtype, rows + (D,), dev)
    _need(dfinal, "dfinal", torch.float32, (N, D, NS), dev)
    need = _bytes(lib.kda_sscan_bwd_workspace_bytes(ctypes.byref(d)))
    f32 = dict(dtype=torch.float32, device=dev)
    own = dict(dtype=x.dtype, device=dev)
    with _on(dev):
        dx, ddt = torch.empty(*rows, D, **own), torch.empty(*rows, D, **own)
        dA = torch.empty(D, NS, **f32)
        dB, dC = torch.empty(*rows, G, NS, **own), torch.empty(*rows, G, NS, **own)
        dskip = torch.empty(D, **f32) if skip is not None else None
        dz = torch.empty(*rows, D, **own) if z is not None else None
        dbias = torch.empty(D, **f32) if dt_bias is not None else None
        dh0 = torch.empty(N, D, NS, **f32) if output_dh0 else None
        ws = _ws(need, dev)
        _check(lib.kda_sscan_bwd(ctypes.byref(d), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(skip), _p(z), _p(dt_bias),
                                 _p(states), _p(dy), _p(dfinal), _p(dx), _p(ddt), _p(dA), _p(dB), _p(dC), _p(dskip),
                                 _p(dz), _p(dbias), _p(dh0), _p(ws), need, _stream(dev)))
    del keep
    return dict(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dskip=dskip, dz=dz, ddt_bias=dbias, dh0=dh0)


def selective_scan_step(x, dt, A, B, C, state, slots=None, skip=None, z=None, dt_bias=None, dt_softplus=False):
    """One token of each sequence: x, dt, z [B,D], B, C [B,G,NS], state [S,D,NS] fp32 updated in place.
    Returns y [B,D]."""
    d, dev, (rows, D, NS, G, N), _ = _scan(x, dt, A, B, C, skip, z, dt_bias, dt_softplus, 1, (None, None))
    if state.dim() != 3:
        raise ValueError("state must be [S, D, NS]")
    _need(state, "state", torch.float32, (state.shape[0], D, NS), dev)
    _slots(slots, rows[0], dev)
    with _on(dev):
        y = torch.empty(rows[0], D, dtype=x.dtype, device=dev)
        _check(_lib().kda_sscan_step(ctypes.byref(d), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(skip), _p(z), _p(dt_bias),
                                     _p(slots), state.shape[0], _p(state), _p(y), _stream(dev)))
    return y


# ---- group norm


def _norm(x, groups, weight, bias, gate, activation, center, eps):
    dev = _gpu(x, "x")
    if x.dim() < 1 or groups < 1 or x.shape[-1] == 0 or x.shape[-1] % groups:
        raise ValueError(f"the last dimension of x must be a positive multiple of groups ({groups}), got {tuple(x.shape)}")
    lead = x.dim() - 1
    W = x.shape[-1]
    C = W // groups
    x_row = _rows(x, "x", x.dtype, x.shape, dev, lead)
    gate_row = _rows(gate, "gate", x.dtype, x.shape, dev, lead)
    first = weight if weight is not None else bias
    shared = first is not None and groups > 1 and first.dim() == 1 and first.shape[0] == C
    for t, name in ((weight, "weight"), (bias, "bias")):
        _need(t, name, torch.float32, (C if shared else W,), dev)
    d = _NormDims(x.numel() // W, groups, C, int(bool(center)), _act(activation, (None, "silu", "sigmoid")), int(shared),
                  float(eps), x_row, gate_row, _DT[x.dtype])
    return d, dev


def group_norm(x, groups, weight=None, bias=None, gate=None, activation=None, center=False, eps=1e-5):
    """Norm over each group of channels of every row of x [..., groups*C]: n = x / rms (or, with
    ``center``, (x - mean) / std), u = n weight + bias, y = act(u), or u act(gate) with a gate of x's
    shape. weight and bias fp32, [groups*C] or [C] (one for all groups). activation: None, "silu",
    "sigmoid". Returns y."""
    d, dev = _norm(x, groups, weight, bias, gate, activation, center, eps)
    with _on(dev):
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        _check(_lib().kda_group_norm_fwd(ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(gate), _p(y), _stream(dev)))
    return y


def group_norm_bwd(x, groups, dy, weight=None, bias=None, gate=None, activation=None, center=False, eps=1e-5):
    """Gradients of sum<dy, y>. Returns dict(dx, dweight, dbias, dgate), None where the input is."""
    d, dev = _norm(x, groups, weight, bias, gate, activation, center, eps)
    _need(dy, "dy", x.dtype, x.shape, dev)
    lib = _lib()
    need = lib.kda_group_norm_bwd_workspace_bytes(ctypes.byref(d)) if weight is not None or bias is not None else 0
    with _on(dev):
        dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
        dw = torch.empty_like(weight) if weight is not None else None
        db = torch.empty_like(bias) if bias is not None else None
        dgate = torch.empty(x.shape, dtype=x.dtype, device=dev) if gate is not None else None
        ws = _ws(need, dev)
        _check(lib.kda_group_norm_bwd(ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(gate), _p(dy), _p(dx), _p(dw),
                                      _p(db), _p(dgate), _p(ws), need, _stream(dev)))
    return dict(dx=dx, dweight=dw, dbias=db, dgate=dgate)


# ---- KDA


def kda_step(q, k, v, g, beta, state, slots=None, scale=None, beta_logits=False):
    """One token of KDA for each sequence: q, k [B,H,K], v [B,HV,V], g [B,HV,K] fp32, beta [B,HV] fp32 (or
    its logits), state [S,HV,K,V] fp32 updated in place (``fwd_states``' final_state is one). K and V up
    to 256. Returns o [B,HV,V]."""
    dev = _gpu(q, "q")
    if q.dim() != 3 or v.dim() != 3 or state.dim() != 4:
        raise ValueError("q must be [B, H, K], v [B, HV, V] and state [S, HV, K, V]")
    (B, H, K), (HV, V) = q.shape, v.shape[1:]
    _need(q, "q", q.dtype, (B, H, K), dev)
    _need(k, "k", q.dtype, (B, H, K), dev)
    _need(v, "v", q.dtype, (B, HV, V), dev)
    _need(g, "g", torch.float32, (B, HV, K), dev)
    _need(beta, "beta", torch.float32, (B, HV), dev)
    _need(state, "state", torch.float32, (state.shape[0], HV, K, V), dev)
    _slots(slots, B, dev)
    d, _ = make_dims(B, 1, H, HV, K, V, 16, scale, "f32" if q.dtype == torch.float32 else "bf16", beta_logits=beta_logits)
    with _on(dev):
        o = torch.empty(B, HV, V, dtype=q.dtype, device=dev)
        _check(_lib().kda_step(ctypes.byref(d), _p(q), _p(k), _p(v), _p(g), _p(beta), _p(slots), state.shape[0], _p(state),
                               _p(o), _stream(dev)))
    return o
