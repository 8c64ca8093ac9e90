"""Operators around the KDA chunk recurrence in a layer: short causal convolution, selective state
space scan, norm per group of channels with an activation, and the single-token forms a served
model runs (``*_step``, with KDA's own as ``kda_step``).

Argument marshalling over the C ABI in ``include/kda_layers.h``; every step of the computation is a
HIP kernel of the library. Tensors are on one GPU, whose current stream the call is enqueued on.
They are contiguous, except that ``x``, ``dt``, ``z``, ``B``, ``C`` and ``gate`` may be column slices
of a wider contiguous tensor (``proj[..., a:b]``). A scan's fp32 tensors [..., NS] with NS of 8, 16, 32 or 64 begin
on a multiple of 16 bytes, as tensors of their own do.

Packed sequences: ``cu_seqlens`` is the host list of cuts, with batch size 1; a caller that has a
device copy (int32) passes it as ``cu_seqlens_dev``, otherwise the call makes one (which copies
from the host, so it cannot be captured into a graph). Both hold the same cuts for as long as the call, or a
graph that has captured it, runs.

Token steps update the state in place. ``slots`` (int32 [B] on the GPU) names the state row of each
batch row; None: row b. A negative slot marks a padding row (no state is touched, its output is
zero); a slot behind the state's last row, or one that an earlier batch row has as well, is refused
on the GPU: no state is touched for that row and its output is NaN.

Nothing here is recorded by autograd (``autograd`` has the differentiable forms). A state that a graph has
saved for its backward is too new for it after a step, as after any in-place operation.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import KdaError, _check, load, make_dims

__all__ = ["short_conv", "short_conv_bwd", "short_conv_step", "selective_scan", "selective_scan_bwd",
           "selective_scan_step", "group_norm", "group_norm_bwd", "kda_step", "SCAN_CHUNK"]

SCAN_CHUNK = 16
_ACT = {None: 0, "silu": 1, "sigmoid": 2}
_DT = {torch.float32: 0, torch.bfloat16: 1}

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
_pi32 = ctypes.POINTER(_i32)
_I32_MAX = 2 ** 31 - 1


def _fit(name, v):
    """Refuses a size that ctypes would cut to its low 32 bits, and so to another call."""
    if not -_I32_MAX <= v <= _I32_MAX:
        raise ValueError(f"{name} ({v}) does not fit 32 bits")
    return v


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


def _launch(dev, fn, *args):
    """Calls fn(*args, stream) with GPU `dev` and its current stream. Kernels go to the current device."""
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        _check(status)


# Torch does not see a write through an address: a step counts its state's version up by hand, so that a graph which
# has saved the state refuses its backward.
_written = torch._C._increment_version


def _refuse(t, name, dtype, shape, dev):
    """Raises for what is wrong with `t`, layout apart."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on GPU {dev} like the others, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need(t, name, dtype, shape, dev):
    """The address of a contiguous tensor of this type and shape on GPU `dev` (None passes)."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dtype, shape, dev)
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name, dtype, shape, dev, lead):
    """As _need for a tensor that may be a column slice: the first `lead` dimensions are its rows.
    Returns the address and the elements between two rows (0: contiguous)."""
    if t is None:
        return None, 0
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr(), 0
    _refuse(t, name, dtype, shape, dev)
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
    return t.data_ptr(), row or 0


def _gpu(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype not in _DT:
        raise ValueError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    return dev


def _act(activation, allowed):
    if activation not in allowed:
        raise ValueError(f"activation must be one of {allowed}, got {activation!r}")
    return _ACT[activation]


def _cuts(cu_seqlens, cu_seqlens_dev, B, dev):
    """(sequences, address of the device cuts or None, host array or None, what must live until the call)."""
    if cu_seqlens is None:
        if cu_seqlens_dev is not None:
            raise ValueError("cu_seqlens_dev needs the host list cu_seqlens beside it")
        return B, None, None, None
    if B != 1:
        raise ValueError("packed sequences need batch size 1")
    cu = list(map(int, cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens))
    if len(cu) < 2:
        raise ValueError("cu_seqlens needs at least two entries")
    if max(cu) > _I32_MAX or min(cu) < -_I32_MAX:
        raise ValueError("cu_seqlens holds a cut that does not fit 32 bits")
    if cu_seqlens_dev is None:
        cu_seqlens_dev = torch.tensor(cu, dtype=torch.int32, device=f"cuda:{dev}")
    ptr = _need(cu_seqlens_dev, "cu_seqlens_dev", torch.int32, (len(cu),), dev)
    return len(cu) - 1, ptr, (_i32 * len(cu))(*cu), cu_seqlens_dev


class _Plan:
    """A size structure, the reference that calls take, and the sizes that the library has answered for it."""

    __slots__ = ("dims", "ref", "sizes")

    def __init__(self, kind, *values):
        self.dims = kind(*values)
        self.ref = ctypes.byref(self.dims)
        self.sizes = {}

    def size(self, query):
        n = self.sizes.get(query)
        if n is None:
            n = getattr(_lib(), query)(self.ref)
            if n > 0:
                self.sizes[query] = n
        return n


# Those of calls without cuts are kept, by their values alone: the library only reads them.
@functools.lru_cache(maxsize=512)
def _plan(kind, *values):
    for (name, field), v in zip(kind._fields_, values):
        if field is _i32:
            _fit(name, v)
    return _Plan(kind, *values)


def _plan_of(kind, cu_dev, cu_host, before, after):
    if cu_host is None:
        return _plan(kind, *before, None, None, *after)
    if max(before) > _I32_MAX:
        raise ValueError(f"{max(before)} does not fit 32 bits, among {[n for n, _ in kind._fields_[:len(before)]]}")
    return _Plan(kind, *before, cu_dev, cu_host, *after)


@functools.lru_cache(maxsize=512)
def _kda_dims(B, H, HV, K, V, scale, dtype, beta_logits):
    for name, v in (("B", B), ("H", H), ("HV", HV), ("K", K), ("V", V)):
        _fit(name, v)
    d, _ = make_dims(B, 1, H, HV, K, V, 16, scale, dtype, beta_logits=beta_logits)
    return d, ctypes.byref(d)


def _bytes(n):
    if n == 0:
        raise KdaError(-1, load().kda_last_error().decode())
    return n


def _ws(like, n):
    """A workspace of n bytes and its address."""
    if not n:
        return None, None
    ws = like.new_empty(n, dtype=torch.uint8)
    return ws, ws.data_ptr()


def _new(like, shape, dtype=None):
    """A tensor of this shape, of the type (but for `dtype`) and on the GPU of `like`, and its address."""
    t = like.new_empty(shape, dtype=dtype)
    return t, t.data_ptr()


def _new_if(cond, like, shape, dtype=None):
    return _new(like, shape, dtype) if cond else (None, None)


def _like(t, row=0):
    """A contiguous tensor of the shape, type and GPU of `t`, and its address. `row`: what _rows found for `t`
    (0: `t` is contiguous itself, and empty_like, the cheapest call, lays the new one out the same)."""
    if t is None:
        return None, None
    r = t.new_empty(t.shape) if row else torch.empty_like(t)
    return r, r.data_ptr()


F32 = torch.float32


# ---- short convolution


def _conv(x, weight, bias, h0, cu_seqlens, cu_seqlens_dev, activation):
    dev = _gpu(x, "x")
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [B, T, D] and weight [D, W]")
    B, T, D = x.shape
    W = weight.shape[1]
    N, cu_dev, cu_host, keep = _cuts(cu_seqlens, cu_seqlens_dev, B, dev)
    px, row = _rows(x, "x", x.dtype, (B, T, D), dev, 2)
    ptrs = (px, _need(weight, "weight", F32, (D, W), dev), _need(bias, "bias", F32, (D,), dev),
            _need(h0, "h0", x.dtype, (N, W - 1, D), dev))
    plan = _plan_of(_ConvDims, cu_dev, cu_host, (B, T, D, W, N), (row, _act(activation, (None, "silu")), _DT[x.dtype]))
    return plan, dev, (B, T, D, W, N), row, ptrs, keep


def short_conv(x, weight, bias=None, h0=None, cu_seqlens=None, cu_seqlens_dev=None, activation="silu",
               output_final_state=False):
    """Causal convolution over the tokens, one filter per channel: u_t = bias + sum_j weight[:, j]
    x_{t-(W-1)+j}, y = u or silu(u). x [B,T,D]; weight [D,W] fp32 (W = 2, 3, 4; the last tap sees the
    current token); bias [D] fp32; h0 [N,W-1,D]: the rows before each sequence's first. Returns
    dict(y [B,T,D], final_state [N,W-1,D] or None: the last W-1 rows of [h0 | x])."""
    plan, dev, (B, T, D, W, N), row, ptrs, keep = _conv(x, weight, bias, h0, cu_seqlens, cu_seqlens_dev, activation)
    y, py = _like(x, row)
    final, pf = _new_if(output_final_state, x, (N, W - 1, D))
    _launch(dev, _lib().kda_short_conv_fwd, plan.ref, *ptrs, py, pf)
    del keep
    return dict(y=y, final_state=final)


def short_conv_bwd(x, weight, dy, bias=None, h0=None, dfinal=None, cu_seqlens=None, cu_seqlens_dev=None,
                   activation="silu"):
    """Gradients of sum<dy, y> + <dfinal, final_state>. Returns dict(dx [B,T,D], dweight [D,W] fp32,
    dbias [D] fp32 or None, dh0 [N,W-1,D] or None)."""
    plan, dev, (B, T, D, W, N), row, ptrs, keep = _conv(x, weight, bias, h0, cu_seqlens, cu_seqlens_dev, activation)
    pdy = _need(dy, "dy", x.dtype, (B, T, D), dev)
    pdf = _need(dfinal, "dfinal", x.dtype, (N, W - 1, D), dev)
    need = plan.size("kda_short_conv_bwd_workspace_bytes")
    (dx, pdx), (dw, pdw), (db, pdb), (dh0, pdh0) = _like(x, row), _like(weight), _like(bias), _like(h0)
    ws, pws = _ws(x, need)
    _launch(dev, _lib().kda_short_conv_bwd, plan.ref, *ptrs, pdy, pdf, pdx, pdw, pdb, pdh0, pws, need)
    del keep
    return dict(dx=dx, dweight=dw, dbias=db, dh0=dh0)


def short_conv_step(x, state, weight, bias=None, slots=None, activation="silu"):
    """One token of each sequence: x [B,D], state [S,W-1,D] of x's type, updated in place. Returns y
    [B,D]."""
    dev = _gpu(x, "x")
    if x.dim() != 2 or weight.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be [B, D], weight [D, W] and state [S, W-1, D]")
    (B, D), S, W = x.shape, state.shape[0], weight.shape[1]
    px, row = _rows(x, "x", x.dtype, (B, D), dev, 1)
    pw = _need(weight, "weight", F32, (D, W), dev)
    pb = _need(bias, "bias", F32, (D,), dev)
    pst = _need(state, "state", x.dtype, (S, W - 1, D), dev)
    psl = _need(slots, "slots", torch.int32, (B,), dev)
    plan = _plan(_ConvDims, B, 1, D, W, B, None, None, row, _act(activation, (None, "silu")), _DT[x.dtype])
    y, py = _like(x, row)
    _launch(dev, _lib().kda_short_conv_step, plan.ref, px, pw, pb, psl, S if S <= _I32_MAX else _fit("S", S), pst, py)
    _written((state,))
    return y


# ---- selective scan


def _scan(x, dt, A, B, C, skip, z, dt_bias, softplus, lead, cuts):
    dev = _gpu(x, "x")
    if x.dim() != lead + 1 or A.dim() != 2 or B.dim() != lead + 2:
        raise ValueError("x must be %s, A [D, NS] and B, C %s" % (("[B, T, D]", "[B, T, G, NS]") if lead == 2 else
                                                                   ("[B, D]", "[B, G, NS]")))
    shape, D, NS, G, dt_ = x.shape, x.shape[-1], A.shape[1], B.shape[-2], x.dtype
    rows = tuple(shape[:-1])
    bc = rows + (G, NS)
    N, cu_dev, cu_host, keep = _cuts(*cuts, rows[0], dev)
    px, rx = _rows(x, "x", dt_, shape, dev, lead)
    pdt, rdt = _rows(dt, "dt", dt_, shape, dev, lead)
    pz, rz = _rows(z, "z", dt_, shape, dev, lead)
    pB, rB = _rows(B, "B", dt_, bc, dev, lead)
    pC, rC = _rows(C, "C", dt_, bc, dev, lead)
    ptrs = (px, pdt, _need(A, "A", F32, (D, NS), dev), pB, pC, _need(skip, "skip", F32, (D,), dev), pz,
            _need(dt_bias, "dt_bias", F32, (D,), dev))
    strides = (rx, rdt, rz, rB, rC)
    plan = _plan_of(_ScanDims, cu_dev, cu_host, (rows[0], rows[1] if lead == 2 else 1, D, NS, G, N),
                    strides + (int(bool(softplus)), _DT[dt_]))
    return plan, dev, (rows, D, NS, N), strides, ptrs, keep


def selective_scan(x, dt, A, B, C, skip=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, cu_seqlens_dev=None,
                   dt_softplus=False, output_final_state=True, save=False):
    """h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t, y_t = <C_t, h_t> + skip x_t, times silu(z_t) with z; dt_t is
    dt + dt_bias, or its softplus with ``dt_softplus``. x, dt, z [B,T,D]; A [D,NS] fp32 (NS <= 64); B, C
    [B,T,G,NS], shared by the D/G channels of a group; skip, dt_bias [D] fp32; h0 [N,D,NS] fp32.
    Returns dict(y [B,T,D], final_state [N,D,NS] fp32 or None, states or None). ``save``: keep the state
    entering every SCAN_CHUNK tokens (fp32 [chunks,D,NS]) for ``selective_scan_bwd``."""
    plan, dev, (rows, D, NS, N), strides, ptrs, keep = _scan(x, dt, A, B, C, skip, z, dt_bias, dt_softplus, 2,
                                                             (cu_seqlens, cu_seqlens_dev))
    ph0 = _need(h0, "h0", F32, (N, D, NS), dev)
    chunks = plan.size("kda_sscan_num_chunks")
    if chunks < 0:
        raise KdaError(-1, _lib().kda_last_error().decode())
    need = plan.size("kda_sscan_fwd_workspace_bytes")
    y, py = _like(x, strides[0])
    final, pf = _new_if(output_final_state, x, (N, D, NS), F32)
    states, ps = _new_if(save, x, (chunks, D, NS), F32)
    ws, pws = _ws(x, need)
    _launch(dev, _lib().kda_sscan_fwd, plan.ref, *ptrs, ph0, py, pf, ps, pws, need)
    del keep
    return dict(y=y, final_state=final, states=states)


def selective_scan_bwd(x, dt, A, B, C, states, dy, skip=None, z=None, dt_bias=None, dfinal=None, cu_seqlens=None,
                       cu_seqlens_dev=None, dt_softplus=False, output_dh0=False):
    """Gradients of sum<dy, y> + <dfinal, final_state>, from the ``states`` of
    ``selective_scan(..., save=True)`` on the same arguments. Returns dict(dx, ddt [B,T,D], dA [D,NS]
    fp32, dB, dC [B,T,G,NS], dskip [D] fp32 or None, dz [B,T,D] or None, ddt_bias [D] fp32 or None, dh0
    [N,D,NS] fp32 or None)."""
    plan, dev, (rows, D, NS, N), strides, ptrs, keep = _scan(x, dt, A, B, C, skip, z, dt_bias, dt_softplus, 2,
                                                             (cu_seqlens, cu_seqlens_dev))
    chunks = plan.size("kda_sscan_num_chunks")
    if chunks < 0:
        raise KdaError(-1, _lib().kda_last_error().decode())
    pst = _need(states, "states", F32, (chunks, D, NS), dev)
    pdy = _need(dy, "dy", x.dtype, x.shape, dev)
    pdf = _need(dfinal, "dfinal", F32, (N, D, NS), dev)
    need = _bytes(plan.size("kda_sscan_bwd_workspace_bytes"))
    rx, rdt, rz, rB, rC = strides
    (dx, pdx), (ddt, pddt), (dz, pdz) = _like(x, rx), _like(dt, rdt), _like(z, rz)
    (dB, pdB), (dC, pdC) = _like(B, rB), _like(C, rC)
    (dA, pdA), (dskip, pds), (dbias, pdb) = _like(A), _like(skip), _like(dt_bias)
    dh0, pdh0 = _new_if(output_dh0, x, (N, D, NS), F32)
    ws, pws = _ws(x, need)
    _launch(dev, _lib().kda_sscan_bwd, plan.ref, *ptrs, pst, pdy, pdf, pdx, pddt, pdA, pdB, pdC, pds, pdz, pdb, pdh0,
            pws, need)
    del keep
    return dict(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dskip=dskip, dz=dz, ddt_bias=dbias, dh0=dh0)


def selective_scan_step(x, dt, A, B, C, state, slots=None, skip=None, z=None, dt_bias=None, dt_softplus=False):
    """One token of each sequence: x, dt, z [B,D], B, C [B,G,NS], state [S,D,NS] fp32 updated in place.
    Returns y [B,D]."""
    plan, dev, (rows, D, NS, _), strides, ptrs, _ = _scan(x, dt, A, B, C, skip, z, dt_bias, dt_softplus, 1,
                                                          (None, None))
    if state.dim() != 3:
        raise ValueError("state must be [S, D, NS]")
    S = state.shape[0]
    pst = _need(state, "state", F32, (S, D, NS), dev)
    psl = _need(slots, "slots", torch.int32, rows, dev)
    y, py = _like(x, strides[0])
    _launch(dev, _lib().kda_sscan_step, plan.ref, *ptrs, psl, S if S <= _I32_MAX else _fit("S", S), pst, py)
    _written((state,))
    return y


# ---- group norm


def _norm(x, groups, weight, bias, gate, activation, center, eps):
    dev = _gpu(x, "x")
    shape = x.shape
    if not shape or groups < 1 or shape[-1] == 0 or shape[-1] % groups:
        raise ValueError(f"the last dimension of x must be a positive multiple of groups ({groups}), got {tuple(shape)}")
    lead, W = len(shape) - 1, shape[-1]
    C = W // groups
    px, x_row = _rows(x, "x", x.dtype, shape, dev, lead)
    pg, gate_row = _rows(gate, "gate", x.dtype, shape, dev, lead)
    first = weight if weight is not None else bias
    shared = first is not None and groups > 1 and first.dim() == 1 and first.shape[0] == C
    n = (C if shared else W,)
    ptrs = (px, _need(weight, "weight", F32, n, dev), _need(bias, "bias", F32, n, dev), pg)
    plan = _plan(_NormDims, x.numel() // W, groups, C, int(bool(center)), _act(activation, (None, "silu", "sigmoid")),
                 int(shared), float(eps), x_row, gate_row, _DT[x.dtype])
    return plan, dev, (x_row, gate_row), ptrs


def group_norm(x, groups, weight=None, bias=None, gate=None, activation=None, center=False, eps=1e-5):
    """Norm over each group of channels of every row of x [..., groups*C]: n = x / rms (or, with
    ``center``, (x - mean) / std), u = n weight + bias, y = act(u), or u act(gate) with a gate of x's
    shape. weight and bias fp32, [groups*C] or [C] (one for all groups). activation: None, "silu",
    "sigmoid". Returns y."""
    plan, dev, (x_row, _), ptrs = _norm(x, groups, weight, bias, gate, activation, center, eps)
    y, py = _like(x, x_row)
    _launch(dev, _lib().kda_group_norm_fwd, plan.ref, *ptrs, py)
    return y


def group_norm_bwd(x, groups, dy, weight=None, bias=None, gate=None, activation=None, center=False, eps=1e-5):
    """Gradients of sum<dy, y>. Returns dict(dx, dweight, dbias, dgate), None where the input is."""
    plan, dev, (x_row, gate_row), ptrs = _norm(x, groups, weight, bias, gate, activation, center, eps)
    pdy = _need(dy, "dy", x.dtype, x.shape, dev)
    need = plan.size("kda_group_norm_bwd_workspace_bytes") if weight is not None or bias is not None else 0
    (dx, pdx), (dw, pdw), (db, pdb), (dgate, pdg) = _like(x, x_row), _like(weight), _like(bias), _like(gate, gate_row)
    ws, pws = _ws(x, need)
    _launch(dev, _lib().kda_group_norm_bwd, plan.ref, *ptrs, pdy, pdx, pdw, pdb, pdg, pws, need)
    return dict(dx=dx, dweight=dw, dbias=db, dgate=dgate)


# ---- KDA


def kda_step(q, k, v, g, beta, state, slots=None, scale=None, beta_logits=False):
    """One token of KDA for each sequence: q, k [B,H,K], v [B,HV,V], g [B,HV,K] fp32, beta [B,HV] fp32 (or
    its logits), state [S,HV,K,V] fp32 updated in place (``fwd_states``' final_state is one). K and V up
    to 256. Returns o [B,HV,V]."""
    dev = _gpu(q, "q")
    if q.dim() != 3 or v.dim() != 3 or state.dim() != 4:
        raise ValueError("q must be [B, H, K], v [B, HV, V] and state [S, HV, K, V]")
    (B, H, K), (HV, V), S, dt = q.shape, v.shape[1:], state.shape[0], q.dtype
    ptrs = (_need(q, "q", dt, (B, H, K), dev), _need(k, "k", dt, (B, H, K), dev), _need(v, "v", dt, (B, HV, V), dev),
            _need(g, "g", F32, (B, HV, K), dev), _need(beta, "beta", F32, (B, HV), dev),
            _need(slots, "slots", torch.int32, (B,), dev))
    pst = _need(state, "state", F32, (S, HV, K, V), dev)
    # by value: a tensor as a key would stand for whatever it held at the first call
    scale = None if scale is None else float(scale)
    _, d = _kda_dims(B, H, HV, K, V, scale, "f32" if dt is F32 else "bf16", bool(beta_logits))
    o, po = _like(v)
    _launch(dev, _lib().kda_step, d, *ptrs, S if S <= _I32_MAX else _fit("S", S), pst, po)
    _written((state,))
    return o
