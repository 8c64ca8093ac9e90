"""Layer operators without a GPU: refusals of the C ABI and the binding, size queries, and the 64-bit
reference's own gradients against differences."""
import ctypes

import pytest
import torch

import chunked_gated_delta_09_amd as kda
from chunked_gated_delta_09_amd import layers
from tests import layer_ref as ref

P = ctypes.c_void_p(256)  # never read: every call here fails its checks
BIG = 1 << 50


def conv_dims(**kw):
    d = layers._ConvDims(2, 10, 64, 4, 2, None, None, 0, 1, 1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def scan_dims(**kw):
    d = layers._ScanDims(2, 10, 64, 16, 1, 2, None, None, 0, 0, 0, 0, 0, 1, 1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def norm_dims(**kw):
    d = layers._NormDims(10, 4, 32, 0, 2, 1, 1e-5, 0, 0, 1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def host_cuts(cu):
    return (ctypes.c_int32 * len(cu))(*cu)


def refused(status, code, text):
    assert status == code, kda.load().kda_last_error().decode()
    assert text in kda.load().kda_last_error().decode()


def packed(d, cu):
    arr = host_cuts(cu)
    d.B, d.T, d.N = 1, max(cu), len(cu) - 1
    d.cu_seqlens_host, d.cu_seqlens_dev = arr, 256
    return arr


def call_conv(d, x=P, w=P, y=P):
    return layers._lib().kda_short_conv_fwd(ctypes.byref(d), x, w, None, None, y, None, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(W=1), -2, "W must be"), (dict(W=5), -2, "W must be"), (dict(D=0), -1, "D must be"), (dict(B=0), -1, "positive"),
    (dict(T=-1), -1, "positive"), (dict(N=3), -1, "N == B"), (dict(act=2), -1, "act"), (dict(dtype=7), -1, "dtype"),
    (dict(x_row=63), -1, "x_row"), (dict(B=1 << 20, N=1 << 20, T=1 << 20), -1, "too many tokens")])
def test_conv_refusals(kw, code, text):
    refused(call_conv(conv_dims(**kw)), code, text)
    assert layers._lib().kda_short_conv_bwd_workspace_bytes(ctypes.byref(conv_dims(**kw))) == 0


@pytest.mark.parametrize("cu,text", [([0, 6, 4, 10], "non-decreasing"), ([1, 4, 10], "cu_seqlens[0]")])
def test_bad_cuts(cu, text):
    d = conv_dims()
    keep = packed(d, cu)
    refused(call_conv(d), -1, text)
    s = scan_dims()
    keep = packed(s, cu)
    refused(layers._lib().kda_sscan_fwd(ctypes.byref(s), *[P] * 13, BIG, None), -1, text)
    del keep


def test_cuts_need_both_copies():
    d = conv_dims()
    keep = packed(d, [0, 4, 10])
    d.cu_seqlens_dev = None
    refused(call_conv(d), -1, "both given or both NULL")
    d.T = 11
    d.cu_seqlens_dev = 256
    refused(call_conv(d), -1, "must equal T")
    del keep


def test_conv_null_and_workspace():
    d = conv_dims()
    refused(call_conv(d, x=None), -1, "x is NULL")
    refused(call_conv(d, w=None), -1, "weight is NULL")
    lib = layers._lib()
    need = lib.kda_short_conv_bwd_workspace_bytes(ctypes.byref(d))
    assert need > 0
    for ws, n, text in [(None, need, "workspace is NULL"), (P, need - 1, "too small"), (ctypes.c_void_p(257), need, "aligned")]:
        refused(lib.kda_short_conv_bwd(ctypes.byref(d), P, P, None, None, P, None, P, P, None, None, ws, n, None), -1, text)


@pytest.mark.parametrize("kw,code,text", [
    (dict(NS=0), -2, "NS"), (dict(NS=65), -2, "NS"), (dict(G=3), -1, "multiple of G"), (dict(G=0), -1, "multiple of G"),
    (dict(softplus=2), -1, "softplus"), (dict(dtype=5), -1, "dtype"), (dict(z_row=1), -1, "z_row"), (dict(b_row=15), -1, "b_row"),
    (dict(B=1 << 15, N=1 << 15, T=60000, D=1 << 20), -1, "too many")])
def test_scan_refusals(kw, code, text):
    d, lib = scan_dims(**kw), layers._lib()
    refused(lib.kda_sscan_fwd(ctypes.byref(d), *[P] * 13, BIG, None), code, text)
    assert lib.kda_sscan_num_chunks(ctypes.byref(d)) == -1
    assert lib.kda_sscan_bwd_workspace_bytes(ctypes.byref(d)) == 0


def test_scan_null_alignment_and_workspace():
    d, lib = scan_dims(), layers._lib()
    odd = ctypes.c_void_p(260)
    a = [P] * 12
    refused(lib.kda_sscan_fwd(ctypes.byref(d), None, *a[1:], None, 0, None), -1, "x is NULL")
    refused(lib.kda_sscan_fwd(ctypes.byref(d), *a[:2], odd, *a[3:], None, 0, None), -1, "A must be 16-byte aligned")
    b = [P] * 20
    need = lib.kda_sscan_bwd_workspace_bytes(ctypes.byref(d))
    refused(lib.kda_sscan_bwd(ctypes.byref(d), *b, None, need, None), -1, "workspace is NULL")
    refused(lib.kda_sscan_bwd(ctypes.byref(d), *b, P, need - 1, None), -1, "too small")
    no_z = list(b)
    no_z[6] = None
    refused(lib.kda_sscan_bwd(ctypes.byref(d), *no_z, P, need, None), -1, "needed for dz")
    # a long sequence of few channels is cut: the forward needs room for the segments
    long = scan_dims(B=1, N=1, T=10000)
    assert lib.kda_sscan_fwd_workspace_bytes(ctypes.byref(long)) > 0
    assert lib.kda_sscan_num_chunks(ctypes.byref(long)) == 625


def test_scan_chunks_of_packed_sequences():
    d = scan_dims()
    keep = packed(d, [0, 0, 1, 17, 50])
    assert layers._lib().kda_sscan_num_chunks(ctypes.byref(d)) == 0 + 1 + 1 + 3
    del keep


@pytest.mark.parametrize("kw,code,text", [
    (dict(C=8193, G=1), -2, "at most 8192"), (dict(C=0), -1, "positive"), (dict(R=-1), -1, "positive"), (dict(eps=0.0), -1, "eps"),
    (dict(eps=float("nan")), -1, "eps"), (dict(center=2), -1, "center"), (dict(act=3), -1, "act"), (dict(shared=5), -1, "shared"),
    (dict(gate_row=127), -1, "gate_row"), (dict(G=1 << 16, C=8192), -1, "G * C")])
def test_norm_refusals(kw, code, text):
    d, lib = norm_dims(**kw), layers._lib()
    refused(lib.kda_group_norm_fwd(ctypes.byref(d), P, None, None, None, P, None), code, text)
    assert lib.kda_group_norm_bwd_workspace_bytes(ctypes.byref(d)) == 0


def test_step_refusals():
    lib = layers._lib()

    def conv(S, slots=P, **kw):
        d = conv_dims(T=1, **kw)
        return lib.kda_short_conv_step(ctypes.byref(d), P, P, None, slots, S, P, P, None)

    refused(conv(0), -1, "S (rows")
    refused(conv(1, slots=None), -1, "a row for each")
    d = conv_dims(T=2)
    refused(lib.kda_short_conv_step(ctypes.byref(d), P, P, None, P, 4, P, P, None), -1, "one token")
    refused(conv(4, B=70000, N=70000), -1, "1 <= B")
    k, _ = kda.make_dims(2, 1, 2, 4, 128, 128, 16)
    args = [P] * 6
    refused(lib.kda_step(ctypes.byref(k), *args, 0, P, P, None), -1, "S (rows")
    for kw, code, text in [(dict(K=257), -2, "at most 256"), (dict(HV=3), -1, "multiple of H"), (dict(T=2), -1, "one token"),
                           (dict(beta_logits=3), -1, "beta_logits"), (dict(scale=float("inf")), -1, "scale")]:
        k, _ = kda.make_dims(2, 1, 2, 4, 128, 128, 16)
        for n, v in kw.items():
            setattr(k, n, v)
        refused(lib.kda_step(ctypes.byref(k), *args, 4, P, P, None), code, text)


def test_binding_refuses_host_tensors_and_wrong_arguments():
    x = torch.zeros(1, 4, 8)
    w = torch.zeros(8, 4)
    with pytest.raises(ValueError, match="GPU tensor"):
        layers.short_conv(x, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        layers.selective_scan(x, x, torch.zeros(8, 4), torch.zeros(1, 4, 1, 4), torch.zeros(1, 4, 1, 4))
    with pytest.raises(ValueError, match="GPU tensor"):
        layers.group_norm(x, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        layers.kda_step(torch.zeros(1, 1, 16), torch.zeros(1, 1, 16), torch.zeros(1, 1, 16), torch.zeros(1, 1, 16),
                        torch.zeros(1, 1), torch.zeros(1, 1, 16, 16))


class _Gpu:
    """Stands in for a GPU tensor's description: strides are checked before anything is launched."""

    def __init__(self, t):
        self.t = t
        self.is_cuda, self.dtype, self.shape = True, t.dtype, t.shape

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("make,row", [
    (lambda: torch.zeros(3, 5, 8), 0), (lambda: torch.zeros(3, 5, 20)[..., 4:12], 20), (lambda: torch.zeros(1, 1, 20)[..., :8], 0),
    (lambda: torch.zeros(3, 1, 20)[..., :8], 20), (lambda: torch.zeros(1, 5, 20)[..., :8], 20), (lambda: torch.zeros(3, 0, 8), 0),
    (lambda: torch.zeros(5, 3, 8).transpose(0, 1), None), (lambda: torch.zeros(3, 5, 16)[..., ::2], None),
    (lambda: torch.zeros(3, 9, 8)[:, :5], None), (lambda: torch.zeros(3, 1, 8).expand(3, 5, 8), None),
    (lambda: torch.zeros(3, 8, 5).transpose(1, 2), None)])
def test_row_strides(make, row):
    t = _Gpu(make())
    if row is None:
        with pytest.raises(ValueError, match="column slice"):
            layers._rows(t, "x", t.dtype, t.shape, 0, 2)
    else:
        got = layers._rows(t, "x", t.dtype, t.shape, 0, 2)
        assert got == (t.data_ptr(), row)


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(1)

    def r(*s):
        return torch.randn(*s, generator=g, dtype=ref.F64).requires_grad_()

    cu = [0, 2, 2, 5]
    assert torch.autograd.gradcheck(lambda x, w, b, h: ref.conv(x, w, b, h, "silu", cu), (r(1, 5, 3), r(3, 4), r(3), r(3, 3, 3)))
    A = -torch.rand(4, 3, generator=g, dtype=ref.F64)
    A.requires_grad_()
    assert torch.autograd.gradcheck(
        lambda x, dt, A, B, C, sk, z, tb, h: ref.scan(x, dt, A, B, C, sk, z, tb, h, True, cu),
        (r(1, 5, 4), r(1, 5, 4), A, r(1, 5, 2, 3), r(1, 5, 2, 3), r(4), r(1, 5, 4), r(4), r(3, 4, 3)))
    for act, center in (("silu", True), ("sigmoid", False)):
        assert torch.autograd.gradcheck(lambda x, w, b, z: ref.norm(x, 2, w, b, z, act, center, 1e-5), (r(3, 8), r(4), r(8), r(3, 8)))
        assert torch.autograd.gradcheck(lambda x, w, b: ref.norm(x, 2, w, b, None, act, center, 1e-5), (r(3, 8), r(8), r(8)))
