"""How the library plans the layer operators' calls, seen through its size queries (no GPU)."""
import ctypes

import pytest
import torch

from chunked_gated_delta_09_amd import layers


def norm_bwd_bytes(R, G, C, shared=0, dtype=torch.bfloat16):
    d = layers._NormDims(R, G, C, 0, 0, shared, 1e-5, 0, 0, layers._DT[dtype])
    return layers._lib().kda_group_norm_bwd_workspace_bytes(ctypes.byref(d))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("G,C", [(g, c) for g in (1, 3, 31, 32, 255, 1023, 4097, 65535) for c in (1, 8, 16, 100, 1000)
                                 if g * c <= 1 << 20])
@pytest.mark.parametrize("R", [1, 7, 1000, 100000])
def test_norm_backward_workspace(R, G, C, dtype):
    """Sums of one weight a channel: no more rows of them than rows of x, and not more bytes than x and a
    call's fixed share (1024 workgroups of at most 4096 channels, two sums, 4 bytes)."""
    got = norm_bwd_bytes(R, G, C, dtype=dtype)
    if R * G > 2 ** 31 - 65:
        assert got == 0  # refused: too many groups
        return
    row = 2 * G * C * 4
    assert 0 < got <= R * row + 256
    assert got <= row + 1024 * 4096 * 2 * 4 + 256


def up(x, m):
    return -(-x // m) * m


def scan_plan(lens, D, NS, G, bwd):
    """Tokens of a segment and of a local one, by the rule of the library's scan: about four workgroups a CU (backward
    two), no cut below two such segments; a call that leaves the chip idle by its latency."""
    NP = next(n for n in (8, 16, 32, 64) if NS <= n)
    tiles = up(D // G, 1024 // NP) // (1024 // NP)
    total, longest, cols = sum(lens), max(lens), G * tiles
    whole, want = max(up(longest, 16), 16), 512 if bwd else 1024
    least = 1
    while least * least * 36 * 36 < longest:
        least += 1
    least *= 16
    seg = up(up(total * cols, want) // want, 16)
    small = seg <= least
    seg = least if small else seg
    if whole <= (4 if small else 2) * seg:
        return whole, whole, NP, tiles
    r = 1
    while r < 4 and (total // seg + len(lens)) * cols * r * 2 <= 2048 and seg // (r * 2) >= least:
        r *= 2
    seg = up(seg, 16 * r)
    return seg, seg // r, NP, tiles


def scan_bytes(lens, packed, D, NS, G, bwd):
    """The workspace that follows from the plan, array by array."""
    seg, lseg, NP, tiles = scan_plan(lens, D, NS, G, bwd)
    nseg, nloc = (sum(max(1, up(n, s) // s) for n in lens) for s in (seg, lseg))
    sizes = [4 * (len(lens) + 1)] * 3 if packed and len(lens) > 64 else []
    if max(lens) > seg:
        sizes += [4 * nloc * D, 4 * nloc * D * NP]
    if bwd:
        sizes += [4 * tiles * sum(lens) * G * 2 * NP, 4 * nseg * D * NP, 4 * nseg * 2 * D]
    return sum(up(s, 256) for s in sizes)


def scan_query(lens, packed, D, NS, G, bwd):
    if packed:
        cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
        host = (ctypes.c_int32 * len(cu))(*cu)
        d = layers._ScanDims(1, cu[-1], D, NS, G, len(lens), 256, host, 0, 0, 0, 0, 0, 1, 0)
    else:
        d = layers._ScanDims(len(lens), lens[0], D, NS, G, len(lens), None, None, 0, 0, 0, 0, 0, 1, 0)
    name = "kda_sscan_bwd_workspace_bytes" if bwd else "kda_sscan_fwd_workspace_bytes"
    return getattr(layers._lib(), name)(ctypes.byref(d))


# lengths, packed or not, channels, states, groups; then segment and local segment of the forward and the backward
CUT = {
    "several_chunks": ([1700], False, 48, 16, 48, (80, 80), (160, 80)),
    "halves": ([688], False, 72, 5, 24, (32, 16), (64, 32)),
    "quarters": ([1999], False, 64, 16, 32, (64, 32), (128, 32)),
    "two_dense": ([261, 261], False, 96, 8, 48, (32, 16), (64, 16)),
    "tiles": ([900], False, 600, 32, 1, (32, 16), (64, 32)),
    "packed": ([538, 0, 1, 149], True, 48, 16, 24, (32, 16), (64, 32)),
    "packed_quarters": ([904, 0, 1, 149], True, 48, 13, 24, (32, 16), (64, 16)),
    "packed_tables": ([0, 1, 2] * 25 + [8300, 40, 700], True, 12, 8, 6, (64, 64), (128, 64)),
}


@pytest.mark.parametrize("name", list(CUT))
def test_scan_segments(name):
    """The cases of the GPU tests of cut sequences are cut as they are meant to be."""
    lens, packed, D, NS, G, fwd, bwd = CUT[name]
    for back, want in ((False, fwd), (True, bwd)):
        assert scan_plan(lens, D, NS, G, back)[:2] == want
        assert scan_query(lens, packed, D, NS, G, back) == scan_bytes(lens, packed, D, NS, G, back)


@pytest.mark.parametrize("lens,packed,D,NS,G", [
    ([2048, 2048], False, 2048, 16, 1), ([16384], False, 2048, 16, 1), ([1], False, 8, 8, 1), ([37] * 5, False, 64, 13, 4),
    ([300, 0, 1, 777], True, 200, 8, 2), ([0, 3] * 50 + [4000], True, 64, 64, 1), ([100000], False, 16, 5, 1)])
def test_scan_workspaces(lens, packed, D, NS, G):
    for back in (False, True):
        assert scan_query(lens, packed, D, NS, G, back) == scan_bytes(lens, packed, D, NS, G, back)
