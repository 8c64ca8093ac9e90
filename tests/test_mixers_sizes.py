"""Sizes and limits of the token mixers' calls, as the library answers them (no GPU)."""
import ctypes
import os
import subprocess
import sys

import pytest

from chunked_gated_delta_09_amd import mixers
from tests.test_mixers_host import P, lin_bwd, lin_dims, lin_fwd, packed, refused, win_bwd, win_dims, win_fwd, win_step

FIRST_QUERY = """
import ctypes
from chunked_gated_delta_09_amd import layers, mixers
cu = list(range(2200)) + [30000]
host = (ctypes.c_int32 * len(cu))(*cu)
if {lin}:
    plan = layers._plan_of(mixers._LinDims, 256, host, (1, cu[-1], 32, 32, 128, 128, len(cu) - 1), (0, 0, 0, 0, 1.0, 1))
else:
    plan = layers._plan_of(mixers._WinDims, None, None, (1, 1 << 22, 255, 1, 256, 1), (0, 0, 0, 8, 1024, 1.0, 1))
print(plan.size("{query}"))
"""


@pytest.mark.parametrize("lin,query", [(True, "kda_lattn_fwd_workspace_bytes"), (True, "kda_lattn_bwd_workspace_bytes"),
                                       (False, "kda_wattn_bwd_workspace_bytes")])
def test_the_first_query_of_a_process_answers_past_32_bits(lin, query):
    """Nothing has declared the library's functions yet when a plan asks for a size."""
    r = subprocess.run([sys.executable, "-c", FIRST_QUERY.format(lin=lin, query=query)], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr
    # a state of every sequence's; do.o of every row and one part of the queries at the least
    least = 2200 * 32 * 128 * 128 * 4 if lin else (1 << 22) * 255 * 4 + 1024 * 2 * 256 * 4 * 10
    assert int(r.stdout) >= least > 1 << 32


@pytest.mark.parametrize("K,V", [(8, 128), (128, 8)])
def test_grids_of_512_threads(K, V):
    """Tiles of 128 columns have workgroups of 512 threads: 2^23 of them are more threads than a launch takes."""
    lib = mixers._lib()
    d = lin_dims(B=2100, N=2100, T=1, H=1 << 12, HV=1 << 12, K=K, V=V)
    if V > 64:  # the forward has tiles of V alone
        refused(lin_fwd(d), -1, "too many segments")
    refused(lin_bwd(d), -1, "too many segments")
    assert lib.kda_lattn_num_states(ctypes.byref(d)) == -1
    assert lib.kda_lattn_bwd_workspace_bytes(ctypes.byref(d)) == 0
    d.K, d.V = 8, 64
    assert lib.kda_lattn_num_states(ctypes.byref(d)) == 2 * 2100  # of 256 threads each


def test_linear_limits_are_of_what_is_launched():
    """The segments' scan is for sequences that are cut, and in the backward for gradients of final states."""
    lib = mixers._lib()
    d = lin_dims(B=40000, N=40000, T=1, H=32, HV=32, K=128, V=128)  # the scan would have 20 million workgroups
    assert lib.kda_lattn_num_states(ctypes.byref(d)) == 2 * 40000
    assert lib.kda_lattn_fwd_workspace_bytes(ctypes.byref(d)) == 0 and lib.kda_lattn_bwd_workspace_bytes(ctypes.byref(d)) > 0
    refused(lin_fwd(d, *[None if i == 5 else P for i in range(8)]), -1, "o is NULL")
    refused(lin_bwd(d, nulls={6, 7}), -1, "dq is NULL")
    refused(lin_bwd(d), -1, "too many segments")
    cu = list(range(40000)) + [50000]  # the last one is cut
    host = packed(d, cu)
    refused(lin_fwd(d), -1, "too many segments")
    refused(lin_bwd(d, nulls={6}), -1, "too many segments")
    assert lib.kda_lattn_num_states(ctypes.byref(d)) == -1
    del host


@pytest.mark.parametrize("B,HV,K,V", [(8192, 32, 256, 256), (32768, 32, 128, 128), (65535, 256, 64, 64)])
def test_linear_steps_have_no_limit_of_whole_sequences(B, HV, K, V):
    d = lin_dims(B=B, N=B, T=1, H=HV, HV=HV, K=K, V=V)
    refused(mixers._lib().kda_lattn_step(ctypes.byref(d), P, P, P, P, P, 4, P, None, None), -1, "o is NULL")


def test_window_limits_are_of_what_is_launched():
    """First tokens have kernels of their own in the backward of sequences longer than the window."""
    lib = mixers._lib()
    d = win_dims(B=4096, N=4096, T=9, H=8, HK=8, sinks=512)
    refused(win_fwd(d, nulls={3}), -1, "o is NULL")
    refused(win_bwd(d), -1, "too many first tokens")
    assert lib.kda_wattn_bwd_workspace_bytes(ctypes.byref(d)) == 0
    d.window = 9
    refused(win_bwd(d, nulls={6}), -1, "dq is NULL")
    assert lib.kda_wattn_bwd_workspace_bytes(ctypes.byref(d)) == 4096 * 9 * 8 * 4


@pytest.mark.parametrize("B,H,HK,sinks", [(4096, 8, 8, 512), (65535, 256, 16, 4)])
def test_window_steps_have_no_limit_of_whole_sequences(B, H, HK, sinks):
    d = win_dims(B=B, N=B, T=1, H=H, HK=HK, sinks=sinks)
    assert mixers._lib().kda_wattn_step_workspace_bytes(ctypes.byref(d)) == 0
    refused(win_step(d, nulls={7}), -1, "o is NULL")


def test_the_join_of_a_window_step_has_its_own_limit():
    """A workgroup for each head of each sequence, where a key head's cache rows are dealt to several."""
    lib = mixers._lib()
    d = win_dims(B=500, N=500, T=1, H=1 << 16, HK=1, D=8, window=1000)
    refused(win_step(d, S=500), -1, "too many heads")
    assert lib.kda_wattn_step_workspace_bytes(ctypes.byref(d)) == ctypes.c_size_t(-1).value
    for change in (dict(window=100), dict(B=250, N=250)):  # one workgroup a key head; fewer than 2^24 of the join
        for n, v in change.items():
            setattr(d, n, v)
        refused(win_step(d, S=500, nulls={7}), -1, "o is NULL")
        d.window = 1000
