"""Workspaces of the routing's C entry, on the host: which calls need one, and that a
call with a smaller one, with none, or with one over an output is refused, beside every
number of experts.  The calls run in a child process without a GPU over fake addresses
(2^56 bytes apart); accepted ones stop at the first CUDA call.
"""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys
sys.path.insert(0, ROOT)
import mx_block_quantization_gb300 as mxq
from mx_block_quantization_gb300 import EBADSHAPE, ECUDA, ENULL, EOVERLAP
L = mxq.lib()
P = [(i + 1) << 56 for i in range(9)]
def route(T, E, workspace, size):
    return L.mxq_moe_route(P[0], mxq.F32, T, E, E, 1, P[1], 1, P[2], P[3], P[4], P[5], P[6], workspace, size, None)
bad = []
for E in (1, 8, 9, 16, 31, 32, 33, 64, 256, 257, 512, 513, 1024):
    for T in (0, 1, 8, 9, 16, 17, 32, 33, 100, 128, 129, 300, 5000, 200000):
        need = L.mxq_moe_route_workspace(T, E)
        at_once = 32 if E <= 256 else 16 if E <= 512 else 8     # tokens without one
        if (need > 0) != (T > at_once):
            bad.append(("need", T, E, need))
        got = [route(T, E, P[7], need), route(T, E, P[7], need + 64)]
        want = [ECUDA, ECUDA]
        if need == 0:
            got.append(route(T, E, None, 0))
            want.append(ECUDA)
        else:
            got += [route(T, E, P[7], need - 1), route(T, E, P[7], 0), route(T, E, None, need), route(T, E, P[4], need)]
            want += [EBADSHAPE, EBADSHAPE, ENULL, EOVERLAP]
        if got != want:
            bad.append((T, E, got, want))
print("BAD", len(bad), bad[:10])
'''


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: never where a GPU is visible")
def test_workspaces_of_every_routing_kernel():
    import mx_block_quantization_gb300 as mxq
    if not mxq.LIB_PATH.exists():
        import __graft_entry__
        __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", CHILD.replace("ROOT", repr(ROOT))], capture_output=True, text=True,
                       timeout=600, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0, f"child crashed or failed (rc {r.returncode}):\n{r.stderr[-3000:]}"
    assert r.stdout.startswith("BAD 0"), r.stdout[-3000:]
