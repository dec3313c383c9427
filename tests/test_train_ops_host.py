"""Host-side argument checks of the training operators' C entries, without a GPU.

Each entry has one valid argument list over fake addresses (2^56 bytes apart, never
dereferenced on the host), which must pass every check and stop at the first CUDA
call, and a list of single changes with the status that the interface states for
them.  The calls run in a child process without a GPU, so a crash fails the test
and no fake pointer can reach a launch.  The workspace queries are host
computations and are tested by their values.
"""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import ctypes, sys
sys.path.insert(0, ROOT)
import mx_block_quantization_gb300 as mxq
from mx_block_quantization_gb300 import EALIGN, EBADDTYPE, EBADSHAPE, ECUDA, ENULL, EOVERLAP, OK
L = mxq.lib()
P = [(i + 1) << 56 for i in range(12)]  # buffers
BIG = 1 << 40
bad = []
def entry(fn, args, changes):
    """args: name -> value in call order; changes: (name=value, ...) -> status"""
    def call(**new):
        assert not set(new) - set(args), new
        return getattr(L, fn)(*{**args, **new}.values())
    rc = call()
    if rc != ECUDA:
        bad.append((fn, "valid arguments", rc))
    for new, want in changes:
        rc = call(**new)
        if rc != want:
            bad.append((fn, new, rc, want))

F32 = mxq.F32
WS = 1 << 30
entry("mxq_moe_route",
      dict(logits=P[0], dtype=F32, tokens=100, experts=16, ld=20, k=4, mask=P[1], renorm=1, weights=P[2], ids=P[3],
           counts=P[4], loss=P[5], routed=P[6], workspace=P[7], workspace_bytes=WS, stream=None),
      [(dict(dtype=7), EBADDTYPE), (dict(tokens=-1), EBADSHAPE), (dict(tokens=1 << 31), EBADSHAPE),
       (dict(experts=0), EBADSHAPE), (dict(experts=1 << 30, ld=1 << 30), EBADSHAPE), (dict(ld=15), EBADSHAPE),
       (dict(ld=1 << 31), EBADSHAPE), (dict(k=0), EBADSHAPE), (dict(k=17), EBADSHAPE),
       (dict(experts=64, ld=64, k=33), EBADSHAPE), (dict(workspace_bytes=0), EBADSHAPE),
       (dict(workspace_bytes=-1), EBADSHAPE)] +
      [({n: None}, ENULL) for n in ("logits", "weights", "ids", "counts", "loss", "routed", "workspace")] +
      [({n: P[8] + 2}, EALIGN) for n in ("logits", "weights", "ids", "counts", "loss", "routed", "workspace")] +
      [(dict(workspace=P[8] + 8), EALIGN), (dict(weights=P[0]), EOVERLAP), (dict(ids=P[2] + 1596), EOVERLAP),
       (dict(loss=P[1] + 96), EOVERLAP), (dict(routed=P[5]), EOVERLAP), (dict(workspace=P[4]), EOVERLAP)] +
      [(dict(mask=None), ECUDA), (dict(dtype=mxq.BF16, logits=P[8] + 2), ECUDA), (dict(ids=P[2] + 1600), ECUDA),
       (dict(tokens=0, logits=None, weights=None, ids=None), ECUDA)])
entry("mxq_moe_route_backward",
      dict(logits=P[0], dtype=F32, tokens=100, experts=16, ld=20, k=4, mask=P[1], renorm=1, ids=P[2], counts=P[3],
           routed=P[4], dweights=P[5], dloss=P[6], dlogits=P[7], ldd=16, stream=None),
      [(dict(dtype=-1), EBADDTYPE), (dict(tokens=-1), EBADSHAPE), (dict(ld=15), EBADSHAPE), (dict(ldd=15), EBADSHAPE),
       (dict(ldd=1 << 31), EBADSHAPE), (dict(k=0), EBADSHAPE), (dict(experts=-4), EBADSHAPE)] +
      [({n: None}, ENULL) for n in ("logits", "ids", "counts", "routed", "dlogits")] +
      [({n: P[8] + 2}, EALIGN) for n in ("logits", "ids", "counts", "routed", "dweights", "dloss", "dlogits")] +
      [(dict(dlogits=p), EOVERLAP) for p in P[:7]] +
      [(dict(tokens=0, logits=None, ids=None, dlogits=None), OK), (dict(mask=None, dweights=None, dloss=None), ECUDA)])
# 100 x 4 assignments to 8 experts: at most 400 + 8 * 127 rows, in whole groups
M = L.mxq_moe_rows(100, 4, 8)
entry("mxq_moe_plan",
      dict(ids=P[0], tokens=100, k=4, experts=8, M=M, offs=P[1], slots=P[2], source=P[3], workspace=P[4],
           workspace_bytes=WS, stream=None),
      [(dict(tokens=-1), EBADSHAPE), (dict(k=0), EBADSHAPE), (dict(experts=0), EBADSHAPE), (dict(M=M - 128), EBADSHAPE),
       (dict(M=M + 1), EBADSHAPE), (dict(M=1 << 31), EBADSHAPE), (dict(tokens=1 << 20, M=1 << 23, workspace_bytes=0), EBADSHAPE),
       (dict(tokens=1 << 20, M=1 << 23, workspace=None), ENULL)] +
      [({n: None}, ENULL) for n in ("ids", "offs", "slots", "source")] +
      [({n: P[8] + 1}, EALIGN) for n in ("ids", "offs", "slots", "source", "workspace")] +
      [(dict(offs=P[0]), EOVERLAP), (dict(slots=P[0] + 1596), EOVERLAP), (dict(source=P[1] + 28), EOVERLAP)])
entry("mxq_moe_dispatch",
      dict(x=P[0], dtype=F32, tokens=100, D=24, ldx=32, k=4, slots=P[1], source=P[2], M=M, rows=P[3], ldr=24, stream=None),
      [(dict(dtype=9), EBADDTYPE), (dict(tokens=-1), EBADSHAPE), (dict(D=-1), EBADSHAPE), (dict(ldx=23), EBADSHAPE),
       (dict(ldr=23), EBADSHAPE), (dict(ldr=1 << 31), EBADSHAPE), (dict(k=0), EBADSHAPE), (dict(M=-128), EBADSHAPE)] +
      [({n: None}, ENULL) for n in ("x", "slots", "source", "rows")] +
      [({n: P[8] + 2}, EALIGN) for n in ("x", "slots", "source", "rows")] +
      [(dict(rows=p), EOVERLAP) for p in P[:3]] +
      [(dict(M=0, source=None, rows=None), OK), (dict(D=0), OK), (dict(tokens=0, x=None, slots=None), ECUDA)])
entry("mxq_moe_combine",
      dict(rows=P[0], dtype=F32, M=M, D=24, ldr=24, tokens=100, k=4, slots=P[1], weights=P[2], y=P[3], ldy=24, stream=None),
      [(dict(dtype=9), EBADDTYPE), (dict(tokens=-1), EBADSHAPE), (dict(D=-1), EBADSHAPE), (dict(ldr=23), EBADSHAPE),
       (dict(ldy=23), EBADSHAPE), (dict(k=1 << 20), EBADSHAPE), (dict(M=-1), EBADSHAPE)] +
      [({n: None}, ENULL) for n in ("rows", "slots", "y")] +
      [({n: P[8] + 2}, EALIGN) for n in ("rows", "slots", "weights", "y")] +
      [(dict(y=p), EOVERLAP) for p in P[:3]] + [(dict(tokens=0), OK), (dict(D=0), OK), (dict(weights=None), ECUDA)])
entry("mxq_moe_combine_backward",
      dict(dy=P[0], dtype=F32, tokens=100, D=24, ldy=24, rows=P[1], ldr=24, M=M, k=4, slots=P[2], source=P[3], weights=P[4],
           drows=P[5], ldd=24, dweights=P[6], stream=None),
      [(dict(dtype=9), EBADDTYPE), (dict(tokens=-1), EBADSHAPE), (dict(ldy=23), EBADSHAPE), (dict(ldr=23), EBADSHAPE),
       (dict(ldd=23), EBADSHAPE), (dict(k=0), EBADSHAPE)] +
      [({n: None}, ENULL) for n in ("dy", "rows", "slots", "source", "weights", "drows", "dweights")] +
      [({n: P[8] + 2}, EALIGN) for n in ("dy", "rows", "slots", "source", "weights", "drows", "dweights")] +
      [(dict(drows=p), EOVERLAP) for p in P[:5]] + [(dict(dweights=p), EOVERLAP) for p in P[:6]] +
      [(dict(tokens=0, M=0), OK)])
for width in (4, 8):
    entry("mxq_embedding",
          dict(ids=P[0], ids_bytes=width, tokens=100, table=P[1], dtype=F32, rows=50, D=24, ldw=24, scale=1.0, y=P[2],
               out_dtype=mxq.BF16, ldy=24, stream=None),
          [(dict(dtype=9), EBADDTYPE), (dict(out_dtype=9), EBADDTYPE), (dict(ids_bytes=2), EBADDTYPE),
           (dict(tokens=1 << 29), EBADSHAPE), (dict(tokens=-1), EBADSHAPE), (dict(rows=-1), EBADSHAPE),
           (dict(D=-1), EBADSHAPE), (dict(ldw=23), EBADSHAPE), (dict(ldy=23), EBADSHAPE)] +
          [({n: None}, ENULL) for n in ("ids", "table", "y")] +
          [(dict(ids=P[8] + 2), EALIGN), (dict(table=P[8] + 2), EALIGN), (dict(y=P[8] + 1), EALIGN),
           (dict(y=P[0]), EOVERLAP), (dict(y=P[1]), EOVERLAP), (dict(tokens=0), OK), (dict(D=0), OK),
           (dict(rows=0, table=None), ECUDA)])
    entry("mxq_embedding_backward",
          dict(ids=P[0], ids_bytes=width, tokens=100, dy=P[1], dtype=F32, D=24, ldd=24, rows=50, padding=-1, scale=1.0,
               dtable=P[2], out_dtype=F32, ldw=24, workspace=P[3], workspace_bytes=WS, stream=None),
          [(dict(dtype=9), EBADDTYPE), (dict(out_dtype=9), EBADDTYPE), (dict(ids_bytes=3), EBADDTYPE),
           (dict(tokens=1 << 29), EBADSHAPE), (dict(rows=-1), EBADSHAPE), (dict(ldd=23), EBADSHAPE),
           (dict(ldw=23), EBADSHAPE), (dict(workspace_bytes=0), EBADSHAPE)] +
          [({n: None}, ENULL) for n in ("ids", "dy", "dtable", "workspace")] +
          [(dict(ids=P[8] + 2), EALIGN), (dict(dy=P[8] + 2), EALIGN), (dict(dtable=P[8] + 2), EALIGN),
           (dict(workspace=P[8] + 8), EALIGN)] +
          [(dict(dtable=p), EOVERLAP) for p in (P[0], P[1], P[3])] +
          [(dict(workspace=p), EOVERLAP) for p in (P[0], P[1])] + [(dict(rows=0), OK), (dict(D=0), OK)])
entry("mxq_orthogonalize",
      dict(g=P[0], dtype=F32, batch=2, m=100, n=50, ld=50, stride=5000, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7,
           scale=1.0, out=P[1], ldo=50, stride_o=5000, workspace=P[2], workspace_bytes=WS, stream=None),
      [(dict(dtype=9), EBADDTYPE), (dict(batch=-1), EBADSHAPE), (dict(batch=65536), EBADSHAPE), (dict(m=-1), EBADSHAPE),
       (dict(m=(1 << 20) + 1, stride=1 << 39, stride_o=1 << 39), EBADSHAPE), (dict(ld=49), EBADSHAPE),
       (dict(ldo=49), EBADSHAPE), (dict(stride=4999), EBADSHAPE), (dict(stride_o=0), EBADSHAPE),
       (dict(stride=-5000), EBADSHAPE), (dict(stride=BIG + 1), EBADSHAPE), (dict(steps=0), EBADSHAPE),
       (dict(steps=65), EBADSHAPE), (dict(a=float("nan")), EBADSHAPE), (dict(b=float("inf")), EBADSHAPE),
       (dict(eps=-1.0), EBADSHAPE), (dict(scale=float("inf")), EBADSHAPE), (dict(workspace_bytes=0), EBADSHAPE)] +
      [({n: None}, ENULL) for n in ("g", "out", "workspace")] +
      [(dict(g=P[8] + 2), EALIGN), (dict(out=P[8] + 1), EALIGN), (dict(workspace=P[8] + 8), EALIGN),
       (dict(out=P[0] + 39996), EOVERLAP), (dict(out=P[2]), EOVERLAP), (dict(workspace=P[0]), EOVERLAP),
       (dict(batch=0), OK), (dict(m=0), OK), (dict(n=0), OK), (dict(batch=1, stride=0, stride_o=0), ECUDA)])

def equal(what, got, want):
    if got != want:
        bad.append((what, got, want))
for T in (0, 1, 100, 4096, 65537):
    for k in (1, 3, 32):
        for E in (1, 8, 257):
            # one assignment to each of the groups but the first, which has the others
            n = T * k
            used = min(n, E)
            rows = L.mxq_moe_rows(T, k, E)
            worst = (used - 1) * 128 + (n - used + 1 + 127) // 128 * 128 if used else 0
            equal(("rows whole groups", T, k, E), rows % 128, 0)
            if rows < worst or rows > n + 127 * min(n, E):
                bad.append(("rows", T, k, E, rows, worst))
            if L.mxq_moe_plan_workspace(T, k, E) < 0 or L.mxq_moe_route_workspace(T, E) < 0:
                bad.append(("workspace", T, k, E))
for args in ((-1, 2, 4), (10, 0, 4), (10, 2, 0), (1 << 31, 1, 1), ((1 << 31) - 1, 2, 4)):
    equal(("rows", args), L.mxq_moe_rows(*args), EBADSHAPE)
    equal(("plan workspace", args), L.mxq_moe_plan_workspace(*args), EBADSHAPE)
for args in ((-1, 4), (4, 0), (1 << 31, 4), (4, 1 << 30)):
    equal(("route workspace", args), L.mxq_moe_route_workspace(*args), EBADSHAPE)
for args in ((-1, 4, 4), (4, -1, 4), (4, 4, -1), (1 << 29, 4, 4)):
    equal(("embedding workspace", args), L.mxq_embedding_backward_workspace(*args), EBADSHAPE)
for args in ((-1, 4, 4), (1, -4, 4), (1, 4, (1 << 20) + 1), (65536, 4, 4), (65535, 1 << 20, 1 << 20)):
    equal(("orthogonalize workspace", args), L.mxq_orthogonalize_workspace(*args), EBADSHAPE)
print("BAD", len(bad))
for b in bad[:20]:
    print(b)
'''


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: never where a GPU is visible")
def test_argument_checks():
    import mx_block_quantization_gb300 as mxq
    if not mxq.LIB_PATH.exists():
        import __graft_entry__
        __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", CHILD.replace("ROOT", repr(ROOT))], capture_output=True, text=True,
                       timeout=600, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0, f"child crashed or failed (rc {r.returncode}):\n{r.stderr[-3000:]}"
    assert "BAD 0" in r.stdout, r.stdout[-3000:]


def test_the_binding_takes_no_cpu_tensors():
    import mx_block_quantization_gb300 as mxq
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    plan = mxq.MoePlan(torch.zeros(3, dtype=torch.int32), ids, torch.zeros(128, dtype=torch.int32))
    for call in (lambda: mxq.moe_route(x, 2), lambda: mxq.moe_plan(ids, 3), lambda: mxq.moe_dispatch(x, plan),
                 lambda: mxq.moe_combine(x, plan), lambda: mxq.embedding(ids, x),
                 lambda: mxq.embedding_backward(ids, torch.zeros(4, 2, 8), 4), lambda: mxq.orthogonalize(x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
