"""Host-side argument checks of the experts' products, grouped routing and AdamW, without
a GPU, as in test_train_ops_host.py: one valid argument list over fake addresses for each
C entry, which has to stop at the first CUDA call, and single changes with their status."""
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
from mx_block_quantization_gb300 import EALIGN, EBADDTYPE, EBADOFFS, EBADSHAPE, ECUDA, ENULL, EOVERLAP, OK
L = mxq.lib()
P = [(i + 1) << 56 for i in range(12)]  # buffers
bad = []
def entry(fn, args, changes):
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

F32, BF16, WS, FAR = mxq.F32, mxq.BF16, 1 << 30, (1 << 24) + 128
entry("mxq_moe_route_groups",
      dict(logits=P[0], dtype=F32, tokens=100, experts=16, ld=20, k=4, bias=P[1], scores=0, groups=4, best=2, mask=P[2], renorm=1,
           scale=2.5, weights=P[3], ids=P[4], counts=P[5], loss=P[6], routed=P[7], workspace=P[8], workspace_bytes=WS, stream=None),
      [(dict(dtype=7), EBADDTYPE), (dict(tokens=-1), EBADSHAPE), (dict(tokens=1 << 31), EBADSHAPE), (dict(experts=0), EBADSHAPE),
       (dict(experts=1 << 30, ld=1 << 30), EBADSHAPE), (dict(ld=15), EBADSHAPE), (dict(ld=1 << 31), EBADSHAPE), (dict(k=0), EBADSHAPE),
       (dict(k=9), EBADSHAPE), (dict(experts=64, ld=64, k=33, best=4), EBADSHAPE), (dict(scores=2), EBADSHAPE), (dict(scores=-1), EBADSHAPE),
       (dict(groups=0), EBADSHAPE), (dict(groups=3), EBADSHAPE), (dict(groups=64, experts=64, ld=64, best=32), EBADSHAPE),
       (dict(best=0), EBADSHAPE), (dict(best=5), EBADSHAPE), (dict(scale=float("inf")), EBADSHAPE), (dict(workspace_bytes=0), EBADSHAPE)] +
      [({n: None}, ENULL) for n in ("logits", "weights", "ids", "counts", "loss", "routed", "workspace")] +
      [({n: P[9] + 2}, EALIGN) for n in ("logits", "bias", "weights", "ids", "counts", "loss", "routed", "workspace")] +
      [(dict(weights=P[0]), EOVERLAP), (dict(ids=P[3] + 1596), EOVERLAP), (dict(counts=P[1] + 60), EOVERLAP),
       (dict(loss=P[2] + 96), EOVERLAP), (dict(routed=P[6]), EOVERLAP), (dict(workspace=P[5]), EOVERLAP)] +
      [(dict(mask=None, bias=None), ECUDA), (dict(dtype=BF16, logits=P[9] + 2), ECUDA), (dict(best=4, k=16), ECUDA),
       (dict(tokens=0, logits=None, weights=None, ids=None), ECUDA)])
entry("mxq_moe_route_groups_backward",
      dict(logits=P[0], dtype=F32, tokens=100, experts=16, ld=20, k=4, scores=1, mask=P[1], renorm=1, scale=1.0, ids=P[2],
           counts=P[3], routed=P[4], dweights=P[5], dloss=P[6], dlogits=P[7], ldd=16, stream=None),
      [(dict(dtype=-1), EBADDTYPE), (dict(tokens=-1), EBADSHAPE), (dict(ld=15), EBADSHAPE), (dict(ldd=15), EBADSHAPE),
       (dict(ldd=1 << 31), EBADSHAPE), (dict(k=17), EBADSHAPE), (dict(scores=3), EBADSHAPE), (dict(scale=float("nan")), EBADSHAPE)] +
      [({n: None}, ENULL) for n in ("logits", "ids", "counts", "routed", "dlogits")] +
      [({n: P[8] + 2}, EALIGN) for n in ("logits", "ids", "counts", "routed", "dweights", "dloss", "dlogits")] +
      [(dict(dlogits=p), EOVERLAP) for p in P[:7]] +
      [(dict(tokens=0, logits=None, ids=None, dlogits=None), OK), (dict(mask=None, dweights=None, dloss=None), ECUDA)])
entry("mxq_moe_linear",
      dict(x=P[0], ldx=256, sx=P[1], w=P[2], ldw=256, stride_w=128 * 256, sw=P[3], offs=P[4], G=3, M=512, N=128, K=256, bias=P[5],
           bias_dtype=F32, activation=2, residual=P[6], ldr=130, dtype=BF16, y=P[7], ldy=129, z=P[8], ldz=128, stream=None),
      [(dict(dtype=9), EBADDTYPE), (dict(bias_dtype=9), EBADDTYPE), (dict(G=0), EBADOFFS), (dict(G=1025), EBADOFFS), (dict(offs=None), EBADOFFS),
       (dict(M=-128), EBADSHAPE), (dict(M=500), EBADSHAPE), (dict(M=FAR), EBADSHAPE), (dict(N=64, ldy=64), EBADSHAPE), (dict(N=FAR), EBADSHAPE),
       (dict(K=100), EBADSHAPE), (dict(K=0), EBADSHAPE), (dict(K=FAR), EBADSHAPE), (dict(activation=4), EBADSHAPE), (dict(activation=-1), EBADSHAPE),
       (dict(ldx=240), EBADSHAPE), (dict(ldx=264), EBADSHAPE), (dict(ldw=128), EBADSHAPE), (dict(stride_w=0), EBADSHAPE),
       (dict(stride_w=40), EBADSHAPE), (dict(ldy=127), EBADSHAPE), (dict(ldz=127), EBADSHAPE), (dict(ldr=127), EBADSHAPE),
       (dict(ldy=1 << 31), EBADSHAPE)] +
      [({n: None}, ENULL) for n in ("x", "sx", "w", "sw", "y")] +
      [({n: P[9] + 8}, EALIGN) for n in ("x", "sx", "w", "sw")] + [(dict(offs=P[9] + 2), EALIGN), (dict(bias=P[9] + 2), EALIGN)] +
      [({n: P[9] + 1}, EALIGN) for n in ("y", "z", "residual")] +
      [(dict(y=p), EOVERLAP) for p in (P[:6] + P[8:9])] + [(dict(z=p), EOVERLAP) for p in P[:8]] +
      [(dict(y=P[6]), EOVERLAP), (dict(y=P[6], ldy=130), ECUDA), (dict(M=0), OK), (dict(N=0), OK), (dict(bias=None, bias_dtype=9), ECUDA),
       (dict(residual=None, ldr=0, z=None, ldz=0), ECUDA), (dict(offs=None, G=0, stride_w=0), ECUDA), (dict(y=P[9] + 2), ECUDA)])
entry("mxq_moe_weight_gradient",
      dict(a=P[0], lda=512, sa=P[1], b=P[2], ldb=512, sb=P[3], offs=P[4], G=3, M=512, N=128, K=256, accumulate=1, dtype=F32, dw=P[5],
           ldd=260, stride_d=260 * 128, stream=None),
      [(dict(dtype=9), EBADDTYPE), (dict(G=0), EBADOFFS), (dict(offs=None), EBADOFFS), (dict(M=130), EBADSHAPE), (dict(N=-128), EBADSHAPE),
       (dict(K=FAR), EBADSHAPE), (dict(lda=511), EBADSHAPE), (dict(lda=520), EBADSHAPE), (dict(ldb=256), EBADSHAPE), (dict(ldd=255), EBADSHAPE),
       (dict(stride_d=260 * 127), EBADSHAPE), (dict(stride_d=-1), EBADSHAPE)] +
      [({n: None}, ENULL) for n in ("a", "sa", "b", "sb", "dw")] + [({n: P[9] + 8}, EALIGN) for n in ("a", "sa", "b", "sb")] +
      [(dict(offs=P[9] + 1), EALIGN), (dict(dw=P[9] + 2), EALIGN)] + [(dict(dw=p), EOVERLAP) for p in P[:5]] +
      [(dict(N=0), OK), (dict(K=0, ldd=0), OK), (dict(M=0, a=None, sa=None, b=None, sb=None), OK),
       (dict(M=0, a=None, sa=None, b=None, sb=None, accumulate=0), ECUDA), (dict(offs=None, G=0, stride_d=0), ECUDA)])
entry("mxq_moe_linear_backward",
      dict(dy=P[0], dtype=BF16, ld_dy=130, z=P[1], ldz=128, activation=3, offs=P[2], G=3, M=512, N=128, dz=P[3], ld_dz=129, dbias=P[4],
           workspace=P[5], workspace_bytes=WS, stream=None),
      [(dict(dtype=9), EBADDTYPE), (dict(G=-1), EBADOFFS), (dict(M=100), EBADSHAPE), (dict(N=100), EBADSHAPE), (dict(activation=7), EBADSHAPE),
       (dict(ld_dy=127), EBADSHAPE), (dict(ldz=127), EBADSHAPE), (dict(ld_dz=127), EBADSHAPE), (dict(workspace_bytes=4 * 128 * 4 - 1), EBADSHAPE)] +
      [({n: None}, ENULL) for n in ("dy", "z", "workspace")] + [({n: P[9] + 1}, EALIGN) for n in ("dy", "z", "dz", "offs", "dbias")] +
      [(dict(workspace=P[9] + 8), EALIGN), (dict(dz=P[0]), EOVERLAP), (dict(dz=P[0], ld_dz=130), ECUDA), (dict(dz=P[1]), EOVERLAP),
       (dict(dbias=P[3]), EOVERLAP), (dict(workspace=P[0]), EOVERLAP), (dict(dbias=P[2]), EOVERLAP),
       (dict(dz=None, dbias=None, workspace=None, workspace_bytes=0), OK), (dict(N=0), OK), (dict(M=0, dbias=None), OK),
       (dict(activation=0, z=None, ldz=0, dz=None), ECUDA), (dict(M=0, dy=None, z=None, dz=None, workspace=None), ECUDA)])

I64 = ctypes.c_int64
def tensors(*entries):
    """(p, grad, copy, n, start, dtype, grad_dtype) of each tensor."""
    flat = []
    for p, g, c, n, s, d, e in entries:
        flat += [p - (1 << 64) if p >> 63 else p, g, c, n, s, d | e << 32]
    return (I64 * len(flat))(*flat)
ONE, TWO = (P[0], P[1], 0, 100, 0, F32, BF16), (P[2], P[3], P[4], 300, 128, BF16, F32)
for bits in (8, 32):
    args = dict(tensors=tensors(ONE, TWO), count=2, bits=bits, m=P[5], v=P[6], m_scale=P[7], v_scale=P[8], total=512, step=1, step_at=None,
                lr=1e-3, lr_at=None, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, grad_scale=P[9], seed=1 << 63, stream=None)
    one = lambda **new: dict(tensors=tensors(tuple({**dict(zip("pgcnsde", ONE)), **new}.values()), TWO))
    entry("mxq_adamw", args,
          [(dict(bits=16), EBADDTYPE), (dict(count=-1), EBADSHAPE), (dict(count=513), EBADSHAPE), (dict(total=-128), EBADSHAPE),
           (dict(total=500), EBADSHAPE), (dict(total=384), EBADSHAPE), (dict(step=0), EBADSHAPE), (dict(step=1 << 31), EBADSHAPE),
           (dict(beta1=1.0), EBADSHAPE), (dict(beta1=float("nan")), EBADSHAPE), (dict(beta2=-0.1), EBADSHAPE), (dict(eps=-1e-8), EBADSHAPE),
           (dict(eps=float("inf")), EBADSHAPE), (dict(weight_decay=float("inf")), EBADSHAPE), (dict(lr=float("nan")), EBADSHAPE),
           (one(d=5), EBADDTYPE), (one(e=2), EBADDTYPE), (one(n=-1), EBADSHAPE), (one(n=513), EBADSHAPE), (one(s=64), EBADSHAPE),
           (one(s=-128), EBADSHAPE), (one(s=1 << 50), EBADSHAPE), (one(p=0), ENULL), (one(g=0), ENULL), (dict(tensors=None), ENULL),
           (dict(m=None), ENULL), (dict(v=None), ENULL), (one(p=P[0] + 2), EALIGN), (one(g=P[1] + 1), EALIGN), (one(c=P[10] + 1), EALIGN),
           (dict(m=P[5] + 8), EALIGN), (dict(v=P[6] + 4), EALIGN), (dict(grad_scale=P[9] + 2), EALIGN), (dict(lr_at=P[10] + 2), EALIGN),
           (dict(step_at=P[10] + 4), EALIGN), (one(p=P[1]), EOVERLAP), (one(p=P[2] + 596), EOVERLAP), (one(p=P[3]), EOVERLAP),
           (one(p=P[5]), EOVERLAP), (one(p=P[6] + 400), EOVERLAP), (one(c=P[0]), EOVERLAP), (one(s=128), EOVERLAP), (dict(v=P[5]), EOVERLAP),
           (dict(lr_at=P[0]), EOVERLAP), (dict(step_at=P[5]), EOVERLAP), (dict(grad_scale=P[6]), EOVERLAP),
           (one(g=P[3]), ECUDA), (dict(count=0, tensors=None), OK), (dict(tensors=tensors((0, 0, 0, 0, 0, F32, F32)), count=1), OK),
           (dict(step_at=P[10], step=0, lr_at=P[11], lr=float("nan"), grad_scale=None), ECUDA)] +
          ([(dict(m_scale=None), ENULL), (dict(v_scale=None), ENULL), (dict(m_scale=P[0]), EOVERLAP), (dict(v_scale=P[7] + 8), EOVERLAP)]
           if bits == 8 else [(dict(m_scale=None, v_scale=None), ECUDA)]))
many = [((P[0] + 4096 * i), P[1] + 4096 * i, 0, 1000, 1024 * i, F32, F32) for i in range(512)]
args = dict(tensors=tensors(*many), count=512, bits=32, m=P[5], v=P[6], m_scale=None, v_scale=None, total=512 * 1024, step=3, step_at=None,
            lr=1e-3, lr_at=None, beta1=0.0, beta2=0.0, eps=0.0, weight_decay=0.0, grad_scale=None, seed=0, stream=None)
entry("mxq_adamw", args, [(dict(tensors=tensors(*many[:-1], (P[0] + 4, P[2], 0, 1000, 1024 * 511, F32, F32))), EOVERLAP)])

def equal(what, got, want):
    if got != want:
        bad.append((what, got, want))
equal("workspace", L.mxq_moe_linear_backward_workspace(512, 256), 4 * 256 * 4)
for args in ((-128, 128), (100, 128), (128, 100), (FAR, 128)):
    equal(("workspace", args), L.mxq_moe_linear_backward_workspace(*args), EBADSHAPE)
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
    x, q, s = torch.zeros(128, 128), torch.zeros(128, 128, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    for call in (lambda: mxq.moe_route_groups(x, 2), lambda: mxq.moe_linear(q, s, q, s), lambda: mxq.moe_linear_backward(x, x),
                 lambda: mxq.moe_weight_gradient(q, s, q, s),
                 lambda: mxq.adamw_step([x], [x], mxq.Moments(torch.zeros(128 * 128), torch.zeros(128 * 128), None, None), 1, lr=0.1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_moments_of_a_list_begin_at_multiples_of_128():
    from mx_block_quantization_gb300 import training
    assert training._moment_starts([]) == ([], 0)
    assert training._moment_starts([1, 128, 129, 0, 5]) == ([0, 128, 256, 512, 512], 640)
    params = [torch.zeros(3, 50), torch.zeros(7)]
    for bits, kind in ((32, torch.float32), (8, torch.uint8)):
        m = training.adamw_moments(params, bits)
        assert m.m.dtype == kind and m.m.shape == m.v.shape == (384,)
        assert (m.m_scale is None) == (bits == 32) and (bits == 32 or m.m_scale.shape == m.v_scale.shape == (12,))
    with pytest.raises(ValueError, match="bits"):
        training.adamw_moments(params, 16)


def test_arguments_that_may_lie_on_the_device(monkeypatch):
    from mx_block_quantization_gb300 import training
    monkeypatch.setattr(training, "_flat", lambda t, name, dtype, shape, device: (name, dtype, shape, device))
    assert training._scalar(0.25, "lr", torch.float32, "there") == (0.25, None)
    assert training._scalar(torch.ones(()), "lr", torch.float32, "there") == (0, ("lr", torch.float32, (), "there"))


def test_the_mixing_of_the_rounding_spreads_its_bits():
    """Neighbouring places and steps: every one of the 32 bits is set in half of 2^16
    numbers (five deviations, 2.5 / 2^8), and differs in half of neighbours'."""
    import numpy as np
    sys.path.insert(0, ROOT)
    from tests.test_gpu_adamw import random_bits
    at = np.arange(1 << 16, dtype=np.int64)
    for seed, t, start in ((0, 1, 0), (1 << 40, 2, 1 << 33), (12345, 1000, 77)):
        a, b, c = random_bits(seed, t, at + start), random_bits(seed, t, at + start + 1), random_bits(seed, t + 1, at + start)
        for bits in (a, a ^ b, a ^ c):
            share = [(bits >> np.uint32(i) & np.uint32(1)).mean() for i in range(32)]
            assert max(abs(s - 0.5) for s in share) < 5 * 0.5 / 2**8
        low, high = (a & 0xFFFF) / 65536.0, (a >> 16) / 65536.0
        assert abs(np.corrcoef(low, high)[0, 1]) < 5 / 2**8
