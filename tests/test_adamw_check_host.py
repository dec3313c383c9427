"""mxq_adamw_check on the host: lists longer than one launch takes, over fake addresses (it
looks at numbers alone)."""
import ctypes

import pytest

import mx_block_quantization_gb300 as mxq
from mx_block_quantization_gb300 import BF16, EALIGN, EBADDTYPE, EBADSHAPE, ENULL, EOVERLAP, F32, OK

P = [(i + 1) << 40 for i in range(8)]
COUNT = 1300


@pytest.fixture(scope="module")
def check():
    if not mxq.LIB_PATH.exists():
        import __graft_entry__
        __graft_entry__.build()
    L = mxq.lib()

    def call(change=None, **new):
        """The list with entry i replaced by change[i]."""
        table = []
        for i in range(COUNT):
            one = dict(p=P[0] + 4096 * i, g=P[1] + 4096 * i, c=0, n=1000, s=1024 * i, d=F32, e=F32)
            one.update((change or {}).get(i, {}))
            table += [one["p"], one["g"], one["c"], one["n"], one["s"], one["d"] | one["e"] << 32]
        args = dict(tensors=(ctypes.c_int64 * len(table))(*table), count=COUNT, bits=32, m=P[2], v=P[3], m_scale=None, v_scale=None,
                    total=1024 * COUNT, step_at=None, lr_at=None, grad_scale=None)
        return L.mxq_adamw_check(*{**args, **new}.values())
    return call


@pytest.mark.parametrize("bits", [32, 8])
def test_faults_anywhere_in_a_long_list(check, bits):
    how = dict(bits=bits, **(dict(m_scale=P[4], v_scale=P[5]) if bits == 8 else {}))
    assert check(**how) == OK
    for i in (0, 511, 512, 1299):
        for new, want in ((dict(d=9), EBADDTYPE), (dict(e=9), EBADDTYPE), (dict(n=-1), EBADSHAPE), (dict(s=100), EBADSHAPE),
                          (dict(s=1024 * COUNT - 896), EBADSHAPE), (dict(p=0), ENULL), (dict(g=0), ENULL),
                          (dict(p=P[6] + 2), EALIGN), (dict(g=P[6] + 1), EALIGN), (dict(c=P[6] + 1), EALIGN),
                          (dict(p=P[0] + 4096 * 700 + 3996), EOVERLAP), (dict(p=P[1] + 4096 * 3), EOVERLAP),
                          (dict(g=P[0] + 4096 * 3), EOVERLAP), (dict(c=P[0] + 4096 * 900), EOVERLAP), (dict(c=P[2] + 64), EOVERLAP),
                          (dict(p=P[3] + 400), EOVERLAP), (dict(s=1024 * 700), EOVERLAP),
                          (dict(g=P[1] + 4096 * 3), OK), (dict(n=0, p=0, g=0), OK), (dict(p=P[6] + 2, d=BF16), OK)):
            if i == 0 and want == EOVERLAP and new.get("s"):
                new = dict(s=1024)
            assert check({i: new}, **how) == want, (i, new)


def test_arguments_of_the_call(check):
    for new, want in ((dict(bits=16), EBADDTYPE), (dict(count=-1), EBADSHAPE), (dict(count=(1 << 24) + 1), EBADSHAPE),
                      (dict(total=100), EBADSHAPE), (dict(total=-128), EBADSHAPE), (dict(total=1 << 45), EBADSHAPE),
                      (dict(tensors=None), ENULL), (dict(m=None), ENULL), (dict(v=None), ENULL), (dict(bits=8), ENULL),
                      (dict(m=P[2] + 8), EALIGN), (dict(v=P[3] + 8), EALIGN), (dict(lr_at=P[6] + 2), EALIGN), (dict(step_at=P[6] + 4), EALIGN),
                      (dict(grad_scale=P[6] + 1), EALIGN), (dict(v=P[2]), EOVERLAP), (dict(lr_at=P[0]), EOVERLAP),
                      (dict(step_at=P[3]), EOVERLAP), (dict(grad_scale=P[2]), EOVERLAP), (dict(grad_scale=P[1]), OK),
                      (dict(count=0, tensors=None), OK)):
        assert check(**new) == want, new
