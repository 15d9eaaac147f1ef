"""CPU checks of the group-norm entry points: workspace sizes and every
refusal, before any launch."""
import ctypes
import math

import pytest
import torch

FAKE = 0x100000   # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def hdq():
    from bit_quantized_video_amd import hdq as H
    return H


def test_workspace(hdq):
    f = hdq.group_norm_workspace_bytes
    for bad in ((0, 5, 8, 2), (1, 0, 8, 2), (1, 5, 0, 1), (1, 5, 8, 3), (1, 5, 8, 0), (1, 5, 8200, 1),
                (1 << 20, 1 << 20, 8, 2)):
        assert f(*bad) == 0, bad
    assert f(1, 1, 1, 1) == 0                            # one launch needs none
    assert f(1, 1, 8, 1, True) == 0 and f(1, 225, 320, 32, True) == 0
    # with many samples of several workgroups each one launch would read them too often
    assert f(64, 225, 320, 32, True) >= 64 * 3 * 320 * 4 and f(1, 12288, 8, 2, True) > 0
    assert f(20000, 16, 512, 32, True) == 0
    assert f(13, 1350, 512, 32, True) >= 13 * 3 * 512 * 4   # coefficients of the two-launch FP8 form
    assert f(1, 100000, 256, 32) >= 3 * 256 * 4 + 32 * 16


def test_refusals(hdq):
    L = hdq.lib
    ws = 1 << 24

    def norm(fp8, x=FAKE, xt=1, n=2, length=50, C=64, G=8, w=FAKE, b=FAKE, eps=1e-5, act=0, y=FAKE, yt=1, had=8,
             ws=FAKE, wsb=ws):
        if not fp8:
            return L.hdq_group_norm(x, xt, n, length, C, G, w, b, eps, act, y, yt, ws, wsb, None)
        t = hdq.Fp8TensorDesc(9, 9, 9, 9, y, FAKE)
        st = L.hdq_group_norm_fp8(x, xt, n, length, C, G, w, b, eps, act, had, ctypes.byref(t), ws, wsb, None)
        assert (t.layout, t.had_block, t.rows, t.cols) == (9, 9, 9, 9)
        return st
    for fp8 in (False, True):
        assert norm(fp8, x=None) == hdq.ERR_INVALID and norm(fp8, y=None) == hdq.ERR_INVALID
        assert norm(fp8, act=2) == hdq.ERR_INVALID
        for eps in (-1e-6, math.nan, math.inf):
            assert norm(fp8, eps=eps) == hdq.ERR_INVALID
        assert norm(fp8, xt=2) == hdq.ERR_UNSUPPORTED
        for kw in (dict(n=0), dict(length=0), dict(length=-1), dict(C=0), dict(G=0), dict(G=7), dict(C=8256, G=8),
                   dict(n=1 << 16, length=1 << 15), dict(x=FAKE + 8), dict(y=FAKE + 8), dict(w=FAKE + 2)):
            assert norm(fp8, **kw) == hdq.ERR_SHAPE, (fp8, kw)
        need = hdq.group_norm_workspace_bytes(1, 100000, 64, 8, fp8)
        big = dict(n=1, length=100000)
        assert norm(fp8, ws=None, **big) == hdq.ERR_WORKSPACE and norm(fp8, wsb=need - 1, **big) == hdq.ERR_WORKSPACE
        assert norm(fp8, ws=FAKE + 8, **big) == hdq.ERR_SHAPE
    assert norm(False, yt=2) == hdq.ERR_UNSUPPORTED
    assert norm(False, xt=0, yt=1, y=FAKE) == hdq.ERR_SHAPE       # in place between types
    assert norm(True, C=60, G=4, had=4) == hdq.ERR_SHAPE          # no multiple of 8
    assert norm(True, had=128) == hdq.ERR_SHAPE and norm(True, had=3) == hdq.ERR_SHAPE
    assert L.hdq_group_norm_fp8(FAKE, 1, 2, 50, 64, 8, None, None, 1e-5, 0, 8, None, FAKE, ws, None) == hdq.ERR_INVALID


def test_binding_refusals(hdq):
    x = torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    for f in (hdq.group_norm, hdq.group_norm_fp8):
        with pytest.raises(ValueError):
            f(x, 8)                       # not on a GPU
