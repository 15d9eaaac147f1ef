"""CPU checks of the FP8 entry points: workspace sizes and every refusal,
before any launch (none of these calls touches a GPU)."""
import ctypes

import pytest
import torch

FAKE = 0x100000   # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def hdq():
    from bit_quantized_video_amd import hdq as H
    return H


def test_workspace(hdq):
    f = hdq.fp8_linear_workspace_bytes
    assert f(0, 128, 16) == 0 and f(8, 12, 16) == 0 and f(8, 128, 0) == 0 and f(8, 128, 16, hdq.DTYPE_I32) == 0
    assert f(8, hdq.FP8_MAX_COLS + 8, 16) == 0
    assert f(1, 16384, 512) == 0 and f(16, 1024, 512) == 0          # quantized within the product's kernel
    assert f(1, 16512, 512) > 0 and f(17, 128, 512) > 0
    M, K = 1000, 1000
    assert f(M, K, 512) >= M * 1024 + 4 * M * 8       # codes and scales


def test_quantize_refusals(hdq):
    def q(x=FAKE, rows=4, cols=64, hb=16, layout=0, codes=FAKE, scale=FAKE):
        t = hdq.Fp8TensorDesc(9, 9, 9, 9, codes, scale)
        st = hdq.lib.hdq_fp8_quantize(x, rows, cols, hb, layout, ctypes.byref(t), None)
        assert (t.layout, t.had_block, t.rows, t.cols) == (9, 9, 9, 9)   # a refused call writes nothing
        return st
    assert q(x=None) == hdq.ERR_INVALID
    assert q(layout=2) == hdq.ERR_INVALID and q(layout=-1) == hdq.ERR_INVALID
    assert q(codes=None) == hdq.ERR_INVALID and q(scale=None) == hdq.ERR_INVALID
    assert hdq.lib.hdq_fp8_quantize(FAKE, 4, 64, 16, 0, None, None) == hdq.ERR_INVALID
    for kw in (dict(rows=0), dict(rows=-1), dict(rows=hdq.FP8_MAX_ROWS + 1), dict(cols=0), dict(cols=60), dict(cols=72),
               dict(hb=0), dict(hb=12), dict(hb=256), dict(cols=hdq.FP8_MAX_COLS + 128), dict(x=FAKE + 2),
               dict(codes=FAKE + 8), dict(scale=FAKE + 2)):
        assert q(**kw) == hdq.ERR_SHAPE, kw


def test_linear_refusals(hdq):
    L = hdq.lib
    need = hdq.fp8_linear_workspace_bytes(300, 512, 512)
    assert need > 0
    ok_w = dict(layout=1, hb=16, rows=512, cols=512, codes=FAKE, scale=FAKE)
    ok_x = dict(layout=0, hb=16, rows=300, cols=512, codes=FAKE, scale=FAKE)
    T = lambda d: hdq.Fp8TensorDesc(d["layout"], d["hb"], d["rows"], d["cols"], d["codes"], d["scale"])

    def lin(x=FAKE, xq=None, M=300, K=512, w=ok_w, y=FAKE, dt=1, ws=FAKE, wsb=need):
        return L.hdq_fp8_linear(x, ctypes.byref(T(xq)) if xq else None, M, K, ctypes.byref(T(w)) if w else None, y, dt,
                                ws, wsb, None)
    assert lin(w=None) == hdq.ERR_INVALID and lin(y=None) == hdq.ERR_INVALID and lin(x=None) == hdq.ERR_INVALID
    assert lin(dt=2) == hdq.ERR_UNSUPPORTED and lin(dt=7) == hdq.ERR_UNSUPPORTED
    for kw in (dict(M=0), dict(M=hdq.FP8_MAX_ROWS + 1), dict(K=0), dict(K=504), dict(K=256), dict(x=FAKE + 2), dict(y=FAKE + 4)):
        assert lin(**kw) == hdq.ERR_SHAPE, kw
    assert lin(w=dict(ok_w, layout=0)) == hdq.ERR_UNSUPPORTED
    assert lin(w=dict(ok_w, rows=0)) == hdq.ERR_SHAPE and lin(w=dict(ok_w, rows=hdq.FP8_MAX_ROWS + 1)) == hdq.ERR_SHAPE
    assert lin(w=dict(ok_w, hb=3)) == hdq.ERR_SHAPE
    assert lin(w=dict(ok_w, codes=None)) == hdq.ERR_INVALID and lin(w=dict(ok_w, scale=None)) == hdq.ERR_INVALID
    assert lin(w=dict(ok_w, codes=FAKE + 4)) == hdq.ERR_SHAPE
    assert lin(xq=dict(ok_x, layout=1)) == hdq.ERR_UNSUPPORTED
    assert lin(xq=dict(ok_x, rows=299)) == hdq.ERR_SHAPE
    assert lin(xq=dict(ok_x, hb=32)) == hdq.ERR_SHAPE            # another rotation than the weights'
    assert lin(xq=dict(ok_x, scale=None)) == hdq.ERR_INVALID
    assert lin(ws=None) == hdq.ERR_WORKSPACE and lin(wsb=need - 1) == hdq.ERR_WORKSPACE
    assert lin(ws=FAKE + 4) == hdq.ERR_SHAPE


def test_binding_refusals(hdq):
    with pytest.raises(ValueError):
        hdq.Fp8Tensor(4, 128, layout=5, device="cpu")
    with pytest.raises(ValueError):
        hdq.Fp8Tensor(4, 100, codes=torch.zeros(4, 100, dtype=torch.uint8))           # rows are 128 bytes
    with pytest.raises(ValueError):
        hdq.Fp8Tensor(4, 100, codes=torch.zeros(4, 128, dtype=torch.int8))
    with pytest.raises(ValueError):
        hdq.Fp8Tensor(4, 300, codes=torch.zeros(4, 384, dtype=torch.uint8), scale=torch.zeros(4, 3))  # [kb, rows]
    with pytest.raises(ValueError):
        hdq.fp8_quantize(torch.zeros(4, 128, dtype=torch.bfloat16), 1)                # not on a GPU
    with pytest.raises(ValueError):                                                   # codes in host memory
        hdq.fp8_linear(None, hdq.Fp8Tensor(16, 128, 1, hdq.FP8_BLOCKS, "cpu"), xq=hdq.Fp8Tensor(4, 128, 1, device="cpu"))
    t = hdq.Fp8Tensor(130, 300, 4, hdq.FP8_BLOCKS, "cpu")
    assert t.codes.shape == (130, 384) and t.scale.shape == (2, 3)
    assert hdq.Fp8Tensor(130, 300, 4, hdq.FP8_ROWS, "cpu").scale.shape == (3, 130)


def test_binding_scratch(hdq):
    """A caller's workspace is used when it fits and refused when it is strided."""
    dev = torch.device("cpu")
    assert hdq._scratch(None, 0, dev) == (None, None, 0)
    ws = torch.zeros(100, dtype=torch.int32)
    t, p, n = hdq._scratch(ws, 400, dev)
    assert t is ws and p == ws.data_ptr() and n == 400
    t, p, n = hdq._scratch(ws, 401, dev)
    assert t is not ws and n == 401 and t.numel() == 401
    with pytest.raises(ValueError):
        hdq._scratch(torch.zeros(100, 2, dtype=torch.uint8)[:, 0], 10, dev)
    with pytest.raises(ValueError):
        hdq._scratch(ws, 10, torch.device("meta"))


def test_binding_falls_back_to_public_torch_calls(hdq):
    public = lambda: 7
    assert hdq._torch_call("_no_such_binding", public) is public
    assert hdq._torch_call("_cuda_getDevice", public) is getattr(torch._C, "_cuda_getDevice", public)


def test_struct_matches_header(hdq, tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("gcc not found")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = [f[0] for f in hdq.Fp8TensorDesc._fields_]
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "hdq.h"\nint main(void) {\n'
                   'printf("%zu\\n", sizeof(hdq_fp8_tensor));\n' +
                   "".join(f'printf("%zu\\n", offsetof(hdq_fp8_tensor, {n}));\n' for n in names) + "return 0; }\n")
    exe = tmp_path / "l"
    subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [ctypes.sizeof(hdq.Fp8TensorDesc)] + [getattr(hdq.Fp8TensorDesc, n).offset for n in names]
