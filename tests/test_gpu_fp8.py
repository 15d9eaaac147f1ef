"""FP8 block-128 quantization and linear layers on the GPU against float32
(coding, equal) and float64 (products) references."""
import math

import pytest
import torch

import fp8_ref as R

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from bit_quantized_video_amd import hdq  # noqa: E402

DEV = torch.device("cuda:0")
LAYOUT = {"rows": hdq.FP8_ROWS, "blocks": hdq.FP8_BLOCKS}


def activations(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.5 * torch.randn(rows, 1, generator=g))
    x[:, torch.randperm(cols, generator=g)[:max(1, cols // 100)]] *= 20.0
    return x.to(torch.bfloat16)


def code_values(codes):
    return codes.view(torch.float8_e4m3fn).float().cpu()


def check_quantized(q, x, had, layout):
    codes, scale = R.quantize(R.rotate(x, had), layout)
    assert q.codes.shape == codes.shape and q.scale.shape == scale.shape
    torch.testing.assert_close(q.scale.cpu(), scale, rtol=0, atol=0, equal_nan=True)
    assert torch.equal(code_values(q.codes), codes)
    assert int(q.codes[:, x.shape[1]:].sum()) == 0


@pytest.mark.parametrize("layout", ["rows", "blocks"])
@pytest.mark.parametrize("rows,cols,had", [
    (1, 8, 1), (1, 8, 8), (3, 16, 2), (5, 24, 4), (17, 120, 8), (16, 128, 128), (129, 128, 64), (40, 136, 8),
    (33, 384, 128), (130, 1000, 8), (257, 1920, 128), (64, 2080, 32), (31, 656, 16), (300, 520, 1), (5, 192, 64), (140, 320, 64)])
def test_quantize_matches_reference(rows, cols, had, layout):
    x = activations(rows, cols, 7 * rows + cols)
    check_quantized(hdq.fp8_quantize(x.to(DEV), had, LAYOUT[layout]), x, had, layout)


@pytest.mark.parametrize("layout", ["rows", "blocks"])
def test_quantize_value_is_within_half_a_step(layout):
    """|code * scale - y| is at most half an E4M3 step: 2^-4 of the value, or
    2^-10 of the scale below the normal range, plus the float32 roundings of
    the rotation (7 additions, one product) and of the two scale factors."""
    rows, cols, had = 150, 640, 128
    x = activations(rows, cols, 5)
    h = torch.ones(1, 1, dtype=torch.float64)
    while h.shape[0] < had:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    y = (x.double().view(rows, -1, had) @ (h / math.sqrt(had))).view(rows, cols)
    mag = (x.double().abs().view(rows, -1, had).sum(2, keepdim=True) / math.sqrt(had)).expand(-1, -1, had).reshape(rows, cols)
    q = hdq.fp8_quantize(x.to(DEV), had, LAYOUT[layout])
    s = R.scale_per_element(q.scale.cpu(), layout, rows)
    v = code_values(q.codes).double() * s
    tol = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s[:, :cols]) * (1 + 2.0 ** -20) + 10 * 2.0 ** -24 * mag
    assert bool(((v[:, :cols] - y).abs() <= tol).all())


@pytest.mark.parametrize("layout", ["rows", "blocks"])
def test_quantize_zero_tiny_and_nonfinite_blocks(layout):
    x = activations(260, 512, 3)
    x[0:128, 128:256] = 0
    x[128:256, 0:128] = 2.0 ** -110          # below the smallest scaled block
    x[200, 300] = math.inf
    x[5, 400] = math.nan
    check_quantized(hdq.fp8_quantize(x.to(DEV), 1, LAYOUT[layout]), x, 1, layout)
    q = hdq.fp8_quantize(x.to(DEV), 32, LAYOUT[layout])
    codes, scale = R.quantize(R.rotate(x, 32), layout)
    torch.testing.assert_close(q.scale.cpu(), scale, rtol=0, atol=0, equal_nan=True)
    assert torch.equal(code_values(q.codes), codes)


def make_linear(M, K, N, had, seed=0):
    x = activations(M, K, seed + M + K)
    w = (0.02 * torch.randn(N, K, generator=torch.Generator().manual_seed(seed + N))).to(torch.bfloat16)
    xq = hdq.fp8_quantize(x.to(DEV), had)
    wq = hdq.fp8_quantize(w.to(DEV), had, hdq.FP8_BLOCKS)
    return x.to(DEV), xq, wq


def check_linear(y, xq, wq):
    ref, tol = R.linear(code_values(xq.codes), xq.scale.cpu(), code_values(wq.codes), wq.scale.cpu(),
                        y.dtype == torch.bfloat16)
    err = (y.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), f"worst error {float((err / tol.clamp_min(1e-300)).max())} of the bound"


SHAPES = [(1, 8, 1, 8), (1, 128, 16, 128), (1, 1920, 577, 128), (2, 1000, 130, 8), (7, 264, 64, 1), (16, 4096, 96, 64),
          (17, 384, 100, 32), (33, 128, 257, 128), (65, 640, 33, 128), (64, 1928, 200, 8), (130, 776, 129, 8),
          (226, 2048, 192, 128), (300, 256, 520, 64), (513, 512, 384, 128), (700, 1160, 301, 8), (1000, 256, 1030, 128),
          (2100, 392, 2050, 8), (4200, 128, 1030, 128), (2304, 640, 4096, 64), (16500, 264, 260, 8),
          (4100, 264, 4200, 8), (4353, 136, 4104, 8), (33, 4224, 100, 128), (1100, 1032, 1000, 8), (20, 40, 6000, 8),
          (1, 12288, 40, 128), (1, 16384, 20, 2), (1, 16512, 20, 128), (4, 4096, 50, 4), (5, 4096, 50, 16), (16, 1024, 33, 32),
          (16, 1032, 33, 8), (3, 24, 3, 1), (1351, 520, 3900, 8), (1700, 264, 2001, 8),
          (3000, 264, 4101, 8), (1290, 128, 1290, 64)]


@pytest.mark.parametrize("y_dtype", [hdq.DTYPE_BF16, hdq.DTYPE_F32])
@pytest.mark.parametrize("M,K,N,had", SHAPES)
def test_linear_matches_reference(M, K, N, had, y_dtype):
    x, xq, wq = make_linear(M, K, N, had)
    y = hdq.fp8_linear(None, wq, xq=xq, y_dtype=y_dtype)
    check_linear(y, xq, wq)
    # quantizing within the call gives the same codes, so the same output
    assert torch.equal(hdq.fp8_linear(x, wq, y_dtype=y_dtype), y)


@pytest.mark.parametrize("y_dtype", [hdq.DTYPE_BF16, hdq.DTYPE_F32])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_linear_nonfinite_and_zero_rows(M, y_dtype):
    K, N = 384, 200
    x = activations(M, K, 9)
    x[M - 1, 130] = math.nan
    if M > 2:
        x[0] = 0
        x[1, 0] = -math.inf
    w = (0.02 * torch.randn(N, K, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16)
    wq = hdq.fp8_quantize(w.to(DEV), 64, hdq.FP8_BLOCKS)
    y = hdq.fp8_linear(x.to(DEV), wq, y_dtype=y_dtype).float().cpu()
    assert bool(torch.isnan(y[M - 1]).all())
    if M > 2:
        assert bool(torch.isnan(y[1]).all()) and bool((y[0] == 0).all())
        assert bool(torch.isfinite(y[2:M - 1]).all())
    wbad = w.clone()
    wbad[130, 5] = math.nan      # the second block of 128 features
    wq = hdq.fp8_quantize(wbad.to(DEV), 64, hdq.FP8_BLOCKS)
    y = hdq.fp8_linear(activations(M, K, 9).to(DEV), wq, y_dtype=y_dtype).float().cpu()
    assert bool(torch.isfinite(y[:, :128]).all()) and bool(torch.isnan(y[:, 128:]).all())


@pytest.mark.parametrize("y_dtype", [hdq.DTYPE_BF16, hdq.DTYPE_F32])
@pytest.mark.parametrize("M,K,N", [(1, 256, 5), (19, 256, 131), (260, 512, 259)])
def test_linear_writes_its_output_only(M, K, N, y_dtype):
    dt = torch.float32 if y_dtype == hdq.DTYPE_F32 else torch.bfloat16
    x, xq, wq = make_linear(M, K, N, 128)
    pad = 4096
    buf = torch.full((M * N + 2 * pad,), -7.0, dtype=dt, device=DEV)
    y = buf[pad:pad + M * N].view(M, N)
    n = hdq.fp8_linear_workspace_bytes(M, K, N, y_dtype)
    ws = torch.full((n + 512,), 77, dtype=torch.uint8, device=DEV)
    hdq.fp8_linear(x, wq, y=y, y_dtype=y_dtype, ws=ws[:n])
    assert torch.equal(y, hdq.fp8_linear(None, wq, xq=xq, y_dtype=y_dtype))
    assert bool((buf[:pad] == -7).all()) and bool((buf[pad + M * N:] == -7).all()) and bool((ws[n:] == 77).all())


def test_checkpoint_codes_are_used_as_given():
    """Weights that come as float8 codes and block scales need no quantization here."""
    M, K, N = 20, 256, 192
    x, xq, wq = make_linear(M, K, N, 1)
    w = hdq.Fp8Tensor(N, K, 1, hdq.FP8_BLOCKS, codes=wq.codes.view(torch.float8_e4m3fn), scale=wq.scale)
    assert torch.equal(hdq.fp8_linear(x, w), hdq.fp8_linear(x, wq))


def test_linear_on_another_stream_and_in_a_graph():
    M, K, N = 150, 640, 320
    x, xq, wq = make_linear(M, K, N, 128)
    want = hdq.fp8_linear(x, wq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = hdq.fp8_linear(x, wq, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    static = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = hdq.fp8_quantize(static, 128)
        yg = hdq.fp8_linear(None, wq, xq=q)
        yx = hdq.fp8_linear(static, wq)
    for seed in range(4):
        xi = activations(M, K, 100 + seed).to(DEV)
        static.copy_(xi)
        g.replay()
        torch.cuda.synchronize()
        eager = hdq.fp8_linear(xi, wq)
        assert torch.equal(yg, eager) and torch.equal(yx, eager)


def test_offsets_past_32_bits():
    """More than 2^32 code bytes of activations: the last rows are those of a small call."""
    K, N, M = 16384, 64, 270000
    wq = hdq.fp8_quantize((0.02 * torch.randn(N, K, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).to(DEV),
                          128, hdq.FP8_BLOCKS)
    tail = activations(200, K, 2).to(DEV)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    x[-200:] = tail
    xq = hdq.fp8_quantize(x, 128)
    del x
    tq = hdq.fp8_quantize(tail, 128)
    assert torch.equal(xq.codes[-200:], tq.codes) and torch.equal(xq.scale[:, -200:], tq.scale)
    for dt in (hdq.DTYPE_BF16, hdq.DTYPE_F32):
        y = hdq.fp8_linear(None, wq, xq=xq, y_dtype=dt)
        assert bool((y[:-200] == 0).all())
        check_linear(y[-200:], tq, wq)


def test_quantize_more_rows_than_one_grid_row():
    """16 threads a row pass 2^32: repeated rows give repeated codes."""
    S, reps, K = 4096, 65537, 8
    x = activations(S, K, 3).to(DEV)
    q, small = hdq.fp8_quantize(x.repeat(reps, 1), 8), hdq.fp8_quantize(x, 8)
    codes = q.codes.view(reps, S, 128)
    for i in range(0, reps, 4096):
        assert bool((codes[i:i + 4096] == small.codes).all())
    assert bool((codes[-1] == small.codes).all()) and bool((q.scale.view(reps, S) == small.scale).all())


def test_linear_more_features_than_one_grid_row():
    """One token, 32 threads a feature past 2^32: the last features are a small layer's."""
    N, tail = 1 << 27, 40
    x = activations(1, 8, 4).to(DEV)
    small = hdq.fp8_quantize((0.02 * torch.randn(tail, 8, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).to(DEV),
                             8, hdq.FP8_BLOCKS)
    codes = torch.zeros(N + tail, 128, dtype=torch.uint8, device=DEV)
    scale = torch.ones(N // 128 + 1, 1, device=DEV)
    codes[N:], scale[-1] = small.codes, small.scale[0]
    w = hdq.Fp8Tensor(N + tail, 8, 8, hdq.FP8_BLOCKS, codes=codes, scale=scale)
    xq = hdq.fp8_quantize(x, 8)
    for y in (hdq.fp8_linear(x, w), hdq.fp8_linear(None, w, xq=xq)):
        assert torch.equal(y[:, N:], hdq.fp8_linear(x, small)) and bool((y[:, :N] == 0).all())
