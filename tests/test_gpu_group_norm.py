"""Channels-last group norm on the GPU against float64, and its FP8 form
against the quantizer's reference and into a linear layer."""
import math

import pytest
import torch

import fp8_ref as R

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from bit_quantized_video_amd import hdq  # noqa: E402

DEV = torch.device("cuda:0")
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def inputs(n, L, C, dtype, seed, offset=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, L, C, generator=g) * (0.5 + torch.rand(C, generator=g)) + offset * torch.randn(n, 1, C, generator=g)
    return x.to(dtype), 1 + 0.2 * torch.randn(C, generator=g), 0.2 * torch.randn(C, generator=g)


def reference(x, groups, w, b, eps, silu):
    """(y in float64, bound before the output's rounding).

    With m = max|x| of a group, std its deviation and u = 2^-24: the thread
    sums lose at most about 2 (rows per thread, < 512) u of a deviation and
    the mean is rounded once, so mean is within 2 u m + 2^-14 std / 16 and the
    relative error of rstd within 2^-14; the bound takes 2 u m / std + 2^-14
    on x_hat = (x - mean) rstd, and 4 u for the last operations.  In practice
    errors are near u: a second, statistical check asks for 2^-20 in the
    2-norm.  SiLU's derivative is below 1.1, its own operations 8 u."""
    n, L, C = x.shape
    v = x.double().view(n, L, groups, C // groups)
    var, mean = torch.var_mean(v, (1, 3), correction=0, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xh = ((v - mean) * rstd).reshape(n, L, C)
    w, b = (torch.ones(C) if w is None else w).double(), (torch.zeros(C) if b is None else b).double()
    t = xh * w + b
    amp = (v.abs().amax((1, 3), keepdim=True) * rstd).expand_as(v).reshape(n, L, C)
    tol = (2 * 2.0 ** -24 * amp + 2.0 ** -14 * (xh.abs() + 1)) * w.abs() + 4 * 2.0 ** -24 * (t.abs() + b.abs())
    if silu:
        t = t * torch.sigmoid(t)
        tol = 1.1 * tol + 8 * 2.0 ** -24 * t.abs()
    return t, tol


def check(y, x, groups, w, b, eps=1e-5, silu=False, norm=True):
    ref, tol = reference(x, groups, w, b, eps, silu)
    half = HALF[y.dtype]
    err = (y.cpu().double() - ref).abs()
    assert bool((err <= tol * (1 + half) + half * ref.abs()).all())
    if norm and float(ref.norm()) > 0:
        assert float(err.norm() / ref.norm()) <= half + 2.0 ** -20


SHAPES = [(1, 1, 1, 1), (2, 1, 8, 4), (1, 2, 32, 32), (3, 7, 58, 1), (2, 77, 300, 30), (1, 1000, 64, 8),
          (2, 225, 320, 32), (1, 513, 1280, 32), (5, 130, 8, 2), (1, 9, 4104, 27), (1, 40, 8192, 32), (2, 33, 8191, 1),
          (13, 90, 512, 32), (40, 3, 96, 32), (1, 20011, 136, 17),
          (2, 700, 256, 32), (1, 1300, 64, 4), (9, 2500, 512, 32), (300, 150, 44, 11), (1, 1021, 24, 8),
          (1, 984, 537, 1), (1, 5400, 64, 64), (2, 2001, 100, 25), (1, 800, 1537, 1)]


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,L,C,G", SHAPES)
def test_group_norm_matches_reference(n, L, C, G, dtype, silu):
    x, w, b = inputs(n, L, C, dtype, n + L + C)
    y = hdq.group_norm(x.to(DEV), G, w.to(DEV), b.to(DEV), 1e-5, hdq.ACT_SILU if silu else hdq.ACT_NONE)
    assert y.dtype == dtype and y.shape == x.shape
    check(y, x, G, w, b, silu=silu, norm=L * (C // G) > 16)


@pytest.mark.parametrize("xt,yt", [(torch.bfloat16, hdq.DTYPE_F32), (torch.float32, hdq.DTYPE_BF16)])
@pytest.mark.parametrize("C", [64, 60, 63])
def test_other_output_type_and_no_affine(C, xt, yt):
    x, w, b = inputs(2, 50, C, xt, C)
    y = hdq.group_norm(x.to(DEV), 3 if C == 63 else 4, y_dtype=yt, eps=1e-3)
    check(y, x, 3 if C == 63 else 4, None, None, eps=1e-3)
    y = hdq.group_norm(x.to(DEV), 1, w.to(DEV), y_dtype=yt)
    check(y, x, 1, w, None)


def test_large_mean_and_an_outlier_keep_their_digits():
    """A mean 2000 times the deviation, and one value 1e6 times it among many:
    the variance is summed about values near the data, not about zero."""
    n, L, C, G = 1, 30000, 32, 4
    g = torch.Generator().manual_seed(4)
    x = torch.randn(n, L, C, generator=g) + 2000.0
    y = hdq.group_norm(x.to(DEV), G, y_dtype=hdq.DTYPE_F32)
    v = x.double().view(n, L, G, C // G)
    var, mean = torch.var_mean(v, (1, 3), correction=0, keepdim=True)
    ref = ((v - mean) / torch.sqrt(var + 1e-5)).view(n, L, C)
    # the float32 mean is off by at most half a step of 2000: 2^-14 of a deviation
    assert float((y.cpu().double() - ref).abs().max()) <= 2.0 ** -14 + 2.0 ** -18
    x = torch.randn(n, L, C, generator=g)
    x[0, 0, 0] = 1e6
    y = hdq.group_norm(x.to(DEV), G)
    check(y, x, G, None, None)
    # the first row is the threads' own reference value: move the outlier
    x[0, 0, 0], x[0, 17003, 9] = 0.5, -1e6
    check(hdq.group_norm(x.to(DEV), G), x, G, None, None)


def test_constant_input_gives_the_bias():
    x = torch.full((2, 100, 64), 3.140625, dtype=torch.bfloat16)
    b = torch.linspace(-1, 1, 64)
    y = hdq.group_norm(x.to(DEV), 8, None, b.to(DEV), y_dtype=hdq.DTYPE_F32)
    assert torch.equal(y.cpu(), b.expand(2, 100, 64))


@pytest.mark.parametrize("L", [40, 3000])
def test_nonfinite_values_stay_in_their_group(L):
    x, w, b = inputs(3, L, 64, torch.float32, 1)
    x[0, 3, 20] = math.nan      # group 2 of 8
    x[1, 0, 0] = math.inf       # group 0
    y = hdq.group_norm(x.to(DEV), 8, w.to(DEV), b.to(DEV)).cpu()
    bad = torch.zeros(3, L, 64, dtype=torch.bool)
    bad[0, :, 16:24] = True
    bad[1, :, 0:8] = True
    assert bool(torch.isnan(y[bad]).all())
    ref, tol = reference(torch.where(bad, torch.zeros_like(x), x), 8, w, b, 1e-5, False)
    assert bool(((y.double() - ref).abs() <= tol + 2.0 ** -24 * ref.abs())[~bad].all())


@pytest.mark.parametrize("n,L,C,G", [(2, 50, 64, 8), (1, 9000, 64, 8)])
def test_in_place_and_guard_bytes(n, L, C, G):
    x, w, b = inputs(n, L, C, torch.bfloat16, 8)
    want = hdq.group_norm(x.to(DEV), G, w.to(DEV), b.to(DEV), act=hdq.ACT_SILU)
    buf = torch.full((x.numel() + 2048,), 9.0, dtype=torch.bfloat16, device=DEV)
    v = buf[1024:1024 + x.numel()].view(x.shape)
    v.copy_(x)
    need = hdq.group_norm_workspace_bytes(n, L, C, G)
    ws = torch.full((need + 256,), 5, dtype=torch.uint8, device=DEV)
    out = hdq.group_norm(v, G, w.to(DEV), b.to(DEV), act=hdq.ACT_SILU, y=v, ws=ws[:need])
    assert out is v and torch.equal(v, want)
    assert bool((buf[:1024] == 9).all()) and bool((buf[1024 + x.numel():] == 9).all()) and bool((ws[need:] == 5).all())


FP8_SHAPES = [(1, 1, 8, 1, 8), (2, 5, 64, 8, 64), (1, 225, 320, 32, 64), (3, 37, 136, 17, 8), (1, 700, 1280, 32, 128),
              (13, 50, 512, 32, 128), (1, 3000, 64, 4, 1), (9, 2500, 512, 32, 16), (2, 18, 4104, 27, 2), (1, 5, 200, 5, 4),
              (1, 6, 160, 5, 32), (3, 170, 512, 32, 128), (2, 33, 504, 21, 8), (1, 1000, 40, 5, 4),
              (7, 16, 256, 256, 64), (5, 17, 264, 8, 1),
              (20, 225, 320, 32, 64), (300, 16, 128, 8, 128), (300, 17, 128, 8, 8), (1, 4097, 16, 4, 16),
              (1, 9000, 320, 32, 64), (2, 3000, 256, 16, 128)]


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,L,C,G,had", FP8_SHAPES)
def test_fp8_form_codes_the_norm(n, L, C, G, had, dtype, silu):
    """code * scale is the rotated norm within half an E4M3 step (2^-4 of the
    value, 2^-10 of the scale for small ones) plus the norm's own bound spread
    over its Hadamard block and the rotation's 8 roundings."""
    x, w, b = inputs(n, L, C, dtype, 3 * L + C)
    q = hdq.group_norm_fp8(x.to(DEV), G, w.to(DEV), b.to(DEV), act=hdq.ACT_SILU if silu else hdq.ACT_NONE, had_block=had)
    assert (q.rows, q.cols, q.had_block, q.layout) == (n * L, C, had, hdq.FP8_ROWS)
    t, tol = reference(x, G, w, b, 1e-5, silu)
    h = torch.ones(1, 1, dtype=torch.float64)
    while h.shape[0] < had:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    h = h / math.sqrt(had)
    spread = lambda v: (v.reshape(n * L, C // had, had).sum(2, keepdim=True) / math.sqrt(had)).expand(-1, -1, had).reshape(n * L, C)
    y = (t.view(n * L, C // had, had) @ h).view(n * L, C)
    s = R.scale_per_element(q.scale.cpu(), "rows", n * L)
    codes = q.codes.view(torch.float8_e4m3fn).float().cpu().double()
    assert int(q.codes[:, C:].sum()) == 0
    err = ((codes * s)[:, :C] - y).abs()
    slack = spread(tol) + 10 * 2.0 ** -24 * spread(t.abs())
    assert bool((err <= torch.maximum(2.0 ** -4 * (y.abs() + slack), 2.0 ** -10 * s[:, :C]) * (1 + 2.0 ** -20) + slack).all())
    # the scale is the block's largest value over 448
    ymax = R.block_view(y, "rows").abs().amax((1, 3))
    smax = R.block_view(slack.contiguous(), "rows").amax((1, 3))
    assert bool(((q.scale.cpu().t().double() * 448 - ymax).abs() <= smax + 3 * 2.0 ** -24 * ymax).all())


def test_norm_projection_chain_in_a_graph():
    """norm -> FP8 codes -> projection, as a decoder's attention block runs it:
    against the float64 product of the same codes, captured and replayed with
    eager work between the replays."""
    n, L, C, G, N, had = 3, 150, 320, 32, 200, 64
    x, w, b = (t.to(DEV) for t in inputs(n, L, C, torch.bfloat16, 1))
    wq = hdq.fp8_quantize((0.02 * torch.randn(N, C, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).to(DEV),
                          had, hdq.FP8_BLOCKS)

    def chain(v):
        q = hdq.group_norm_fp8(v, G, w, b, had_block=had)
        return q, hdq.fp8_linear(None, wq, xq=q)
    q, y = chain(x)
    ref, tol = R.linear(q.codes.view(torch.float8_e4m3fn).float().cpu(), q.scale.cpu(),
                        wq.codes.view(torch.float8_e4m3fn).float().cpu(), wq.scale.cpu(), True)
    assert bool(((y.cpu().double() - ref).abs() <= tol).all())
    static = x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain(static)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg, yg = chain(static)
        ng = hdq.group_norm(static, G, w, b, act=hdq.ACT_SILU)
    for seed in range(4):
        xi = inputs(n, L, C, torch.bfloat16, 50 + seed)[0].to(DEV)
        static.copy_(xi)
        g.replay()
        torch.cuda.synchronize()
        qe, ye = chain(xi)
        assert torch.equal(qg.codes, qe.codes) and torch.equal(qg.scale, qe.scale) and torch.equal(yg, ye)
        assert torch.equal(ng, hdq.group_norm(xi, G, w, b, act=hdq.ACT_SILU))


def test_group_norm_on_another_stream():
    x, w, b = (t.to(DEV) for t in inputs(2, 500, 64, torch.bfloat16, 1))
    want = hdq.group_norm(x, 8, w, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = hdq.group_norm(x, 8, w, b, stream=s)
    q = hdq.group_norm_fp8(x, 8, w, b, had_block=8, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    assert torch.equal(q.codes, hdq.group_norm_fp8(x, 8, w, b, had_block=8).codes)


def test_group_norm_past_32_bit_offsets():
    """More than 2^32 elements: the last sample is a small call's."""
    C, L, n = 256, 1 << 18, 68
    x = torch.zeros(n, L, C, dtype=torch.bfloat16, device=DEV)
    tail = inputs(1, L, C, torch.bfloat16, 6)[0].to(DEV)
    x[-1:] = tail
    y = hdq.group_norm(x, 32)
    want = hdq.group_norm(tail, 32)
    # other chunks of rows, so other float32 partial sums: at most one bf16 step apart
    d = (y[-1:].float() - want.float()).abs()
    assert bool((d <= 2.0 ** -7 * want.float().abs() + 2.0 ** -20).all())
    assert bool((y[:-1] == 0).all())


def test_more_samples_than_one_launch_takes():
    """256 threads a sample pass 2^32: repeated samples give repeated outputs."""
    S, reps, C, G = 4096, 4097, 8, 2
    x, w, b = (t.to(DEV) for t in inputs(S, 1, C, torch.bfloat16, 12))
    big = x.repeat(reps, 1, 1)
    y = hdq.group_norm(big, G, w, b)
    assert bool((y.view(reps, S, 1, C) == hdq.group_norm(x, G, w, b)).all())
    del y
    q, small = hdq.group_norm_fp8(big, G, w, b, had_block=8), hdq.group_norm_fp8(x, G, w, b, had_block=8)
    assert bool((q.codes.view(reps, S, 128) == small.codes).all()) and bool((q.scale.view(reps, S) == small.scale).all())


def test_fp8_rows_past_one_launch():
    """16 threads a row pass 2^32: rows of period 4096 give codes of that period,
    and those of a sample with the same statistics within one E4M3 step."""
    S, reps, C, G = 4096, 65537, 8, 2
    x, w, b = (t.to(DEV) for t in inputs(1, S, C, torch.bfloat16, 13, offset=0.0))
    q = hdq.group_norm_fp8(x.repeat(1, reps, 1), G, w, b)
    codes, scale = q.codes.view(reps, S, 128), q.scale.view(reps, S)
    for i in range(0, reps, 4096):
        assert bool((codes[i:i + 4096] == codes[0]).all())
    assert bool((codes[-1] == codes[0]).all()) and bool((scale == scale[0]).all())
    small = hdq.group_norm_fp8(x, G, w, b)
    value = lambda c, s: c.view(torch.float8_e4m3fn).float()[:, :C] * s.view(-1, 1)
    v, t = value(codes[0].contiguous(), scale[0]), value(small.codes, small.scale)
    # nearly equal inputs can fall to either side of a rounding border: one step
    step = torch.maximum(2.0 ** -3 * t.abs(), 2.0 ** -9 * small.scale.view(-1, 1))
    assert bool(((v - t).abs() <= step * (1 + 2.0 ** -10)).all())
