"""The group norm at the ends of its input range: long runs of rows on a large
mean, magnitudes up to the types' largest and, without eps, small ones."""
import math

import pytest
import torch

import fp8_ref as R

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from bit_quantized_video_amd import hdq  # noqa: E402

DEV = torch.device("cuda:0")
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def exact(x, groups, eps):
    """(normalized values, the largest |x| of their group times rstd) in float64; x [n, L, C]."""
    n, L, C = x.shape
    v = x.double().view(n, L, groups, C // groups)
    var, mean = torch.var_mean(v, (1, 3), correction=0, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    amp = (v.abs().amax((1, 3), keepdim=True) * rstd).expand_as(v)
    return ((v - mean) * rstd).reshape(n, L, C), amp.reshape(n, L, C)


def bound(ref, amp, dtype):
    """The kernel's error on |ref|, u = 2^-24.  A thread's mean of k <= 16 rows is
    their first one plus a float32 sum of differences: off by u max|x| (the last
    rounding) and 16 u of the rows' mean distance from the first, about two
    deviations over a group's threads.  Means are joined in float64 and rounded
    to float32 in a pair and at the end, u / 2 of max|x| each.  So the mean is
    off by 2 u max|x| + 32 u deviations.  Squared deviations: 2 u each for the
    difference, 16 u for the sum, 2 u for a pair's variance, so rstd 10 u of itself;
    four roundings follow (rstd, times the weight, the difference, the last
    multiply-add).  Then the output's rounding."""
    tol = 2 * U * amp + 32 * U * (ref.abs() + 1)
    return tol * (1 + HALF[dtype]) + HALF[dtype] * ref.abs()


def test_long_runs_keep_a_large_mean():
    """512 samples leave one workgroup a sample, 513 channels one thread a
    channel: 5000 rows of one thread, on a mean 2000 times the deviation."""
    n, L, C = 512, 5000, 513
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(n, L, C, generator=g, device=DEV).add_(2000.0)
    y = hdq.group_norm(x, C)
    for i in (0, 200, 511):
        ref, amp = exact(x[i:i + 1], C, 1e-5)
        err = (y[i:i + 1].double() - ref).abs()
        assert bool((err <= bound(ref, amp, torch.float32)).all()), float(err.max())


def test_a_group_per_channel_in_many_samples():
    """More than 2^26 groups, whose chunks are joined by a wave each (2^32 threads):
    repeated samples give repeated outputs, in place."""
    S, reps, L, C = 1024, 418, 513, 157
    assert S * reps * C > 1 << 26
    if torch.cuda.mem_get_info(DEV)[0] < 80 << 30:
        pytest.skip("needs 80 GB of free GPU memory")
    x = torch.randn(S, L, C, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    big = x.repeat(reps, 1, 1)
    hdq.group_norm(big, C, y=big)
    y = hdq.group_norm(x, C)
    ref, amp = exact(x[-1:], C, 1e-5)
    assert bool(((y[-1:].double() - ref).abs() <= bound(ref, amp, torch.bfloat16)).all())
    for part in big.view(reps, S, L, C).split(32):
        assert bool((part == y).all())
    del big, part
    torch.cuda.empty_cache()


# every way of the group norm: kept slabs (4, 8, 16 rows a thread), streamed
# ones, joined chunks, three launches; vectors of 8, 4 and 1 channels, in one
# group or several
SHAPES = [(2, 77, 300, 30), (1, 225, 64, 8), (1, 500, 32, 4), (3, 7, 58, 1), (13, 600, 512, 32), (300, 300, 44, 11),
          (1, 984, 537, 1), (2, 2001, 100, 25), (1, 30000, 64, 8), (2, 9000, 520, 65)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,L,C,G", SHAPES)
def test_large_finite_values_are_normalized(n, L, C, G, dtype):
    g = torch.Generator().manual_seed(n + L + C)
    base = torch.randn(n, L, C, generator=g)
    one = base.clone()
    one[0, L // 2, C // 2] = 2e19                      # one value whose square is past float32
    first = base.clone()
    first[0, 0, 0] = -1e30                             # it is its thread's first row
    ends = 3.3e38 * torch.sign(base)                   # differences are past float32
    for x in (one, first, 2e19 * base, 3e37 * base, ends):
        x = x.to(dtype)
        assert bool(torch.isfinite(x).all())
        ref, amp = exact(x, G, 1e-5)
        y = hdq.group_norm(x.to(DEV), G).cpu().double()
        err = (y - ref).abs()
        assert bool((err <= bound(ref, amp, dtype)).all()), float(err.nan_to_num(nan=math.inf).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,L,C,G", SHAPES)
def test_small_values_without_eps(n, L, C, G, dtype):
    x = (1e-27 * torch.randn(n, L, C, generator=torch.Generator().manual_seed(n + L + C))).to(dtype)
    ref, amp = exact(x, G, 0.0)
    err = (hdq.group_norm(x.to(DEV), G, eps=0.0).cpu().double() - ref).abs()
    assert bool((err <= bound(ref, amp, dtype)).all()), float(err.nan_to_num(nan=math.inf).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,L,C,G", SHAPES + [(1, 1, 64, 8), (3, 1, 320, 32), (2, 16, 520, 65)])
def test_channels_that_differ_but_do_not_vary(n, L, C, G, dtype):
    """Every row the same: a thread's deviations are zero, its channels' means
    differ by more, or without eps by less, than float32's squares hold."""
    row = torch.randn(n, 1, C, generator=torch.Generator().manual_seed(C)).expand(n, L, C)
    for scale, eps in ((1e20, 1e-5), (3e37, 0.0), (1e-27, 0.0)):
        x = (scale * row).to(dtype)
        ref, amp = exact(x, G, eps)
        err = (hdq.group_norm(x.to(DEV), G, eps=eps).cpu().double() - ref).abs()
        assert bool((err <= bound(ref, amp, dtype)).all()), (scale, float(err.nan_to_num(nan=math.inf).max()))


@pytest.mark.parametrize("L", [4096, 40000])
def test_means_that_grow_past_a_float32_square(L):
    """Every row's deviations from its thread's mean have finite squares, the
    distance of neighbouring channels' means has not."""
    x = torch.full((1, L, 64), 2.6e19)
    x[:, :L // 2] = 1.8e19
    x[:, :, 1::2] *= -1
    x = x.to(torch.bfloat16)
    ref, amp = exact(x, 8, 1e-5)
    err = (hdq.group_norm(x.to(DEV), 8).cpu().double() - ref).abs()
    assert bool((err <= bound(ref, amp, torch.bfloat16)).all()), float(err.nan_to_num(nan=math.inf).max())


@pytest.mark.parametrize("n,L,C,G", [(1, 225, 320, 32), (13, 600, 512, 32), (1, 9000, 64, 4), (2, 3000, 256, 16),
                                     (5, 17, 264, 11)])
def test_fp8_form_of_large_finite_values(n, L, C, G):
    """Codes of the normalized values: half an E4M3 step (2^-4 of the value,
    2^-10 of the scale for small ones) beside the norm's own bound."""
    x = (1e20 * torch.randn(n, L, C, generator=torch.Generator().manual_seed(L))).to(torch.bfloat16)
    ref, amp = exact(x, G, 1e-5)
    q = hdq.group_norm_fp8(x.to(DEV), G)
    ref, slack = ref.view(n * L, C), bound(ref, amp, torch.float32).view(n * L, C)
    s = R.scale_per_element(q.scale.cpu(), "rows", n * L)
    v = (q.codes.view(torch.float8_e4m3fn).float().cpu().double() * s)[:, :C]
    tol = torch.maximum(2.0 ** -4 * (ref.abs() + slack), 2.0 ** -10 * s[:, :C]) * (1 + 2.0 ** -20) + slack
    assert bool(((v - ref).abs() <= tol).all())


@pytest.mark.parametrize("n,L,C,G", [(1, 8, 4096, 64), (1, 4000, 4096, 64), (300, 200, 4096, 4096)])
def test_silu_of_float32_outputs(n, L, C, G):
    """A zero weight leaves the bias: y = t / (1 + e^-t) of chosen t.  e^-t =
    2^(-t log2 e) of a float32 product (2 |t| u of itself: the product and the
    constant rounded) and an exponential and a reciprocal of one step each (2 u),
    a sum and a product (u): 2 |t| u e^-t / (1 + e^-t) + 6 u.  From e^-t past
    float32 on, and where the reciprocal would be subnormal, y is 0: up to 2^-119."""
    t = torch.cat((torch.linspace(-110, 110, C // 2), torch.linspace(-4, 4, C // 2)))
    x = torch.randn(n, L, C, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    y = hdq.group_norm(x.to(DEV), G, torch.zeros(C, device=DEV), t.to(DEV), act=hdq.ACT_SILU, y_dtype=hdq.DTYPE_F32)
    assert bool((y == y[0, 0]).all())
    t = t.double()
    ref = t * torch.sigmoid(t)
    tol = (2 * t.abs() * torch.sigmoid(-t) + 6) * U * ref.abs() + 2.0 ** -119
    assert bool(((y[0, 0].cpu().double() - ref).abs() <= tol).all())
