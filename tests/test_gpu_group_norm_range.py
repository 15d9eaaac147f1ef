"""The group norm at the ends of its input range: long runs of rows on a large mean."""
import pytest
import torch

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
    difference, 16 u for the sum, 2 u for a pair's root, so rstd 10 u of itself;
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
