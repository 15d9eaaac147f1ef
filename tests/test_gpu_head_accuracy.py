"""Accuracy of the rotation and of the norms' root on the GPU, on inputs whose
result is the cosine, the sine or the reciprocal root itself, and in the 2-norm
on ordinary ones.  u is half a step of float32."""
import math

import pytest
import torch

from test_gpu_heads import BF, DEV, F32, KIND, make, plan

pytestmark = pytest.mark.gpu
from bit_quantized_video_amd import hdq  # noqa: E402

U = 2.0 ** -24


def unit(T, D, split):
    """Pairs (1, 0): rotated ones are (cosine, sine), no rounding beside theirs."""
    x = torch.zeros(T, 1, D)
    j = torch.arange(D // 2)
    ia, ib = (j, j + D // 2) if split else (2 * j, 2 * j + 1)
    x[..., ia] = 1.0
    return x, ia, ib


@pytest.mark.parametrize("D,part", [(64, 64), (128, 128), (80, 80), (72, 72), (64, 32), (50, 50)])
@pytest.mark.parametrize("split", [True, False])
def test_next_to_a_zero(D, part, split):
    """Angles next to quarter turns: the small one of cosine and sine is right to its
    own size.  The fraction of a turn is known to 2^-53 of the position's turns and
    kept in two floats; cosine and sine of the first are within 4 u of themselves, the second
    comes in to first order (its square is below 2^-49) and rounds once.  One float for the fraction
    alone would be off by up to 2 pi 2^-27 next to a quarter turn."""
    T = 64
    g = torch.Generator().manual_seed(D + part)
    quarter = torch.randint(0, 4, (T, part // 2), generator=g).double() / 4
    off = torch.randn(T, part // 2, generator=g, dtype=torch.float64) * 10.0 ** -(2 + 4 * torch.rand(T, part // 2, generator=g, dtype=torch.float64))
    frac = quarter + off                                     # turns at position 1: one plan a token
    x, ia, ib = unit(1, part, split)
    full = torch.zeros(1, 1, D)
    full[..., :part] = x
    one = torch.ones(1, dtype=torch.int64, device=DEV)
    layout = hdq.ROPE_HALF if split else hdq.ROPE_INTERLEAVED
    small = 0
    for t in range(T):
        r = hdq.Rope(part, layout, turns=frac[t].to(DEV))
        y = hdq.rope(full.to(DEV), one, r).cpu().double()[0, 0]
        # off is exact beside the quarter to 2^-54; angles from it alone, so that float64's cosine is next to its zero
        a = 2 * math.pi * (frac[t] - quarter[t])
        q = (4 * quarter[t]).long()
        cos = torch.stack((torch.cos(a), -torch.sin(a), -torch.cos(a), torch.sin(a)))[q, torch.arange(part // 2)]
        sin = torch.stack((torch.sin(a), torch.cos(a), -torch.sin(a), -torch.cos(a)))[q, torch.arange(part // 2)]
        for got, want in ((y[ia], cos), (y[ib], sin)):
            assert bool(((got - want).abs() <= 6 * U * want.abs() + 2.0 ** -48).all())
            small += int((want.abs() < 2.0 ** -6).sum())
    assert small > T * part // 8


@pytest.mark.parametrize("D", [64, 128, 96, 72, 40, 8])
def test_root(D):
    """Heads of an element 1 among integers whose squares add up exactly: the result
    there is the reciprocal root.  The instruction's (1 unit, 2 u) takes one Newton
    step: half the rounding of d r, one of the result, 1.5 u, and the division by dim, half of it
    and of 1 / dim's rounding in the root, 1 u."""
    g = torch.Generator().manual_seed(D)
    x = torch.randint(-40, 41, (1, 400, 5, D), generator=g).float()
    x[..., 3] = 1.0
    y = hdq.qk_norm_rope(x.to(DEV), norm=KIND["rms"], eps=0.0).cpu().double()[..., 3]
    ref = 1.0 / torch.sqrt(x.double().square().mean(-1))
    exact = D & (D - 1) == 0                                  # 1 / dim and the product are
    assert float(((y - ref) / ref).abs().max()) <= (1.5 if exact else 2.5) * U * (1 + 1e-5)


@pytest.mark.parametrize("D,dims,split", [(64, (16, 24, 24), False), (128, (128,), True), (80, (40,), True), (72, (72,), False)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_and_rotation_in_the_2_norm(D, dims, split, kind):
    """Ordinary float32 heads.  A norm is within 30 u (17 u without the mean's 12; see
    test_gpu_head_norm.py), a rotation within 4 + 1 u of a pair's cosine and sine, two
    products and a sum, 8 u of its length: worst cases all at once, and far above what random roundings
    leave.  Those are independent: their root mean square is a third of the bound on one, and a dozen
    of them are 12 ** 0.5 / 3 < 2 u together."""
    T = 400
    q = make((1, T, 6, D), F32, D)
    g = torch.Generator().manual_seed(D)
    pos = torch.randint(0, 100000, (len(dims), 1, T), generator=g)
    turns, r = plan(dims, split)
    y = hdq.qk_norm_rope(q.to(DEV), norm=KIND[kind], positions=pos.to(DEV), rope=r).cpu().double()
    x = q.double()
    x = x - x.mean(-1, keepdim=True) if kind == "layer" else x
    x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    R = sum(dims)
    axis = torch.cat([torch.full((d // 2,), i) for i, d in enumerate(dims)])
    t = pos.movedim(0, 2)[:, :, axis].double() * turns       # to 2^-36 of a turn, float64's own
    a = (2 * math.pi * torch.frac(t)).unsqueeze(2)
    j = torch.arange(R // 2)
    ia, ib = (j, j + R // 2) if split else (2 * j, 2 * j + 1)
    ref = x.clone()
    ref[..., ia] = x[..., ia] * torch.cos(a) - x[..., ib] * torch.sin(a)
    ref[..., ib] = x[..., ib] * torch.cos(a) + x[..., ia] * torch.sin(a)
    assert float((y - ref).norm() / ref.norm()) <= 2 * U
