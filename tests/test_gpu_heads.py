"""Head norms and rotary positions on the GPU against float64: layouts, axes,
parts of the head, odd head sizes, strides, types, ranges, streams, graphs."""
import math
from fractions import Fraction

import pytest
import torch

import heads_ref as R

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from bit_quantized_video_amd import hdq  # noqa: E402

DEV = torch.device("cuda:0")
KIND = {"none": hdq.HEAD_NORM_NONE, "layer": hdq.HEAD_NORM_LAYER, "rms": hdq.HEAD_NORM_RMS}
BF, F32 = torch.bfloat16, torch.float32


def make(shape, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * (0.5 + torch.rand(shape[-1], generator=g)) + 0.3 * torch.randn(shape[-1], generator=g)
    return (x * spread).to(dtype)


def weights(D, seed):
    g = torch.Generator().manual_seed(seed)
    return [1 + 0.2 * torch.randn(D, generator=g), 0.2 * torch.randn(D, generator=g)]


def positions(axes, B, T, seed, text=0, top=5000):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, top, (axes, B, T), generator=g)
    p[:, :, :text] = -1
    if axes > 1 and T > text:
        p[-1, 0, -1] = -7          # negative on one axis alone: not rotated either
    return p


def plan(dims, split, scale=1.0):
    turns = torch.cat([hdq.rope_turns(d) for d in dims])
    return turns, hdq.Rope(dims, hdq.ROPE_HALF if split else hdq.ROPE_INTERLEAVED, scale=scale, turns=turns.to(DEV))


def reference(x, kind, w, b, eps, dims, split, turns, pos, scale):
    y = x.double()
    y, tol = R.head_norm(x, kind, eps, w, b) if kind != "none" else (y, torch.zeros_like(y))
    return R.rotate(y, tol, dims, split, turns, pos, scale) if dims else (y, tol)


@pytest.mark.parametrize("D,dims,split", [
    (64, (64,), True), (64, (64,), False), (64, (16, 24, 24), False), (64, (16, 24, 24), True), (128, (96,), True),
    (80, (80,), True), (80, (40,), True), (80, (20, 30, 30), True), (96, (48,), False), (72, (72,), False), (256, (64, 192), True),
    (512, (512,), True), (512, (512,), False), (320, (100,), True), (40, (40,), True), (8, (8,), True), (8, (2,), False),
    (2, (2,), True), (1, (), True), (6, (6,), False), (21, (14,), True), (200, (2, 4, 6), True), (64, (), False)])
@pytest.mark.parametrize("kind", ["none", "layer", "rms"])
def test_queries_and_keys(D, dims, split, kind):
    B, T, Hq, Hk = 2, 9, 6, 3
    q, k = make((B, T, Hq, D), BF, 1), make((B, T, Hk, D), BF, 2)
    (qw, qb), (kw, kb) = weights(D, 3), weights(D, 4)
    pos = positions(max(1, len(dims)), B, T, 5, text=2)
    turns, r = plan(dims, split, 1.25) if dims else (None, None)
    dev = [t.to(DEV) for t in (qw, kw, qb, kb)]
    out = hdq.qk_norm_rope(q.to(DEV), k.to(DEV), KIND[kind], *dev, eps=1e-5, positions=pos.to(DEV) if dims else None, rope=r)
    for y, x, w, b in zip(out, (q, k), (qw, kw), (qb, kb)):
        ref, tol = reference(x, kind, w, b, 1e-5, dims, split, turns, pos, 1.25)
        assert y.dtype == BF and y.shape == x.shape and y.is_contiguous()
        assert R.close(y, ref, tol)


@pytest.mark.parametrize("B,T,H,D", [(1, 1, 1, 64), (1, 1, 30, 64), (7, 1, 24, 128), (1, 300, 1, 64), (3, 5, 2, 8), (1, 17, 1, 8),
                                     (1, 2, 130, 64), (4, 33, 3, 128), (1, 65, 7, 512), (2, 3, 11, 96), (1, 5000, 2, 16)])
def test_sizes(B, T, H, D):
    """Few and many tokens and heads: several tokens a wave, several waves a token."""
    x = make((B, T, H, D), F32, 6)
    pos = positions(1, B, T, 7)
    turns, r = plan((D,), True)
    w, b = weights(D, 8)
    y = hdq.qk_norm_rope(x.to(DEV), norm=hdq.HEAD_NORM_LAYER, q_weight=w.to(DEV), q_bias=b.to(DEV), positions=pos.to(DEV), rope=r)
    ref, tol = reference(x, "layer", w, b, 1e-6, (D,), True, turns, pos, 1.0)
    assert R.close(y, ref, tol)


@pytest.mark.parametrize("x_type,y_type", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("D", [64, 50])
def test_types(x_type, y_type, D):
    q, k = make((2, 5, 4, D), x_type, 9), make((2, 5, 1, D), x_type, 10)
    pos = positions(1, 2, 5, 11)
    turns, r = plan((D,), False)
    code = hdq.DTYPE_F32 if y_type == F32 else hdq.DTYPE_BF16
    out = hdq.qk_norm_rope(q.to(DEV), k.to(DEV), hdq.HEAD_NORM_RMS, positions=pos.to(DEV), rope=r, y_dtype=code)
    for y, x in zip(out, (q, k)):
        ref, tol = reference(x, "rms", None, None, 1e-6, (D,), False, turns, pos, 1.0)
        assert y.dtype == y_type and R.close(y, ref, tol)


@pytest.mark.parametrize("view", ["qkv", "heads first", "odd base", "odd stride", "expanded", "in place", "out views"])
def test_views(view):
    B, T, H, D = 2, 7, 5, 64
    pos = positions(1, B, T, 12, text=1).to(DEV)
    turns, r = plan((D,), True)
    full = make((B, T, 3 * H, D), BF, 13).to(DEV)
    q, k, kw = full[:, :, :H], full[:, :, H:2 * H], {}
    if view == "heads first":
        q, k = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k))
    elif view == "odd base":
        flat = make((B * T * H * D + 1,), BF, 14).to(DEV)
        q = k = flat[1:].view(B, T, H, D)
    elif view == "odd stride":
        q = k = make((B, T, H, D + 3), BF, 15).to(DEV)[..., :D]
    elif view == "expanded":
        q = q[:, :, :1].expand(B, T, H, D)
        pos = pos[:, :1].expand(1, B, T)
    before, want = full.clone(), [t.clone() for t in (q, k)]
    if view == "in place":
        kw = dict(q_out=q, k_out=k)
    elif view == "out views":
        room = torch.full((B, H, T, 2, D), 7.0, dtype=BF, device=DEV)
        kw = dict(q_out=room[:, :, :, 0].transpose(1, 2), k_out=torch.empty(B, T, H, D + 1, dtype=BF, device=DEV)[..., 1:])
    out = hdq.qk_norm_rope(q, k, hdq.HEAD_NORM_LAYER, positions=pos, rope=r, **kw)
    for y, x in zip(out, want):
        ref, tol = reference(x.cpu(), "layer", None, None, 1e-6, (D,), True, turns, pos.cpu(), 1.0)
        assert R.close(y, ref, tol)
    if view == "in place":
        assert out[0].data_ptr() == full.data_ptr() and torch.equal(full[:, :, 2 * H:], before[:, :, 2 * H:])
    else:
        assert torch.equal(full, before)
    if view == "out views":
        assert bool((room[:, :, :, 1] == 7.0).all())


def test_position_shapes():
    x = make((2, 6, 2, 64), F32, 16).to(DEV)
    _, r = plan((64,), False)
    p = torch.arange(6, device=DEV)
    want = hdq.rope(x, p.expand(1, 2, 6).contiguous(), r)
    for q in (p, p.expand(2, 6), p.expand(1, 6), torch.stack((p, p), 1).t()):
        assert torch.equal(hdq.rope(x, q, r), want)
    assert torch.equal(hdq.rope(x[0], p, r), want[0])
    assert torch.equal(hdq.rope(x, p, r, out=torch.empty_like(x)), want)
    _, r3 = plan((16, 24, 24), False)
    p3 = torch.stack((p, 2 * p, 3 * p))
    assert torch.equal(hdq.rope(x, p3, r3), hdq.rope(x, p3.unsqueeze(1).expand(3, 2, 6), r3))
    assert torch.equal(hdq.rope(x, torch.stack((p, 2 * p, 3 * p), 1).t(), r3), hdq.rope(x, p3, r3))
    for bad in (p[:5], p.int(), p3, p.cpu()):
        with pytest.raises(ValueError):
            hdq.rope(x, bad, r)
    with pytest.raises(ValueError):
        hdq.rope(x, None, r)


@pytest.mark.parametrize("split", [True, False])
def test_far_positions(split):
    """Positions to 2^52: the fraction of a turn against exact rationals of the
    same float64 frequencies."""
    D, pos = 64, [0, 1, 4095, (1 << 20) + 3, (1 << 31) - 1, (1 << 40) + 12345, (1 << 52) + 1]
    turns, r = plan((D,), split)
    x = make((len(pos), 3, D), F32, 17)
    y = hdq.rope(x.to(DEV), torch.tensor(pos, device=DEV), r).cpu().double()
    frac = torch.tensor([[float(Fraction(p) * Fraction(float(t)) % 1) for t in turns] for p in pos], dtype=torch.float64)
    cos, sin = torch.cos(2 * math.pi * frac).unsqueeze(1), torch.sin(2 * math.pi * frac).unsqueeze(1)
    j = torch.arange(D // 2)
    ia, ib = (j, j + D // 2) if split else (2 * j, 2 * j + 1)
    a, b = x.double()[..., ia], x.double()[..., ib]
    tol = 13 * R.U * (a.abs() + b.abs())           # as heads_ref.rotate's, and the output's rounding
    assert bool(((y[..., ia] - (a * cos - b * sin)).abs() <= tol).all())
    assert bool(((y[..., ib] - (b * cos + a * sin)).abs() <= tol).all())


def test_unrotated_tokens_keep_their_bits():
    x = make((1, 8, 3, 64), BF, 18)
    x[0, 2, 1, 5], x[0, 2, 1, 37], x[0, 3, 0, 63] = math.inf, math.nan, -math.inf
    for split in (True, False):
        _, r = plan((48,), split)
        p = torch.tensor([5, 6, -1, -(1 << 40), 7, 8, 9, 10], device=DEV)
        y = hdq.rope(x.to(DEV), p, r).cpu()
        assert torch.equal(y[0, 2:4].view(torch.int16), x[0, 2:4].view(torch.int16))
        assert torch.equal(y[..., 48:].view(torch.int16), x[..., 48:].view(torch.int16))


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_range(kind):
    """Magnitudes whose squares leave float32, zeros, and NaN or infinities that
    stay in their head."""
    for eps in (0.0, 1e-6):
        x = make((1, 8, 4, 96), F32, 19)
        for i, s in enumerate((1e30, 3e37, 1e-30, 1e-37, 1.0, 1e18, 1e-12, 1e-20)):
            x[0, i] *= s
        ref, tol = R.head_norm(x, kind, eps, None, None)
        # inputs below the normals lose bits when scaled: 2^-149 of the largest, 1e-37 here
        tol = tol + (2.0 ** -149 / 1e-38 if eps == 0.0 else 0.0)
        assert R.close(hdq.qk_norm_rope(x.to(DEV), norm=KIND[kind], eps=eps), ref, tol + 2.0 ** -126)
    x = make((1, 3, 4, 64), BF, 20)
    x[0, 0, 1] = 0
    x[0, 1, 2, 7], x[0, 2, 3, 9] = math.nan, math.inf
    w, b = weights(64, 21)
    y = hdq.qk_norm_rope(x.to(DEV), norm=KIND[kind], eps=0.0, q_weight=w.to(DEV), q_bias=b.to(DEV), y_dtype=hdq.DTYPE_F32).cpu()
    bad = torch.zeros(1, 3, 4, dtype=torch.bool)
    bad[0, 1, 2] = bad[0, 2, 3] = True
    assert bool(torch.isnan(y[bad]).all()) and bool(torch.isfinite(y[~bad]).all())
    assert torch.equal(y[0, 0, 1], b)


def test_empty_and_refused():
    x = torch.empty(2, 0, 4, 64, dtype=BF, device=DEV)
    assert hdq.qk_norm_rope(x, x, hdq.HEAD_NORM_RMS)[1].shape == x.shape
    q = make((2, 3, 4, 64), BF, 22).to(DEV)
    for args, kw in (((q, q[:, :2]), {}), ((q, q[..., :32]), {}), ((q,), dict(q_out=q[:, :2])), ((q.half(),), {}),
                     ((q[..., ::2],), {}), ((q,), dict(norm=1, q_weight=torch.ones(64, device=DEV, dtype=BF))),
                     ((q,), dict(norm=1, q_weight=torch.ones(32, device=DEV)))):
        with pytest.raises(ValueError):
            hdq.qk_norm_rope(*args, **kw)
    with pytest.raises(hdq.HdqError):
        hdq.qk_norm_rope(q, q_out=torch.empty(2, 3, 1, 64, dtype=BF, device=DEV).expand(2, 3, 4, 64))


def test_stream_and_graph():
    q, k = make((1, 50, 6, 64), BF, 23).to(DEV), make((1, 50, 2, 64), BF, 24).to(DEV)
    pos = positions(1, 1, 50, 25).to(DEV)
    _, r = plan((64,), True)
    want = hdq.qk_norm_rope(q, k, hdq.HEAD_NORM_RMS, positions=pos, rope=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hdq.qk_norm_rope(q, k, hdq.HEAD_NORM_RMS, positions=pos, rope=r, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = hdq.qk_norm_rope(q, k, hdq.HEAD_NORM_RMS, positions=pos, rope=r)
    for i in range(3):
        q.copy_(make(q.shape, BF, 30 + i))
        pos.add_(i)
        want = hdq.qk_norm_rope(q, k, hdq.HEAD_NORM_RMS, positions=pos, rope=r)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_elements_past_32_bits():
    """A head stride that takes the last heads past 2^32 elements."""
    H, T, D = 3, 4, 64
    stride = (1 << 31) + 64
    buf = torch.empty(2 * stride + T * D, dtype=BF, device=DEV)
    x = buf.as_strided((T, H, D), (D, stride, 1))
    src = make((T, H, D), BF, 26)
    x.copy_(src)
    pos = torch.arange(T, device=DEV)
    turns, r = plan((D,), True)
    ref, tol = reference(src.unsqueeze(0), "rms", None, None, 1e-6, (D,), True, turns, pos.cpu().view(1, 1, T), 1.0)
    y = hdq.qk_norm_rope(x, norm=hdq.HEAD_NORM_RMS, positions=pos, rope=r, q_out=x)
    assert R.close(y.unsqueeze(0), ref, tol)
