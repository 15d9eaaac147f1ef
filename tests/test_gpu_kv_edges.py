"""The key-value cache on the GPU at the shapes next to its limits: Hadamard
blocks of 2 and 4, heads of 16 to 512 elements that fill their lanes or not,
sums that leave float32, tokens that are left out beside others."""
import math

import pytest
import torch

import heads_ref as R
from test_gpu_heads import BF, DEV, F32, KIND, make, plan, positions, reference
from test_gpu_kv_cache import FMT, filled

pytestmark = pytest.mark.gpu
from bit_quantized_video_amd import hdq  # noqa: E402

SHAPES = [(64, 64, 2), (64, 32, 4), (128, 128, 4), (128, 64, 2), (24, 8, 2), (24, 24, 8), (16, 16, 16), (16, 8, 4), (40, 40, 4), (8, 8, 2),
          (32, 32, 32), (48, 16, 16), (48, 48, 4), (112, 16, 16), (112, 112, 8), (384, 128, 128), (384, 384, 64), (504, 8, 8),
          (504, 504, 4), (512, 8, 2), (512, 256, 128), (192, 64, 64), (160, 32, 32)]


@pytest.mark.parametrize("dim,group,had", SHAPES)
@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_write_and_read(dim, group, had, fmt, dtype):
    slots, heads, T = 23, 5, 9
    c, bufs = filled(slots, heads, dim, fmt, group, had, 1)
    k, v = make((T, heads, dim), dtype, 2, 3.0), make((T, heads, dim), dtype, 3, 0.1)
    at = torch.randperm(slots, generator=torch.Generator().manual_seed(4))[:T]
    hdq.cache_write(c, k.to(DEV), v.to(DEV), at.to(DEV))
    ids = torch.arange(slots)
    got = hdq.cache_read(c, ids.to(DEV), y_dtype=hdq.DTYPE_F32)
    for n, x, y in zip(("k", "v"), (k, v), got):
        q, s = R.encode(x.float(), fmt, group, had)
        bufs[n + "_codes"][at], bufs[n + "_scale"][at] = R.to_bytes(q, fmt), s
        assert torch.equal(getattr(c, n + "_codes").cpu(), bufs[n + "_codes"])
        assert torch.equal(getattr(c, n + "_scale").cpu(), bufs[n + "_scale"])
        assert torch.equal(y.cpu(), R.decode(R.from_bytes(bufs[n + "_codes"], fmt), bufs[n + "_scale"], group, had))


@pytest.mark.parametrize("dim,group,had", SHAPES[::2])
@pytest.mark.parametrize("split", [True, False])
def test_step_equals_its_parts(dim, group, had, split):
    """Norm and rotation to float32 and then the cache, against both in one pass: bit for bit where both
    calls take heads the same way, 16 elements a lane or 8 (the cache takes 16 where blocks and groups lie
    within half a head, and adds in another order where not), else both within the bounds."""
    T, H = 7, 3
    x = make((1, T, 3 * H, dim), F32, 5)
    pos = positions(1, 1, T, 6, text=1)
    turns, r = plan((dim,), split)
    d, p = x.to(DEV), pos.to(DEV)
    q, k, v = d[:, :, :H], d[:, :, H:2 * H], d[:, :, 2 * H:]
    at = torch.randperm(12, generator=torch.Generator().manual_seed(7))[:T]
    a, b = (hdq.KvCache(12, H, dim, hdq.CACHE_INT8, group, had, device=DEV) for _ in range(2))
    qo, ko = hdq.qk_norm_rope(q, k, KIND["layer"], positions=p, rope=r)
    hdq.cache_write(a, ko, v, at.to(DEV))
    qf = hdq.qkv_to_cache(b, q, k, v, at.to(DEV), KIND["layer"], positions=p, rope=r)
    within = lambda size: size == dim or dim // 2 % size == 0
    if dim % 16 != 0 or (within(had) and within(group)):
        assert torch.equal(qf, qo)
        for n in ("k_codes", "k_scale", "v_codes", "v_scale"):
            assert torch.equal(getattr(a, n), getattr(b, n)), n
    for y in (qo, qf):
        assert R.close(y, *reference(x[:, :, :H], "layer", None, None, 1e-6, (dim,), split, turns, pos, 1.0))
    z, bound = R.code_bound(*[t[0] for t in reference(x[:, :, H:2 * H], "layer", None, None, 1e-6, (dim,), split, turns, pos, 1.0)],
                            "int8", group, had)
    for c in (a, b):
        val = c.k_codes.cpu().view(torch.int8).double() * c.k_scale.cpu().double().repeat_interleave(group, 2)
        assert bool(((val[at] - z).abs() <= bound).all())


@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("dim,had", [(64, 64), (96, 32), (40, 8)])
def test_sums_past_float32(fmt, dim, had):
    """A block whose butterflies leave float32 counts as one with an infinity; those beside it do not."""
    k = make((1, 4, 2, dim), F32, 7)
    k[0, 1, 0, :had], k[0, 2, 1, :had] = 3e38, 2e38 / had
    c = hdq.KvCache(4, 2, dim, FMT[fmt], 8, had, device=DEV)
    hdq.cache_write(c, k.to(DEV), k.to(DEV), torch.arange(4, device=DEV))
    q, s = R.encode(k[0], fmt, 8, had)
    assert torch.equal(torch.isnan(c.k_scale.cpu()), torch.isnan(s)) and bool(torch.isnan(s[1, 0, :had // 8]).any())
    assert not bool(torch.isnan(s[2]).any())
    assert torch.equal(torch.nan_to_num(c.k_scale.cpu(), 7.0), torch.nan_to_num(s, 7.0))
    assert torch.equal(c.k_codes.cpu(), R.to_bytes(q, fmt))


@pytest.mark.parametrize("dim", [64, 128, 80, 72])
def test_tokens_left_out(dim):
    """A padded batch: tokens without a slot, of NaN, at no position, change nothing of the others and nothing of the cache."""
    T, H = 13, 2
    x = make((1, T, 3 * H, dim), BF, 8)
    out = torch.tensor([0, 3, 4, 7, 12])
    live = torch.ones(T, dtype=torch.bool)
    live[out] = False
    bad = x.clone()
    bad[0, out] = math.nan
    pos = torch.arange(100, 100 + T)
    none = pos.clone()
    none[out] = -1
    at = torch.arange(T)
    left = at.clone()
    left[out] = torch.tensor([-1, 20, 1 << 40, -(1 << 62), 20])
    _, r = plan((dim,), True)
    caches = []
    for t, p, s in ((x, pos, at), (bad, none, left)):
        c = hdq.KvCache(20, H, dim, hdq.CACHE_FP8, device=DEV)
        d = t.to(DEV)
        y = hdq.qkv_to_cache(c, d[:, :, :H], d[:, :, H:2 * H], d[:, :, 2 * H:], s.to(DEV), KIND["layer"], positions=p.to(DEV), rope=r)
        caches.append((y.cpu()[0], c.k_codes.cpu(), c.k_scale.cpu(), c.v_codes.cpu(), c.v_scale.cpu()))
    for a, b in zip(*caches):
        assert torch.equal(a[:T][live], b[:T][live])
    for b in caches[1][1:]:
        assert not bool(b[out].any()) and not bool(b[T:].any())
