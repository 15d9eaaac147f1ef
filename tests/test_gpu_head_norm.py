"""Layer norms of heads whose elements lie far from zero, or are all one value,
on the GPU against float64: what is subtracted is the head's mean to within
its deviations, not to within its elements."""
import pytest
import torch

from test_gpu_heads import BF, DEV, F32, KIND

pytestmark = pytest.mark.gpu
from bit_quantized_video_amd import hdq  # noqa: E402

U = 2.0 ** -24                                   # half a step of float32

# Heads of 16 elements a lane (multiples of 16) and of 8.
DIMS = [16, 48, 64, 72, 80, 96, 112, 128, 200, 240, 256, 512, 5, 21, 50]


def norm(x, dtype=F32, **kw):
    code = hdq.DTYPE_F32 if dtype == F32 else hdq.DTYPE_BF16
    return hdq.qk_norm_rope(x.to(DEV), norm=KIND["layer"], y_dtype=code, **kw).cpu()


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_constant_heads(D, dtype, eps):
    """No deviations: the biases, bit for bit, at any magnitude."""
    g = torch.Generator().manual_seed(D)
    value = torch.randn(1, 40, 7, 1, generator=g) * 10.0 ** (torch.arange(40) % 8 - 3).float().view(1, 40, 1, 1)
    value[0, 5], value[0, 6], value[0, 7] = 3e38, -1e30, 1e-30
    x = value.to(dtype).expand(1, 40, 7, D)
    w, b = torch.randn(D, generator=g), torch.randn(D, generator=g)
    y = norm(x, q_weight=w.to(DEV), q_bias=b.to(DEV), eps=eps)
    assert torch.equal(y, b.expand(1, 40, 7, D))


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("offset", [0.0, 0.5, 2.0, 30.0, 1e3, 1e4, -3e5])
def test_offset_heads(D, offset):
    """Deviations of 1 about any mean, in the 2-norm of all heads.

    With u half a step: a sum takes at most 10 additions in a chain, and 1 / dim
    and the product with it one rounding each, so a mean is within 12 u of the
    mean magnitude of what is summed.  That is values whose own mean is at most a deviation
    from 0, so of a mean magnitude of at most root 2 deviations: 17 u of a deviation.  The
    subtractions, the two products and the sum take another 5 u of an element, the
    sum of squares 12 u, half of it in the root, and the root 2 u.  17 + 5 + 8 = 30 u,
    and 2 u for the terms of second order."""
    g = torch.Generator().manual_seed(D + 1)
    x = torch.randn(3, 50, 5, D, generator=g) + offset
    x64 = x.double()
    d = x64 - x64.mean(-1, keepdim=True)
    ref = d / torch.sqrt(d.square().mean(-1, keepdim=True) + 1e-6)
    off = float((norm(x).double() - ref).norm() / ref.norm())
    assert off <= 32 * U, off / U


@pytest.mark.parametrize("D", [64, 80, 50])
def test_first_element_far_off(D):
    """The element that stands out is the first one: the bound is the same."""
    g = torch.Generator().manual_seed(D + 2)
    x = torch.randn(1, 60, 3, D, generator=g) + 1000.0
    x[..., 0] = 4000.0
    x64 = x.double()
    d = x64 - x64.mean(-1, keepdim=True)
    ref = d / torch.sqrt(d.square().mean(-1, keepdim=True) + 1e-6)
    rows = (norm(x).double() - ref).norm(dim=-1) / ref.norm(dim=-1)
    assert float(rows.max()) <= 32 * U


@pytest.mark.parametrize("D", [64, 96, 50])
def test_a_head_does_not_change_its_neighbours(D):
    """Heads side by side in a wave: an ordinary head has the same bits beside one that is far off."""
    g = torch.Generator().manual_seed(D + 3)
    x = torch.randn(1, 9, 8, D, generator=g)
    far = x.clone()
    far[:, ::2, 1::2] += 5000.0
    far[:, 1::2, ::3] *= 1e30
    same = (far == x).all(-1)
    assert bool(same.any()) and not bool(same.all())
    assert torch.equal(norm(far)[same], norm(x)[same])


@pytest.mark.parametrize("D", [64, 80, 72])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_constant_keys_into_the_cache(D, dtype):
    """The same in the pass that writes the cache: codes and scales of the biases."""
    g = torch.Generator().manual_seed(D + 4)
    k = (100.0 * torch.randn(1, 12, 3, 1, generator=g)).to(dtype).expand(1, 12, 3, D)
    b = torch.randn(D, generator=g)
    b[0] = 4.0
    c = hdq.KvCache(12, 3, D, hdq.CACHE_INT8, device=DEV)
    k = k.contiguous().to(DEV)
    hdq.qkv_to_cache(c, None, k, k, torch.arange(12, device=DEV), KIND["layer"], k_bias=b.to(DEV), eps=0.0)
    top = b.abs().max()
    assert torch.equal(c.k_scale.cpu(), (top / 127).expand(12, 3, 1))
    assert torch.equal(c.k_codes.view(torch.int8).cpu(), torch.round(b * (127 / top)).to(torch.int8).expand(12, 3, D))


@pytest.mark.parametrize("D", [64, 80, 72, 21])
@pytest.mark.parametrize("eps", [1e-38, 1e-30, 1e-20, 1e30])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_eps_next_to_a_heads_size(D, eps, kind):
    """Finite heads with an eps far below their squares (whose scaled value leaves
    float32's normals) or far above them: heads without deviations give the
    biases, the others what the formula gives."""
    g = torch.Generator().manual_seed(D + 5)
    sizes = torch.tensor([3e38, 1e30, 1e10, 1.0, 1e-10, 1e-18])
    x = torch.randn(1, 6, 4, D, generator=g).clamp(-1, 1) * sizes.view(1, 6, 1, 1)
    x[:, :, 1] = sizes.view(1, 6, 1)
    x[:, :, 2] = 0
    b = torch.randn(D, generator=g)
    y = hdq.qk_norm_rope(x.to(DEV), norm=KIND[kind], q_bias=b.to(DEV), eps=eps).cpu()
    x64, e64 = x.double(), float(torch.tensor(eps))
    d = x64 - x64.mean(-1, keepdim=True) if kind == "layer" else x64
    d[:, :, 1] = 0 if kind == "layer" else d[:, :, 1]     # float64's own rounding of a constant head's mean
    ref = d / torch.sqrt(d.square().mean(-1, keepdim=True) + e64)
    # a float32 norm of 32 u (see test_offset_heads) and the sum with the bias
    assert bool(((y.double() - (ref + b)).abs() <= 32 * U * (1 + ref.abs()) + U * (ref + b).abs()).all())
    assert torch.equal(y[0, :, 2], b.expand(6, D))
