"""The FP8 layer's stated accuracy in the 2-norm, in every kernel and product
form: an output that is off by a small factor, or lacks part of a sum, passes an
elementwise worst case but not this."""
import pytest
import torch

import fp8_ref as R

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from bit_quantized_video_amd import hdq  # noqa: E402

DEV = torch.device("cuda:0")

# up to 16 tokens; 32 x 64 tiles with K in four groups, K that does not divide
# evenly among them; 64 x 64 tiles; 128 x 256 and 256 x 256 tiles
SHAPES = [(16, 4096, 96), (1, 12288, 2000), (3, 136, 700), (33, 4224, 100), (226, 648, 192), (64, 1928, 200),
          (1000, 256, 1030), (700, 1160, 640), (1351, 520, 3900), (4100, 264, 4200), (3000, 264, 4101), (2304, 640, 4096)]


def codes(rows, cols, layout, seed, outliers=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.5 * torch.randn(rows, 1, generator=g))
    if outliers:
        x[:, torch.randperm(cols, generator=g)[:max(1, cols // 100)]] *= 20.0
    return hdq.fp8_quantize(x.to(torch.bfloat16).to(DEV), 1, layout)


def relative_error(y, xq, wq):
    value = lambda t: t.codes.view(torch.float8_e4m3fn).float().cpu()
    ref, _ = R.linear(value(xq), xq.scale.cpu(), value(wq), wq.scale.cpu(), False)
    return float((y.cpu().double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_bf16_output(M, K, N):
    """Rounding: half a step of 2^-7 2^e each way is 2^-7 2^e / sqrt(12) in the
    mean square, on values of 2^e times a mantissa between 1 and 2 whose mean
    square is 2.1 for spread values (4 / 3 is enough): at most 2^-9 of the norm.
    The products' alignment costs 1.3e-5 as stated; 2^-12 leaves room for others
    than Gaussian codes."""
    xq, wq = codes(M, K, hdq.FP8_ROWS, M + K), codes(N, K, hdq.FP8_BLOCKS, N)
    assert relative_error(hdq.fp8_linear(None, wq, xq=xq), xq, wq) <= 2.0 ** -9 + 2.0 ** -12
    xq = codes(M, K, hdq.FP8_ROWS, M + K + 1, outliers=True)
    assert relative_error(hdq.fp8_linear(None, wq, xq=xq), xq, wq) <= 2.0 ** -9 + 2.0 ** -12


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_fp32_output(M, K, N):
    """Exact products.  A block's sum takes four matrix instructions, each with at
    most two roundings of 2^-23 of a partial sum, then the scale pair's and the
    multiply-add's: 20 x 2^-24 of a block's sum, which is 1 / sqrt(kb) of the
    result for independent blocks, kb times if all lean the same way; and the
    multiply-adds' roundings of partial results, at most sqrt(kb) 2^-24 of the
    result for independent ones.  Together below 32 sqrt(kb) 2^-24."""
    xq, wq = codes(M, K, hdq.FP8_ROWS, M + K), codes(N, K, hdq.FP8_BLOCKS, N)
    err = relative_error(hdq.fp8_linear(None, wq, xq=xq, y_dtype=hdq.DTYPE_F32), xq, wq)
    assert err <= 32 * R.blocks(K) ** 0.5 * 2.0 ** -24


def test_public_stream_calls_give_the_same(monkeypatch):
    """What the binding falls back to, on the current stream and within another's context."""
    xq, wq = codes(64, 256, hdq.FP8_ROWS, 1), codes(96, 256, hdq.FP8_BLOCKS, 2)
    want = hdq.fp8_linear(None, wq, xq=xq)
    monkeypatch.setattr(hdq, "_current_device", torch.cuda.current_device)
    monkeypatch.setattr(hdq, "_current_stream", lambda index: torch.cuda.current_stream(index).cuda_stream)
    assert torch.equal(hdq.fp8_linear(None, wq, xq=xq), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = hdq.fp8_linear(None, wq, xq=xq)
    s.synchronize()
    assert torch.equal(y, want)
