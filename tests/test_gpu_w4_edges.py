"""The 4-bit layer on the GPU: nothing behind the tokens, the weights' rows or the
output takes part in a result."""
import math

import pytest
import torch

import heads_ref as R
from test_gpu_heads import BF, DEV, F32, make

pytestmark = pytest.mark.gpu
from bit_quantized_video_amd import hdq  # noqa: E402


@pytest.mark.parametrize("M", [1, 2, 3, 15, 16, 17, 33, 64, 65])
@pytest.mark.parametrize("N,K,group", [(17, 32, 32), (33, 64, 64), (16, 96, 32), (40, 160, 32), (48, 192, 64), (5, 1120, 32),
                                       (20, 2016, 32), (12300, 96, 32), (20, 4128, 32), (20, 8224, 32)])
def test_nan_behind_the_tokens(M, N, K, group):
    """Tokens in front of a block of NaN: each form's reads past the last column and token are zeros."""
    codes, scale, z = R.w4_random(N, K, group, True, M + N)
    x = make((M, K), BF, 1)
    room = torch.full((M * K + 64 * K + 16384,), math.nan, dtype=BF, device=DEV)
    room[:M * K] = x.to(DEV).flatten()
    w = hdq.w4_pack(codes.to(DEV), scale.to(DEV), z.to(DEV))
    y = hdq.w4_linear(room[:M * K].view(M, K), w, y_dtype=hdq.DTYPE_F32)
    assert bool(torch.isfinite(y).all())
    ref, tol = R.w4_linear(x, codes, scale, z, group)
    assert R.close(y, ref, tol)
