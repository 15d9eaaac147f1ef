"""Plain references of the FP8 block-128 layer: the coding in float32 on the
CPU (the operator's own roundings, so codes and scales are equal) and the
products in float64."""
import math

import torch

BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def rotate(x, had):
    """float32 rows x H_had / sqrt(had): butterflies of strides 1, 2, 4, ..."""
    x = x.float().clone()
    rows, cols = x.shape
    h = 1
    while h < had:
        v = x.view(rows, cols // (2 * h), 2, h)
        u, w = v[:, :, 0].clone(), v[:, :, 1].clone()
        v[:, :, 0], v[:, :, 1] = u + w, u - w
        h *= 2
    return x * torch.tensor(1.0 / math.sqrt(had), dtype=torch.float32) if had > 1 else x


def block_view(y, layout):
    """y padded with zeros to whole blocks, [row blocks, rows, column blocks, 128]."""
    rows, cols = y.shape
    per = 1 if layout == "rows" else BLOCK
    p = torch.zeros(-(-rows // per) * per, blocks(cols) * BLOCK, dtype=y.dtype)
    p[:rows, :cols] = y
    return p.view(-1, per, blocks(cols), BLOCK)


def quantize(y, layout):
    """(code values float32 [rows, 128 kb], scales in the operator's layout) of float32 y."""
    rows = y.shape[0]
    v = block_view(y, layout)
    a = v.abs().amax((1, 3), keepdim=True)
    bad = ~torch.isfinite(v).all(3, keepdim=True).all(1, keepdim=True)
    live = (a >= 2.0 ** -100) & ~bad
    safe = torch.where(live, a, torch.ones_like(a))
    codes = torch.where(live, v * (torch.full_like(safe, 448.0) / safe), torch.zeros_like(v)).to(torch.float8_e4m3fn).float()
    scale = torch.where(live, a / 448.0, torch.where(bad, torch.full_like(a, math.nan), torch.zeros_like(a)))
    scale = scale.reshape(-1, v.shape[2])
    return codes.reshape(-1, v.shape[2] * BLOCK)[:rows], scale.t().contiguous() if layout == "rows" else scale


def scale_per_element(scale, layout, rows):
    """The operator's scales as float64 [rows, 128 kb]."""
    s = scale.double()
    s = s.t() if layout == "rows" else s.repeat_interleave(BLOCK, 0)[:rows]
    return s.repeat_interleave(BLOCK, 1)


def linear(xc, xs, wc, ws, out_bf16):
    """(y in float64, bound on the kernel's error) from code values and scales.

    Each product of a block is exact.  fp32 output: the block's 128 products
    and the blocks are summed in float32, at most 128 + blocks + 8 roundings
    (scale products, the halving sum over waves) of 2^-24 of the sum of
    magnitudes.  bf16 output: also 2^-14 of a block's largest product for each
    of its 128 (the matrix instruction's alignment), and the rounding of the
    result, 2^-8 of it."""
    M, ld = xc.shape
    N, kb = wc.shape[0], ld // BLOCK
    xd = xc.double() * scale_per_element(xs, "rows", M)
    wd = wc.double() * scale_per_element(ws, "blocks", N)
    y = xd @ wd.t()
    tol = (128 + kb + 8) * 2.0 ** -24 * (xd.abs() @ wd.abs().t())
    if out_bf16:
        xm = xd.abs().view(M, kb, BLOCK).amax(2)
        wm = wd.abs().view(N, kb, BLOCK).amax(2)
        tol = tol + 128 * 2.0 ** -14 * (xm @ wm.t())  # the largest product is at most the product of the largest
        tol = tol + 2.0 ** -8 * (y.abs() + tol)
    return y, tol
