"""Plain references, on the CPU, of the head norms, rotary positions, the
quantized key-value cache and the 4-bit group-scaled layer: products, norms
and angles in float64 with bounds on the kernels' errors, codings in the
operators' own float32 roundings."""
import math

import torch

import fp8_ref

U = 2.0 ** -24                                   # half a step of float32
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
TOP = {"int8": 127.0, "fp8": 448.0, "int4": 7.0}


def head_norm(x, kind, eps, w, b):
    """(norm of float64 [..., dim], bound on the float32 evaluation).

    A sum of up to 512 terms takes at most 3 + 6 additions in a chain (in a lane
    and over lanes; a square's products are fused), so a sum of squares is
    within 16 u of itself, and with the division by dim, eps, the reciprocal
    root (2 units), the two products: 24 u of |x rstd w|.  A mean is within
    16 u of the mean magnitude and rounded to u of itself, which shifts every
    deviation alike; the variance moves by the square of that shift."""
    x = x.double()
    D = x.shape[-1]
    w = (torch.ones(D) if w is None else w).double()
    b = (torch.zeros(D) if b is None else b).double()
    shift = torch.zeros_like(x[..., :1])
    if kind == "layer":
        shift = 18 * U * x.abs().amax(-1, keepdim=True)
        x = x - x.mean(-1, keepdim=True)
    var = x.square().mean(-1, keepdim=True) + eps
    rstd = torch.where(var > 0, 1 / torch.sqrt(torch.where(var > 0, var, torch.ones_like(var))), torch.zeros_like(var))
    xh = x * rstd
    s = shift * rstd
    tol = (s + xh.abs() * (24 * U + 2 * s + s * s)) * w.abs() + 2 * U * ((xh * w).abs() + b.abs())
    return xh * w + b, tol


def rotate(x, tol, dims, split, turns, pos, scale=1.0):
    """x float64 [batch, length, heads, dim] with error `tol`, turned; pos int64
    [axes, batch, length].  The angle's fraction is rounded to float32 (u / 2 of a
    turn at most), its sine and cosine are within 4 u, their products with scale
    and the element and the sum within 4 u: 12 u of the pair's magnitudes, and
    what the reference's own float64 product loses."""
    R = sum(dims)
    axis = torch.cat([torch.full((d // 2,), i) for i, d in enumerate(dims)])
    live = (pos >= 0).all(0)
    p = pos.movedim(0, 2)[:, :, axis]
    # the product exactly: positions in two parts of 26 bits, each times turns' two halves would be needed; float64
    # products of a position below 2^26 lose half a step, which `lost` counts
    t = p.double() * turns
    lost = (2 * math.pi * t.abs() * 2.0 ** -52).unsqueeze(2)
    ang = (2 * math.pi * torch.frac(t)).unsqueeze(2)
    cos, sin = scale * torch.cos(ang), scale * torch.sin(ang)
    out, err = x.clone(), tol.clone()
    j = torch.arange(R // 2)
    ia, ib = (j, j + R // 2) if split else (2 * j, 2 * j + 1)
    a, b, ta, tb = x[..., ia], x[..., ib], tol[..., ia], tol[..., ib]
    out[..., ia], out[..., ib] = a * cos - b * sin, b * cos + a * sin
    e = scale * (ta + tb) + (12 * U + lost) * scale * (a.abs() + b.abs())
    err[..., ia], err[..., ib] = e, e
    keep = live[:, :, None, None]
    return torch.where(keep, out, x), torch.where(keep, err, tol)


def close(y, ref, tol):
    """y within the bound and the rounding of its type."""
    half = HALF[y.dtype]
    return bool(((y.cpu().double() - ref).abs() <= tol * (1 + half) + half * ref.abs()).all())


# ---- cache ---------------------------------------------------------------------

def hadamard(y, had):
    """float32 [..., dim], the operator's own butterflies."""
    return fp8_ref.rotate(y.reshape(-1, y.shape[-1]).float(), had).view(y.shape) if had > 1 else y.float()


def encode(x, fmt, group, had):
    """(code values float32 [..., dim], scales [..., dim / group]) of float32 x, in the operator's roundings."""
    v = hadamard(x, had).unflatten(-1, (-1, group))
    a, top = v.abs().amax(-1, keepdim=True), TOP[fmt]
    bad = ~torch.isfinite(v).all(-1, keepdim=True)
    live = (a >= 2.0 ** -100) & ~bad
    safe = torch.where(live, a, torch.ones_like(a))
    t = torch.where(live, v * (torch.full_like(safe, top) / safe), torch.zeros_like(v))
    q = t.to(torch.float8_e4m3fn).float() if fmt == "fp8" else torch.round(t).clamp(-top, top)
    scale = torch.where(live, a / top, torch.where(bad, torch.full_like(a, math.nan), torch.zeros_like(a)))
    return q.flatten(-2), scale.squeeze(-1)


def to_bytes(q, fmt):
    """Code values to the cache's bytes."""
    if fmt == "fp8":
        return q.to(torch.float8_e4m3fn).view(torch.uint8)
    b = q.to(torch.int8).view(torch.uint8)
    return b if fmt == "int8" else (b[..., 0::2] & 15) | (b[..., 1::2] << 4)


def from_bytes(b, fmt):
    if fmt == "fp8":
        return b.view(torch.float8_e4m3fn).float()
    if fmt == "int8":
        return b.view(torch.int8).float()
    q = torch.stack((b & 15, b >> 4), -1).flatten(-2).to(torch.int16)
    return torch.where(q > 7, q - 16, q).float()


def decode(q, scale, group, had):
    """float32 values in the operator's roundings."""
    return hadamard((q.unflatten(-1, (-1, group)) * scale.unsqueeze(-1)).flatten(-2), had)


def code_bound(y, tol, fmt, group, had):
    """Bound on |code scale - Hadamard(y)| for float64 y known to `tol`: half a
    step of the code (of E4M3: 2^-4 of the value, 2^-10 of the scale's unit below
    its normals), and the rotation's error."""
    H = torch.ones(1, 1, dtype=torch.float64)
    while H.shape[0] < had:
        H = torch.cat((torch.cat((H, H), 1), torch.cat((H, -H), 1)), 0)
    blocks = y.unflatten(-1, (-1, had))
    z = (blocks @ (H / math.sqrt(had))).flatten(-2)
    spread = lambda v: (v.unflatten(-1, (-1, had)).sum(-1, keepdim=True).expand(blocks.shape) / math.sqrt(had)).flatten(-2)
    err = spread(tol) + (math.log2(had) + 2) * U * spread(y.abs())
    scale = (z.abs() + err).unflatten(-1, (-1, group)).amax(-1, keepdim=True) / TOP[fmt]
    scale = scale.expand(*scale.shape[:-1], group).flatten(-2)
    step = 2.0 ** -4 * (z.abs() + err) + 2.0 ** -10 * scale if fmt == "fp8" else 0.5 * scale
    return z, err + step * (1 + 8 * U) + 8 * U * scale * TOP[fmt]


# ---- 4-bit weights ---------------------------------------------------------------

def w4_random(N, K, group, zero, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scale = (0.002 + 0.01 * torch.rand(N, K // group, generator=g)).to(torch.bfloat16)
    z = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8) if zero else None
    return codes, scale, z


def w4_values(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def w4_linear(x, codes, scale, zero, group):
    """(y float64, bound): a group's sums of (16 + u) x and (16 + z) x, beside each other
    or one after the other, round at most group + 8 times (a matrix instruction adds
    several products before it rounds), the scaled sums once a group and once a wave more."""
    N = codes.shape[0]
    u = w4_values(codes).double().view(N, -1, group)
    z = zero.double().unsqueeze(2) if zero is not None else torch.full((N, u.shape[1], 1), 8.0, dtype=torch.float64)
    s = scale.double().unsqueeze(2)
    xd = x.double()
    y = xd @ ((u - z) * s).flatten(1).t()
    big = xd.abs() @ ((32 + u + z) * s.abs()).flatten(1).t()
    rest = xd.abs() @ ((u - z).abs() * s.abs()).flatten(1).t()
    return y, (group + 10) * U * big + (u.shape[1] + 20) * U * rest


def w4_pack(codes, scale, zero, group):
    """The packed buffers of include/hdq.h's tiles, byte for byte."""
    N, K = codes.shape[0], 2 * codes.shape[1]
    tn, tk, groups = -(-N // 16), -(-K // 128), 128 // group
    u = torch.zeros(tn * 16, tk * 128, dtype=torch.int64)
    u[:N, :K] = w4_values(codes).long()
    # [tile n][row][tile k][word s][quarter][8] -> [tile n][tile k][quarter][row][word][8]
    v = u.view(tn, 16, tk, 4, 4, 8).permute(0, 2, 4, 1, 3, 5)
    place = torch.tensor([4 * ((e >> 1) + 4 * (e & 1)) for e in range(8)])
    words = (v << place).sum(-1)
    words = ((words << 3) & 0xffffffff) | (words >> 29)
    packed = torch.stack([(words >> (8 * i)) & 255 for i in range(4)], -1).to(torch.uint8).flatten()

    def per_group(t):
        full = torch.zeros(tn * 16, -(-tk // 4) * 4 * groups, dtype=t.dtype)
        full[:N, :K // group] = t
        return full.view(tn, 16, -1, 4 * groups).transpose(1, 2).contiguous().flatten()
    return packed, per_group(scale), per_group(zero) if zero is not None else None


def w4_quantize(w, group, zero):
    """(codes, scale, zero) of bf16 weights in the operator's float32 roundings."""
    N, K = w.shape
    v = w.float().view(N, K // group, group)
    ok = torch.isfinite(v).all(2, keepdim=True)
    hi, lo = v.amax(2, keepdim=True).clamp(min=0), v.amin(2, keepdim=True).clamp(max=0)
    raw = (0.5 * hi - 0.5 * lo) / 7.5 if zero else torch.maximum(hi, -lo) / 7.0
    live = ok & (raw >= 2.0 ** -100)
    s = torch.where(live, raw.to(torch.bfloat16).float(), torch.zeros_like(raw))
    safe = torch.where(live, s, torch.ones_like(s))
    z = torch.where(live, torch.round(-lo / safe).clamp(max=15), torch.zeros_like(s)) if zero else torch.full_like(s, 8.0)
    u = torch.where(live, (torch.round(v / safe) + z).clamp(0, 15), z.expand_as(v)).to(torch.uint8).view(N, K)
    scale = torch.where(ok, s, torch.full_like(s, math.nan)).to(torch.bfloat16).squeeze(2)
    return u[:, 0::2] | (u[:, 1::2] << 4), scale, z.to(torch.uint8).squeeze(2) if zero else None
