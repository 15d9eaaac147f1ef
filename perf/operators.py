"""Measured cases of the FP8 block-128 linear layer and of the channels-last group norm.

The operators, each with a plain form in elementary torch operations and a 64-bit form:

  quantize   block-Hadamard rotation and E4M3 codes with one float32 scale per 128 elements of a
             row (activations) or per 128 x 128 block (weights);
  linear     y = x W^T: a bf16 x is quantized as above within the call (input "bf16"), or comes
             as codes and scales (input "codes");
  norm       group norm over channels-last data [n, length, channels], with an optional SiLU;
  norm_fp8   the same norm, its result quantized for a linear layer, and that layer.

`own` selects the framework's calls; otherwise run() computes the plain forms.
"""
import math

import torch

own = False

# The hidden sizes, token counts and layer shapes below are this repository's own (synth.py):
# 17776 = 13 latent frames x 1350 patches + 226 text tokens, 1920 -> 5760 and 3072 -> 12288
# projections, 12288 inner features.  The group norms take a latent grid of 30 x 45 positions
# and its upsampled forms.
BLOCK = 128


def listed():
    return [
        # FFN-down activations of a whole video, rotated in blocks of 128: the largest quantization
        dict(name="quantize video", op="quantize", layout="rows", rows=17776, cols=12288, had=128, x="gelu"),
        # the text tokens alone, a last block of 104 elements, rotated in blocks of 8: latency counts
        dict(name="quantize text", op="quantize", layout="rows", rows=226, cols=1000, had=8, x="outliers"),
        # a QKV projection's weights, unrotated, in 128 x 128 blocks: done once when a layer is loaded
        dict(name="quantize weights", op="quantize", layout="blocks", rows=5760, cols=1920, had=1, x="weights"),
        # one token through a projection: a conditioning vector, or a step of single-token serving
        dict(name="linear one token", op="linear", input="bf16", M=1, K=1920, N=5760, had=128, y="bf16", x="outliers"),
        # text tokens from a text encoder of width 4096, few rows on a long reduction
        dict(name="linear text", op="linear", input="bf16", M=226, K=4096, N=1920, had=64, y="bf16", x="outliers"),
        # three latent frames whose codes are shared by several projections, float32 output
        dict(name="linear frames codes", op="linear", input="codes", M=4050, K=1920, N=5760, had=128, y="f32", x="outliers"),
        # FFN up-projection of a whole video: the largest product
        dict(name="linear video", op="linear", input="bf16", M=17776, K=3072, N=12288, had=128, y="bf16", x="lognormal"),
        # a small map, odd sizes, channels that are no multiple of 8, float32
        dict(name="norm odd f32", op="norm", n=2, L=77, C=300, G=30, act="none", dtype="f32"),
        # latent frames normed one by one, with SiLU
        dict(name="norm latent", op="norm", n=13, L=1350, C=512, G=32, act="silu", dtype="bf16"),
        # eight frames at 240 x 360 normed together, as a video decoder does: the largest norm
        dict(name="norm decoder", op="norm", n=1, L=8 * 240 * 360, C=256, G=32, act="silu", dtype="bf16"),
        # one small map into a projection, channels no multiple of 128
        dict(name="norm to linear map", op="norm_fp8", n=1, L=225, C=320, G=32, act="none", had=64, N=320, y="bf16"),
        # latent frames into a QKV projection
        dict(name="norm to linear frames", op="norm_fp8", n=13, L=1350, C=512, G=32, act="none", had=128, N=1536, y="bf16"),
    ]


def _size(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v))) // step * step or step


def draw(rng):
    op = rng.choice(["quantize", "quantize", "linear", "linear", "linear", "linear", "norm", "norm", "norm_fp8", "norm_fp8"])
    if op == "quantize":
        layout = rng.choice(["rows", "rows", "blocks"])
        had = rng.choice([1, 8, 32, 64, 128])
        cols = _size(rng, 128, 12288, max(8, had))
        rows = _size(rng, 1, min(17776, (17776 * 12288) // cols))
        return dict(op=op, layout=layout, rows=rows, cols=cols, had=had, x=rng.choice(["outliers", "lognormal", "weights"]))
    if op == "linear":
        had = rng.choice([1, 16, 64, 128])
        K = _size(rng, 128, 12288, max(8, had))
        N = _size(rng, 64, 12288)
        M = _size(rng, 1, 17776)
        while M * K * N > 17776 * 3072 * 12288:
            M = max(1, M // 2)
        return dict(op=op, input=rng.choice(["bf16", "bf16", "codes"]), M=M, K=K, N=N, had=had,
                    y=rng.choice(["bf16", "bf16", "f32"]), x=rng.choice(["outliers", "lognormal"]))
    if op == "norm":
        G = rng.choice([1, 8, 32, 32])
        C = _size(rng, max(32, G), 1024, G)
        n = _size(rng, 1, 16)
        L = _size(rng, 1, max(1, (8 * 240 * 360 * 256) // (2 * C * n)))
        return dict(op=op, n=n, L=L, C=C, G=G, act=rng.choice(["none", "silu"]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    had = rng.choice([1, 8, 64])
    G = rng.choice([8, 16, 32])
    C = _size(rng, 64, 1280, 64)
    n = _size(rng, 1, 13)
    L = _size(rng, 1, 5400)
    return dict(op=op, n=n, L=L, C=C, G=G, act=rng.choice(["none", "silu"]), had=had, N=_size(rng, 64, 4096), y="bf16")


# ---- inputs -----------------------------------------------------------------------------------

def _device():
    return torch.device("cuda:0")


def _generator(seed, stream):
    g = torch.Generator(device=_device())
    g.manual_seed(1000003 * int(seed) + stream)
    return g


def _activations(kind, rows, cols, gen):
    """bf16 [rows, cols] with the distributions of synth.py, drawn on the device."""
    z = torch.randn(rows, cols, generator=gen, device=_device())
    if kind == "weights":
        z.mul_(0.02)
    elif kind == "outliers":  # 1% of the channels are 20 times as large
        ch = torch.randperm(cols, generator=gen, device=_device())[:max(1, cols // 100)]
        z[:, ch] *= 20.0
    elif kind == "lognormal":  # a magnitude of its own for each token
        z.mul_(torch.randn(rows, 1, generator=gen, device=_device()).mul_(0.5).exp_())
    elif kind == "gelu":  # GELU outputs and heavy tails
        z = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
        z.add_(torch.randn(rows, cols, generator=gen, device=_device()).pow_(3).mul_(0.5))
    return z.to(torch.bfloat16)


def prepare(case, seed):
    """Inputs of one pass; a linear layer's weights are already in FP8 blocks, as a program keeps them."""
    c = case
    s = {"case": dict(c)}
    if c["op"] == "quantize":
        s["x"] = _activations(c["x"], c["rows"], c["cols"], _generator(seed, 1))
        return s
    if c["op"] == "linear":
        x = _activations(c["x"], c["M"], c["K"], _generator(seed, 1))
        if c["input"] == "codes":
            s["x_codes"], s["x_scale"] = _quantize(x, c["had"], "rows")
        else:
            s["x"] = x
        K = c["K"]
    else:
        gen = _generator(seed, 2)
        n, L, C = c["n"], c["L"], c["C"]
        x = torch.randn(n, L, C, generator=gen, device=_device())
        x = x * (0.5 + torch.rand(1, 1, C, generator=gen, device=_device())) + 2.0 * torch.randn(n, 1, C, generator=gen, device=_device())
        s["x"] = x if c.get("dtype") == "f32" else x.to(torch.bfloat16)
        s["weight"] = 1.0 + 0.2 * torch.randn(C, generator=gen, device=_device())
        s["bias"] = 0.2 * torch.randn(C, generator=gen, device=_device())
        if c["op"] == "norm":
            return s
        K = C
    w = _activations("weights", c["N"], K, _generator(seed, 3))
    s["w_codes"], s["w_scale"] = _quantize(w, c["had"], "blocks")
    return s


# ---- the plain forms --------------------------------------------------------------------------

def _rotate(x, had):
    """Rows of float32 x times H_had / sqrt(had) in blocks: butterflies of strides 1, 2, 4, ..."""
    if had == 1:
        return x
    rows, cols = x.shape
    h = 1
    while h < had:
        v = x.view(rows, cols // (2 * h), 2, h)
        x = torch.stack((v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]), 2).view(rows, cols)
        h *= 2
    return x * torch.tensor(1.0 / math.sqrt(had), dtype=torch.float32, device=x.device)


def _pad(v, rows, cols):
    if v.shape == (rows, cols):
        return v
    out = torch.zeros(rows, cols, dtype=v.dtype, device=v.device)
    out[:v.shape[0], :v.shape[1]] = v
    return out


def _quantize_f32(y, layout):
    """E4M3 codes [rows, K up to a multiple of 128] (zeros past K) and scales of float32 y."""
    rows, cols = y.shape
    kb = -(-cols // BLOCK)
    if layout == "rows":
        y = _pad(y, rows, kb * BLOCK).view(rows, kb, BLOCK)
        amax = y.abs().amax(2, keepdim=True)
    else:
        rb = -(-rows // BLOCK)
        y = _pad(y, rb * BLOCK, kb * BLOCK).view(rb, BLOCK, kb, BLOCK)
        amax = y.abs().amax((1, 3), keepdim=True)
    live = amax >= 2.0 ** -100
    inv = torch.where(live, torch.full_like(amax, 448.0) / torch.where(live, amax, 1.0), 0.0)
    codes = (y * inv).to(torch.float8_e4m3fn).view(-1, kb * BLOCK)[:rows]
    scale = torch.where(live, amax / 448.0, 0.0)
    # activations' scales are kept with the blocks outermost: [blocks, rows]
    return codes.contiguous(), scale.view(rows, kb).t().contiguous() if layout == "rows" else scale.view(-1, kb)


def _quantize(x, had, layout):
    return _quantize_f32(_rotate(x.float(), had), layout)


def _linear(xc, xs, wc, ws, y):
    M, ld = xc.shape
    N, kb = wc.shape[0], ld // BLOCK
    xd = (xc.float().view(M, kb, BLOCK) * xs.t().unsqueeze(2)).view(M, ld)
    wd = wc.float().view(N, kb, BLOCK) * ws.repeat_interleave(BLOCK, 0)[:N].unsqueeze(2)
    out = torch.matmul(xd, wd.view(N, ld).t())
    return out if y == "f32" else out.to(torch.bfloat16)


def _norm(x, weight, bias, groups, act, eps=1e-5):
    n, L, C = x.shape
    v = x.float().view(n, L, groups, C // groups)
    mean = v.mean((1, 3), keepdim=True, dtype=torch.float64)
    d = v - mean.float()
    var = (d * d).mean((1, 3), keepdim=True, dtype=torch.float64)
    t = (d * (var + eps).rsqrt().float()).view(n, L, C) * weight + bias
    return t / (1.0 + torch.exp(-t)) if act == "silu" else t


def _run_plain(s):
    c = s["case"]
    if c["op"] == "quantize":
        codes, scale = _quantize(s["x"], c["had"], c["layout"])
        return {"codes": codes, "scale": scale}
    if c["op"] == "linear":
        xc, xs = (s["x_codes"], s["x_scale"]) if c["input"] == "codes" else _quantize(s["x"], c["had"], "rows")
        return _linear(xc, xs, s["w_codes"], s["w_scale"], c["y"])
    t = _norm(s["x"], s["weight"], s["bias"], c["G"], c["act"])
    if c["op"] == "norm":
        return t if c["dtype"] == "f32" else t.to(torch.bfloat16)
    xc, xs = _quantize_f32(_rotate(t.view(-1, c["C"]), c["had"]), "rows")
    return _linear(xc, xs, s["w_codes"], s["w_scale"], c["y"]).view(c["n"], c["L"], c["N"])


# ---- the framework's calls --------------------------------------------------------------------

def _run_own(s):
    from bit_quantized_video_amd import hdq
    c = s["case"]
    if c["op"] == "quantize":
        q = hdq.fp8_quantize(s["x"], c["had"], hdq.FP8_ROWS if c["layout"] == "rows" else hdq.FP8_BLOCKS)
        return {"codes": q.codes.view(torch.float8_e4m3fn), "scale": q.scale}
    act = hdq.ACT_SILU if c.get("act") == "silu" else hdq.ACT_NONE
    if c["op"] == "norm":
        return hdq.group_norm(s["x"], c["G"], s["weight"], s["bias"], 1e-5, act)
    K = c["K"] if c["op"] == "linear" else c["C"]
    w = hdq.Fp8Tensor(c["N"], K, c["had"], hdq.FP8_BLOCKS, codes=s["w_codes"], scale=s["w_scale"])
    y_dtype = hdq.DTYPE_F32 if c["y"] == "f32" else hdq.DTYPE_BF16
    if c["op"] == "linear":
        if c["input"] == "codes":
            xq = hdq.Fp8Tensor(c["M"], K, c["had"], hdq.FP8_ROWS, codes=s["x_codes"], scale=s["x_scale"])
            return hdq.fp8_linear(None, w, xq=xq, y_dtype=y_dtype)
        return hdq.fp8_linear(s["x"], w, y_dtype=y_dtype)
    xq = hdq.group_norm_fp8(s["x"], c["G"], s["weight"], s["bias"], 1e-5, act, had_block=c["had"])
    return hdq.fp8_linear(None, w, xq=xq, y_dtype=y_dtype).view(c["n"], c["L"], c["N"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ------------------------------------------------------------

def _fp8_bytes(rows, cols, layout):
    kb = -(-cols // BLOCK)
    return rows * kb * BLOCK + 4 * kb * (rows if layout == "rows" else -(-rows // BLOCK))


def work(case):
    """Inputs read once, outputs written once; two operations per multiply-add, log2(had) additions
    per rotated element, and a handful per element of the elementwise parts."""
    c = case
    if c["op"] == "quantize":
        e = c["rows"] * c["cols"]
        return {"bytes": 2 * e + _fp8_bytes(c["rows"], c["cols"], c["layout"]), "flops": e * (3 + math.log2(c["had"]))}
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        xb = 2 * M * K if c["input"] == "bf16" else _fp8_bytes(M, K, "rows")
        return {"bytes": xb + _fp8_bytes(N, K, "blocks") + M * N * (4 if c["y"] == "f32" else 2), "flops": 2.0 * M * N * K}
    e = c["n"] * c["L"] * c["C"]
    if c["op"] == "norm":
        return {"bytes": e * (8 if c["dtype"] == "f32" else 4) + 8 * c["C"], "flops": 8.0 * e}
    M, N = c["n"] * c["L"], c["N"]
    return {"bytes": 2 * e + 8 * c["C"] + _fp8_bytes(N, c["C"], "blocks") + M * N * (4 if c["y"] == "f32" else 2),
            "flops": 8.0 * e + 2.0 * M * N * c["C"]}


# ---- the definition in 64 bits ----------------------------------------------------------------

def _e4m3_64(t):
    """Nearest E4M3 value of |t| <= 448 in float64, ties to even: steps of 2^(e - 3), at least 2^-9."""
    _, e = torch.frexp(t)  # |t| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(t), (e - 1).clamp_(min=-6) - 3)
    return torch.round(t / step) * step


def _hadamard_64(had):
    h = torch.ones(1, 1, dtype=torch.float64, device=_device())
    while h.shape[0] < had:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h / math.sqrt(had)


def _blocks_64(y, layout):
    """E4M3 values and scales of float64 y, laid out as the operator's."""
    rows, cols = y.shape
    kb = -(-cols // BLOCK)
    y = torch.nn.functional.pad(y, (0, kb * BLOCK - cols))
    amax = y.abs().unflatten(1, (kb, BLOCK)).amax(2)  # [rows, kb]
    if layout == "blocks":
        rb = -(-rows // BLOCK)
        amax = torch.nn.functional.pad(amax, (0, 0, 0, rb * BLOCK - rows)).unflatten(0, (rb, BLOCK)).amax(1)
        each = amax.repeat_interleave(BLOCK, 0)[:rows]
    else:
        each = amax
    each = each.unsqueeze(2)
    t = torch.where(each > 0, y.unflatten(1, (kb, BLOCK)) * 448.0 / each, 0.0)
    return _e4m3_64(t).flatten(1), amax / 448.0


def _values_64(v, scale, layout):
    each = scale if layout == "rows" else scale.repeat_interleave(BLOCK, 0)[:v.shape[0]]
    return (v.unflatten(1, (-1, BLOCK)) * each.unsqueeze(2)).flatten(1)


def _rotate_64(x, had):
    return (x.double().unflatten(1, (-1, had)) @ _hadamard_64(had)).flatten(1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        # 2048 rows (whole blocks) at a time: the 64-bit temporaries of a whole video are tens of GB
        parts = [_blocks_64(_rotate_64(p, c["had"]), c["layout"]) for p in s["x"].split(2048)]
        v, scale = (torch.cat(t, 0) for t in zip(*parts))
        return {"codes": v, "scale": scale.t().contiguous() if c["layout"] == "rows" else scale}
    if c["op"] == "linear":
        if c["input"] == "codes":
            x = _values_64(s["x_codes"].double(), s["x_scale"].double().t(), "rows")
        else:
            x = _values_64(*_blocks_64(_rotate_64(s["x"], c["had"]), "rows"), "rows")
    else:
        n, L, C, G = c["n"], c["L"], c["C"], c["G"]
        g = s["x"].double().unflatten(2, (G, C // G))
        var, mean = torch.var_mean(g, (1, 3), correction=0, keepdim=True)
        t = ((g - mean) / torch.sqrt(var + 1e-5)).flatten(2) * s["weight"].double() + s["bias"].double()
        if c["act"] == "silu":
            t = t * torch.sigmoid(t)
        if c["op"] == "norm":
            return t
        x = _values_64(*_blocks_64(_rotate_64(t.flatten(0, 1), c["had"]), "rows"), "rows")
    w = _values_64(s["w_codes"].double(), s["w_scale"].double(), "blocks")
    y = x @ w.t()
    return y if c["op"] == "linear" else y.view(c["n"], c["L"], c["N"])
