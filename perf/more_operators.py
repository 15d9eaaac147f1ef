"""Measured cases of the operators around a transformer block's linear layers.

The operators, each with a plain form in elementary torch operations and a 64-bit form:

  w4     y = x W^T for few tokens, W in 4-bit codes with one scale (and zero point) per group of
         a row's elements;
  rope   rotary positions of one tensor: interleaved or half layout, part of the head, one to three
         position axes, frequencies scaled for long contexts; tokens at a negative position are left;
  qk     a norm of queries and keys over each head (layer or RMS) and the same rotation, in one pass;
  cache  keys and values quantized (INT8, FP8 or INT4 with a scale per group, rotated in Hadamard
         blocks) into slots of a cache, and slots read back;
  step   queries and keys normed and rotated, keys and values quantized into the cache, in one pass.

`own` selects the framework's calls; otherwise run() computes the plain forms.
"""
import math

import torch

own = False

# Sizes are this repository's own where it has them: 17776 = 226 text tokens + 13 latent frames of
# 30 x 45 patches, 1920 = 30 heads of 64, 1920 -> 5760 projections, 12288 inner features, a text
# encoder of width 4096.  The others are generic.
TEXT, FRAMES, ROWS, COLS = 226, 13, 30, 45


def listed():
    return [
        # one token through a QKV projection: a step of single-token serving, latency counts
        dict(name="w4 one token", op="w4", M=1, K=1920, N=5760, G=128, zero=False, y="bf16"),
        # the modulation projections of 30 blocks, two of 3 x 1920 each, from one conditioning vector
        dict(name="w4 modulation", op="w4", M=1, K=512, N=345600, G=64, zero=True, y="f32"),
        # a few text tokens, odd sizes, small groups
        dict(name="w4 thirteen tokens", op="w4", M=13, K=4096, N=1921, G=32, zero=True, y="bf16"),
        # a batch of 64 tokens through the widest layer
        dict(name="w4 batch", op="w4", M=64, K=12288, N=4096, G=128, zero=False, y="bf16"),
        # one new token in each of 7 sequences at far positions, 96 of 128 elements, scaled frequencies
        dict(name="rope far tokens", op="rope", B=7, T=1, H=24, D=128, R="96", layout="half", far=True, dtype="bf16"),
        # the queries of a whole video in time, row and column; its text tokens are not rotated
        dict(name="rope video", op="rope", B=1, T=17776, H=30, D=64, R="16,24,24", layout="interleaved", far=False,
             dtype="bf16"),
        # a short float32 batch with fewer key heads, heads of 80
        dict(name="qk short f32", op="qk", B=3, T=77, H=20, Hk=4, D=80, R="80", layout="half", far=False, norm="rms",
             dtype="f32"),
        # a whole video's queries and keys where the QKV projection left them: the largest case
        dict(name="qk video", op="qk", B=1, T=17776, H=30, Hk=30, D=64, R="16,24,24", layout="interleaved", far=False,
             norm="layer", dtype="bf16"),
        # one latent frame written in 4 bits, the last four read for the next step
        dict(name="cache frame int4", op="cache", write=1350, read=5400, slots=17776, H=30, D=64, fmt="int4", G=64, had=64,
             y="bf16"),
        # the whole history read back from 8 bits
        dict(name="cache read int8", op="cache", write=0, read=17550, slots=17776, H=30, D=64, fmt="int8", G=32, had=1,
             y="bf16"),
        # one token of single-token serving into the cache
        dict(name="step one token", op="step", B=1, T=1, H=30, Hk=30, D=64, R="64", layout="half", far=True, norm="rms",
             dtype="bf16", fmt="fp8", G=64, had=1, slots=17776),
        # three latent frames into the cache
        dict(name="step frames", op="step", B=1, T=4050, H=30, Hk=30, D=64, R="16,24,24", layout="interleaved", far=False,
             norm="layer", dtype="bf16", fmt="fp8", G=64, had=64, slots=17776),
    ]


def _size(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v))) // step * step or step


def draw(rng):
    op = rng.choice(["w4", "w4", "w4", "w4", "rope", "rope", "qk", "qk", "qk", "cache", "cache", "cache", "step", "step"])
    if op == "w4":
        G = rng.choice([32, 64, 128])
        K, N = _size(rng, 256, 12288, G), _size(rng, 64, 65536)
        while N * K > 345600 * 512:
            N //= 2
        M = rng.choice([1, 1, _size(rng, 2, 16), _size(rng, 2, 64)])
        while M * N * K > 64 * 12288 * 4096 and M > 1:
            M //= 2
        return dict(op=op, M=M, K=K, N=N, G=G, zero=rng.random() < 0.5, y=rng.choice(["bf16", "bf16", "f32"]))
    if op == "cache":
        D = rng.choice([64, 64, 96, 128, 256])
        had = rng.choice([1, 32, D & -D])
        G = rng.choice([32, D & -D, D])
        H = _size(rng, 1, 2048 // D)
        slots = _size(rng, 64, 17776 * 30 * 64 // (H * D) if H * D > 1920 else 17776)
        write = rng.choice([0, 1, _size(rng, 1, slots // 3)])
        y = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, write=write, read=_size(rng, 1, slots // 2 if y == "f32" else slots), slots=slots, H=H, D=D,
                    fmt=rng.choice(["int8", "fp8", "int4"]), G=G, had=min(had, 128), y=y)
    D = rng.choice([64, 64, 80, 96, 128, 128, 256])
    layout = rng.choice(["interleaved", "half"])
    R = rng.choice([f"{D}", f"{D}", f"{D // 2}", f"{D // 4},{D // 8 * 3},{D // 8 * 3}"])
    H = _size(rng, 1, 3840 // D)
    Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0])
    B = rng.choice([1, 1, _size(rng, 1, 32)])
    T = _size(rng, 1, max(1, 17776 * 30 * 64 // (B * H * D)))
    c = dict(op=op, B=B, T=T, H=H, D=D, R=R, layout=layout, far=rng.random() < 0.5)
    if op == "rope":
        return dict(c, dtype=rng.choice(["bf16", "bf16", "f32"]))
    c = dict(c, Hk=Hk, norm=rng.choice(["layer", "rms"]))
    if op == "qk":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(c, dtype=dtype, T=max(1, c["T"] // 2) if dtype == "f32" else c["T"])
    c["T"] = max(1, c["T"] // 2)
    return dict(c, dtype="bf16", fmt="fp8", G=rng.choice([D & -D, D]), had=rng.choice([1, min(128, D & -D)]),
                slots=B * c["T"] + _size(rng, 1, 4096))


# ---- inputs -----------------------------------------------------------------------------------

LEVELS = {"int8": 127.0, "fp8": 448.0, "int4": 7.0}
EPS = 1e-6


def _device():
    return torch.device("cuda:0")


def _generator(seed, stream):
    g = torch.Generator(device=_device())
    g.manual_seed(1000003 * int(seed) + stream)
    return g


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=_device())


def _axes(c):
    """Rotated elements of each position axis."""
    return [int(r) for r in c["R"].split(",")]


def _dtype(c):
    return torch.float32 if c.get("dtype", c.get("y")) == "f32" else torch.bfloat16


def _w4_inputs(c, seed):
    """bf16 tokens with a few large channels; 4-bit codes [N, K / 2] (even elements in the low
    nibbles, 0 to 15), bf16 scales and zero points [N, K / G] of Gaussian weights."""
    M, K, N, G = c["M"], c["K"], c["N"], c["G"]
    gen = _generator(seed, 1)
    x = _randn(gen, M, K)
    x[:, torch.randperm(K, generator=gen, device=_device())[:max(1, K // 100)]] *= 20.0
    w = _randn(gen, N, K // G, G).mul_(0.02)
    if c["zero"]:
        w.add_(_randn(gen, N, K // G, 1).mul_(0.01))
        lo = w.amin(2, keepdim=True).clamp_(max=0.0)
        scale = ((w.amax(2, keepdim=True).clamp_(min=0.0) - lo) / 15.0).to(torch.bfloat16)
        zero = torch.round(-lo / scale.float()).clamp_(0, 15)
    else:
        scale = (w.abs().amax(2, keepdim=True) / 7.0).to(torch.bfloat16)
        zero = torch.full((), 8.0, device=_device())
    u = torch.round(w.div_(scale.float())).add_(zero).clamp_(0, 15).to(torch.uint8).view(N, K)
    return dict(x=x.to(torch.bfloat16), codes=u[:, 0::2] | (u[:, 1::2] << 4), scale=scale.view(N, K // G),
                zero=zero.to(torch.uint8).view(N, K // G) if c["zero"] else None)


def _positions(c, gen):
    """int64 [axes, B, T].  One axis: each sequence has its own first position, far ones past 2^20.
    Three: time, row and column of a video's patches in order, behind its text tokens (negative)."""
    B, T, axes = c["B"], c["T"], len(_axes(c))
    t = torch.arange(T, device=_device()).expand(B, T)
    if axes == 1:
        top = 1 << 20 if c["far"] else 4096
        return (t + torch.randint(0, top, (B, 1), generator=gen, device=_device()) + (top if c["far"] else 0)).unsqueeze(0)
    p = t - TEXT if T > TEXT else t
    if c["far"]:
        p = torch.where(p < 0, p, p + 100000 * ROWS * COLS)
    pos = torch.stack((p // (ROWS * COLS), p // COLS % ROWS, p % COLS))
    return torch.where(p < 0, -1, pos)


def _turns(c):
    """float64 [R / 2]: turns per position of every rotated pair, 10000^(-2 j / axis size) / (2 pi),
    far cases interpolated: slow pairs (less than a turn over 8192 positions) by a factor of 128, fast
    ones (more than 32 turns) not at all, those between in proportion.  And the scale of the result."""
    parts = [torch.arange(0, r, 2, dtype=torch.float64, device=_device()).div_(-r) for r in _axes(c)]
    turns = torch.pow(10000.0, torch.cat(parts)) / (2.0 * math.pi)
    if not c["far"]:
        return turns, 1.0
    ramp = ((8192.0 * turns - 1.0) / 31.0).clamp_(0.0, 1.0)
    return turns * ramp + turns / 128.0 * (1.0 - ramp), 0.1 * math.log(128.0) + 1.0


def _heads_inputs(c, seed):
    """Queries, keys (and values) as views of one projection's output, norm weights, positions."""
    B, T, H, Hk, D = c["B"], c["T"], c["H"], c.get("Hk", 0), c["D"]
    gen = _generator(seed, 2)
    n = H + 2 * Hk
    qkv = (_randn(gen, B, T, n, D) * (0.5 + torch.rand(n, D, generator=gen, device=_device())) +
           0.3 * _randn(gen, n, D)).to(_dtype(c))
    s = {"q": qkv[:, :, :H], "k": qkv[:, :, H:H + Hk], "v": qkv[:, :, H + Hk:]}
    s["positions"] = _positions(c, gen)
    s["turns"], s["scale"] = _turns(c)
    for name in ("q", "k"):
        s[name + "_weight"] = 1.0 + 0.2 * _randn(gen, D)
        s[name + "_bias"] = 0.2 * _randn(gen, D) if c.get("norm") == "layer" else None
    return s


def _cache_inputs(c, seed, H, write):
    """A filled cache: codes [slots, H, D] (INT4: [slots, H, D / 2] bytes, even elements in the low
    nibbles, two's complement), scales [slots, H, D / G]; distinct slots for the new tokens."""
    slots, D, G, fmt = c["slots"], c["D"], c["G"], c["fmt"]
    gen = _generator(seed, 3)
    s = {"slots": torch.randperm(slots, generator=gen, device=_device())[:write]}
    for name in ("k", "v"):
        if fmt == "fp8":
            codes = (_randn(gen, slots, H, D) * 120.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        elif fmt == "int8":
            codes = torch.randint(-127, 128, (slots, H, D), generator=gen, device=_device(), dtype=torch.int8).view(torch.uint8)
        else:
            q = torch.randint(-7, 8, (slots, H, D), generator=gen, device=_device(), dtype=torch.int8).view(torch.uint8) & 15
            codes = q[..., 0::2] | (q[..., 1::2] << 4)
        s[name + "_codes"] = codes
        s[name + "_scale"] = (0.02 + 0.02 * torch.rand(slots, H, D // G, generator=gen, device=_device())) * (7.0 / LEVELS[fmt])
    return s


def _inputs(case, seed):
    c = dict(case)
    if c["op"] == "w4":
        s = _w4_inputs(c, seed)
    elif c["op"] == "cache":
        s = _cache_inputs(c, seed, c["H"], c["write"])
        gen = _generator(seed, 4)
        for name in ("k", "v"):
            x = _randn(gen, c["write"], c["H"], c["D"])
            x[..., ::13] *= 6.0  # channels that stand out, as keys have them
            s[name] = x.to(torch.bfloat16)
        # the new tokens among slots of the past, in no order
        past = torch.randperm(c["slots"], generator=gen, device=_device())
        s["read"] = torch.cat((s["slots"], past))[:c["read"]]
    else:
        s = _heads_inputs(c, seed)
        if c["op"] == "step":
            s.update(_cache_inputs(c, seed, c["Hk"], c["B"] * c["T"]))
    s["case"] = c
    return s


def prepare(case, seed):
    """Inputs of one pass; with the framework's calls also what a program keeps: packed weights,
    rotary plan, cache."""
    s = _inputs(case, seed)
    c = s["case"]
    if own:
        from bit_quantized_video_amd import hdq
        if c["op"] == "w4":
            s["w"] = hdq.w4_pack(s["codes"], s["scale"], s["zero"])
        if c["op"] in ("rope", "qk", "step"):
            layout = hdq.ROPE_HALF if c["layout"] == "half" else hdq.ROPE_INTERLEAVED
            s["rope"] = hdq.Rope(_axes(c), layout, turns=s["turns"], scale=s["scale"])
        if c["op"] in ("cache", "step"):
            fmt = {"int8": hdq.CACHE_INT8, "fp8": hdq.CACHE_FP8, "int4": hdq.CACHE_INT4}[c["fmt"]]
            s["cache"] = hdq.KvCache(c["slots"], s["k_codes"].shape[1], c["D"], fmt, c["G"], c["had"], k_codes=s["k_codes"],
                                     k_scale=s["k_scale"], v_codes=s["v_codes"], v_scale=s["v_scale"])
    return s


# ---- the plain forms --------------------------------------------------------------------------

def _w4(s):
    c = s["case"]
    b = s["codes"]
    u = torch.stack((b & 15, b >> 4), 2).view(c["N"], -1, c["G"]).float()
    z = s["zero"].float().unsqueeze(2) if c["zero"] else 8.0
    w = ((u - z) * s["scale"].float().unsqueeze(2)).view(c["N"], c["K"])
    y = torch.matmul(s["x"].float(), w.t())
    return y if c["y"] == "f32" else y.to(torch.bfloat16)


def _rotary(x, s):
    """float32 [B, T, H, D] rotated; angles in 64 bits."""
    c = s["case"]
    R = sum(_axes(c))
    axis = torch.cat([torch.full((r // 2,), i, device=_device()) for i, r in enumerate(_axes(c))])
    pos = s["positions"]  # [axes, B, T]
    turn = pos.movedim(0, 2)[:, :, axis].double() * s["turns"]
    angle = ((turn - torch.floor(turn)) * (2.0 * math.pi)).unsqueeze(2)
    cos, sin = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * s["scale"]).float()
    if c["layout"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., R:]), 3)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), 4).flatten(3), x[..., R:]), 3)
    return torch.where((pos >= 0).all(0)[:, :, None, None], y, x)


def _head_norm(x, kind, weight, bias):
    x = x.float()
    if kind == "layer":
        x = x - x.mean(3, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(3, keepdim=True) + EPS) * weight
    return y if bias is None else y + bias


def _butterflies(x, had):
    """Rows of float32 x times H_had / sqrt(had) in blocks: butterflies of strides 1, 2, 4, ..."""
    shape, h = x.shape, 1
    while h < had:
        v = x.reshape(-1, 2, h)
        x = torch.stack((v[:, 0] + v[:, 1], v[:, 0] - v[:, 1]), 1)
        h *= 2
    x = x.reshape(shape)
    return x * torch.tensor(1.0 / math.sqrt(had), dtype=torch.float32, device=x.device) if had > 1 else x


def _store(codes, scale, slots, x, c):
    """float32 [tokens, H, D] rotated and quantized into slots of the cache."""
    y = _butterflies(x, c["had"]).unflatten(2, (-1, c["G"]))
    amax, top = y.abs().amax(3, keepdim=True), LEVELS[c["fmt"]]
    live = amax >= 2.0 ** -100
    q = y * torch.where(live, torch.full_like(amax, top) / torch.where(live, amax, 1.0), 0.0)
    q = q.flatten(2)
    if c["fmt"] == "fp8":
        q = q.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        q = torch.round(q).clamp_(-top, top).to(torch.int8).view(torch.uint8)
        if c["fmt"] == "int4":
            q = (q[..., 0::2] & 15) | (q[..., 1::2] << 4)
    codes[slots] = q
    scale[slots] = torch.where(live, amax / top, 0.0).squeeze(3)


def _load(codes, scale, slots, c):
    q = codes[slots]
    if c["fmt"] == "fp8":
        v = q.view(torch.float8_e4m3fn).float()
    elif c["fmt"] == "int8":
        v = q.view(torch.int8).float()
    else:
        q = torch.stack((q & 15, q >> 4), 3).flatten(2).to(torch.int8)
        v = torch.where(q > 7, q - 16, q).float()
    v = (v.unflatten(2, (-1, c["G"])) * scale[slots].unsqueeze(3)).flatten(2)
    return _butterflies(v, c["had"]).to(_dtype(c))


def _run_plain(s):
    c = s["case"]
    if c["op"] == "w4":
        return _w4(s)
    if c["op"] == "rope":
        return _rotary(s["q"].float(), s).to(_dtype(c))
    if c["op"] == "cache":
        if c["write"]:
            for name in ("k", "v"):
                _store(s[name + "_codes"], s[name + "_scale"], s["slots"], s[name].float(), c)
        return [_load(s[name + "_codes"], s[name + "_scale"], s["read"], c) for name in ("k", "v")]
    q = _rotary(_head_norm(s["q"], c["norm"], s["q_weight"], s["q_bias"]), s).to(_dtype(c))
    k = _rotary(_head_norm(s["k"], c["norm"], s["k_weight"], s["k_bias"]), s)
    if c["op"] == "qk":
        return {"q": q, "k": k.to(_dtype(c))}
    _store(s["k_codes"], s["k_scale"], s["slots"], k.flatten(0, 1), c)
    _store(s["v_codes"], s["v_scale"], s["slots"], s["v"].float().flatten(0, 1), c)
    return _step_outputs(q, s)


def _step_outputs(q, s):
    """The queries and the cache, its codes as the FP8 values they are."""
    f8 = torch.float8_e4m3fn
    return {"q": q, "k": s["k_codes"].view(f8), "k_scale": s["k_scale"], "v": s["v_codes"].view(f8), "v_scale": s["v_scale"]}


# ---- the framework's calls --------------------------------------------------------------------

def _run_own(s):
    from bit_quantized_video_amd import hdq
    c = s["case"]
    if c["op"] == "w4":
        return hdq.w4_linear(s["x"], s["w"], y_dtype=hdq.DTYPE_F32 if c["y"] == "f32" else hdq.DTYPE_BF16)
    if c["op"] == "rope":
        return hdq.rope(s["q"], s["positions"], s["rope"])
    if c["op"] == "cache":
        if c["write"]:
            hdq.cache_write(s["cache"], s["k"], s["v"], s["slots"])
        return list(hdq.cache_read(s["cache"], s["read"], y_dtype=hdq.DTYPE_F32 if c["y"] == "f32" else hdq.DTYPE_BF16))
    norm = hdq.HEAD_NORM_LAYER if c["norm"] == "layer" else hdq.HEAD_NORM_RMS
    weights = (s["q_weight"], s["k_weight"], s["q_bias"], s["k_bias"])
    if c["op"] == "qk":
        q, k = hdq.qk_norm_rope(s["q"], s["k"], norm, *weights, eps=EPS, positions=s["positions"], rope=s["rope"])
        return {"q": q, "k": k}
    q = hdq.qkv_to_cache(s["cache"], s["q"], s["k"], s["v"], s["slots"], norm, *weights, eps=EPS, positions=s["positions"],
                         rope=s["rope"])
    return _step_outputs(q, s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ------------------------------------------------------------

def _cache_token_bytes(c, H):
    """Codes and scales of one token's keys and values."""
    return 2 * H * (c["D"] // (2 if c["fmt"] == "int4" else 1) + 4 * (c["D"] // c["G"]))


def work(case):
    """Inputs read once, outputs written once; two operations per multiply-add, six per rotated or
    normed element, log2(had) additions per Hadamard-rotated one and four per coded one."""
    c = case
    if c["op"] == "w4":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": N * K // 2 + N * (K // c["G"]) * (3 if c["zero"] else 2) + 2 * M * K + M * N * (4 if c["y"] == "f32" else 2),
                "flops": 2.0 * M * N * K}
    if c["op"] == "cache":
        e, each = 2 * c["H"] * c["D"], _cache_token_bytes(c, c["H"])
        return {"bytes": c["write"] * (2 * e + each + 8) + c["read"] * (e * (4 if c["y"] == "f32" else 2) + each + 8),
                "flops": (c["write"] + c["read"]) * e * (4.0 + math.log2(c["had"]))}
    tokens, size = c["B"] * c["T"], 4 if c["dtype"] == "f32" else 2
    e = tokens * (c["H"] + (c["Hk"] if c["op"] == "qk" else 0)) * c["D"]
    nbytes, flops = 2 * e * size + 8 * tokens * len(_axes(c)), 6.0 * e * (1 if c["op"] == "rope" else 2)
    if c["op"] == "step":
        kv = tokens * 2 * c["Hk"] * c["D"]
        nbytes += kv * size + tokens * (_cache_token_bytes(c, c["Hk"]) + 8)
        flops += 6.0 * kv + kv * (4.0 + math.log2(c["had"]))
    return {"bytes": nbytes, "flops": flops}


# ---- the definition in 64 bits ----------------------------------------------------------------

def _rotary_64(x, c, s):
    """float64 [B, T, H, D]: pairs as complex numbers times scale e^(i angle)."""
    R, first = sum(_axes(c)), 0
    out = x.clone()
    live = (s["positions"] >= 0).all(0)[:, :, None, None]
    for i, r in enumerate(_axes(c)):
        pairs = torch.arange(first // 2, (first + r) // 2, device=_device())
        ia, ib = (pairs, pairs + R // 2) if c["layout"] == "half" else (2 * pairs, 2 * pairs + 1)
        turn = s["positions"][i].double().unsqueeze(2) * s["turns"][pairs]
        e = torch.polar(torch.full_like(turn, s["scale"]), 2.0 * math.pi * torch.frac(turn)).unsqueeze(2)
        z = torch.complex(x[..., ia], x[..., ib]) * e
        out[..., ia], out[..., ib] = z.real, z.imag
        first += r
    return torch.where(live, out, x)


def _head_norm_64(x, kind, weight, bias):
    x = x.double()
    mean = x.mean(3, keepdim=True) if kind == "layer" else 0.0
    y = (x - mean) / torch.sqrt((x - mean).square().mean(3, keepdim=True) + EPS) * weight.double()
    return y if bias is None else y + bias.double()


def _hadamard_64(x, had):
    h = torch.ones(1, 1, dtype=torch.float64, device=_device())
    while h.shape[0] < had:
        h = torch.kron(torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64, device=_device()), h)
    return (x.unflatten(2, (-1, had)) @ (h / math.sqrt(had))).flatten(2)


def _e4m3_64(t):
    """Nearest E4M3 value of |t| <= 448 in float64, ties to even: steps of 2^(e - 3), at least 2^-9."""
    _, e = torch.frexp(t)  # |t| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(t), (e - 1).clamp_(min=-6) - 3)
    return torch.round(t / step) * step


def _quantize_64(x, c):
    """(code values, scales) of float64 [tokens, H, D]."""
    y = _hadamard_64(x, c["had"]).unflatten(2, (-1, c["G"]))
    top = LEVELS[c["fmt"]]
    amax = y.abs().amax(3, keepdim=True)
    t = y * (top / amax)
    return (_e4m3_64(t) if c["fmt"] == "fp8" else torch.round(t)).flatten(2), (amax / top).squeeze(3)


def _code_values_64(codes, c):
    if c["fmt"] == "fp8":
        return codes.view(torch.float8_e4m3fn).double()
    if c["fmt"] == "int8":
        return codes.view(torch.int8).double()
    q = torch.stack((codes % 16, codes // 16), 3).flatten(2).double()
    return (q + 8.0) % 16.0 - 8.0


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "w4":
        out = []
        for r in range(0, c["N"], 32768):  # a slice of the rows at a time: 64-bit weights are large
            b = s["codes"][r:r + 32768].long()
            u = torch.stack((b % 16, b // 16), 2).flatten(1).double()
            each = lambda t: t[r:r + 32768].double().repeat_interleave(c["G"], 1)
            out.append(s["x"].double() @ ((u - (each(s["zero"]) if c["zero"] else 8.0)) * each(s["scale"])).t())
        return torch.cat(out, 1)
    if c["op"] == "rope":
        return _rotary_64(s["q"].double(), c, s)
    if c["op"] == "cache":
        out = []
        for name in ("k", "v"):
            v, scale = _code_values_64(s[name + "_codes"], c), s[name + "_scale"].double()
            if c["write"]:
                v[s["slots"]], scale[s["slots"]] = _quantize_64(s[name].double(), c)
            v = v[s["read"]] * scale[s["read"]].repeat_interleave(c["G"], 2)
            out.append(_hadamard_64(v, c["had"]))
        return out
    q = _rotary_64(_head_norm_64(s["q"], c["norm"], s["q_weight"], s["q_bias"]), c, s)
    k = _rotary_64(_head_norm_64(s["k"], c["norm"], s["k_weight"], s["k_bias"]), c, s)
    if c["op"] == "qk":
        return {"q": q, "k": k}
    out = {"q": q}
    for name, x in (("k", k), ("v", s["v"].double())):
        v, scale = _code_values_64(s[name + "_codes"], c), s[name + "_scale"].double()
        v[s["slots"]], scale[s["slots"]] = _quantize_64(x.flatten(0, 1), c)
        out[name], out[name + "_scale"] = v, scale
    return out
