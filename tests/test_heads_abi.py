"""CPU checks of the 4-bit layer's, the head norms' and the key-value cache's
entry points: struct layouts, sizes, rotary frequencies, packing, and every
refusal, before any launch."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

import heads_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "hdq.h")
FAKE = 0x100000   # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def hdq():
    from bit_quantized_video_amd import hdq as H
    return H


def test_structs_match_the_header(hdq, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not found")
    structs = {"hdq_w4_tensor": hdq.W4TensorDesc, "hdq_heads": hdq.HeadsDesc, "hdq_head_norm": hdq.HeadNormDesc,
               "hdq_rope": hdq.RopeDesc, "hdq_kv_cache": hdq.KvCacheDesc}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "hdq.h"', "int main(void) {"]
    for c, cls in structs.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f[0]} %zu\\n", offsetof({c}, {f[0]}));' for f in cls._fields_]
    (tmp_path / "s.c").write_text("\n".join(lines) + "return 0; }")
    subprocess.check_call(["gcc", "-I", os.path.dirname(HEADER), str(tmp_path / "s.c"), "-o", str(tmp_path / "s")])
    got = dict(ln.split() for ln in subprocess.check_output([str(tmp_path / "s")], text=True).splitlines())
    for c, cls in structs.items():
        assert int(got[c]) == ctypes.sizeof(cls), c
        for f in cls._fields_:
            assert int(got[f"{c}.{f[0]}"]) == getattr(cls, f[0]).offset, (c, f[0])


def test_constants_match_the_header(hdq):
    text = open(HEADER).read()
    names = [n for n in dir(hdq) if re.match(r"(W4|HEAD|ROPE|CACHE)_", n)]
    assert len(names) >= 20
    for n in names:
        m = re.search(rf"#define HDQ_{n} \(?([\d <]+)\)?", text)
        assert m and eval(m.group(1)) == getattr(hdq, n), n


def test_w4_bytes(hdq):
    assert hdq.lib.hdq_w4_bytes(1, 32, 32, 0) == 1024 and hdq.lib.hdq_w4_bytes(17, 160, 32, 0) == 4 * 1024
    assert hdq.lib.hdq_w4_bytes(17, 160, 32, 1) == 2 * 512 and hdq.lib.hdq_w4_bytes(17, 160, 32, 2) == 2 * 256
    assert hdq.lib.hdq_w4_bytes(5760, 1920, 128, 0) == 5760 * 1920 // 2
    assert hdq.lib.hdq_w4_bytes(1 << 27, 1 << 22, 64, 0) == 1 << 48
    for bad in ((0, 32, 32, 0), (1, 0, 32, 0), (1, 48, 32, 0), (1, 64, 16, 0), (1, 160, 64, 0), (1, 64, 64, 3),
                ((1 << 27) + 1, 64, 64, 0), (1, (1 << 22) + 32, 32, 0)):
        assert hdq.lib.hdq_w4_bytes(*bad) == 0, bad


def test_w4_pack_reference_is_a_bijection():
    """The reference packing keeps every code (all nibbles present once)."""
    codes, scale, zero = R.w4_random(33, 160, 32, True, 1)
    p, s, z = R.w4_pack(codes, scale, zero, 32)
    w = sum(p.view(-1, 4)[:, i].long() << (8 * i) for i in range(4))
    w = (w >> 3) | ((w & 7) << 29)                # the words are kept rotated
    u = torch.bincount(torch.stack([(w >> (4 * i)) & 15 for i in range(8)]).flatten(), minlength=16)
    want = torch.bincount(R.w4_values(codes).flatten().long(), minlength=16)
    want[0] += p.numel() * 2 - want.sum()
    assert torch.equal(u, want)
    # row 17, column 43: tile row 1, lane 17 % 16 + 16 * (43 / 8 % 4), word 43 / 32, nibble of 43 % 8 = 3
    lane, word, nib = 1 + 16 * (43 // 8 % 4), 43 // 32, (3 >> 1) + 4 * (3 & 1)
    assert (int(w[((1 * 2 + 0) * 64 + lane) * 4 + word]) >> (4 * nib)) & 15 == int(R.w4_values(codes)[17, 43])
    assert s[(1 * 16 + 1) * 16 + 4] == scale[17, 4] and z[(1 * 16 + 1) * 16 + 1] == zero[17, 1]
    assert s.numel() == 3 * 256 and z.numel() == 3 * 256


def test_w4_refusals(hdq):
    L, T = hdq.lib, hdq.W4TensorDesc
    ok = T(100, 128, 64, FAKE, FAKE, None)
    lin = lambda w=ok, x=FAKE, M=3, y=FAKE, t=1, ws=None, n=0: L.hdq_w4_linear(x, M, w, y, t, ws, n, None)
    need, big = L.hdq_w4_linear_workspace_bytes(64, 100, 4096), T(100, 4096, 64, FAKE, FAKE, None)
    assert need >= 2 * 64 * 100 * 4 and L.hdq_w4_linear_workspace_bytes(1, 100, 32640) == 0
    assert lin(big, M=64) == hdq.ERR_WORKSPACE and lin(big, M=64, ws=FAKE, n=need - 1) == hdq.ERR_WORKSPACE
    assert lin(big, M=64, ws=FAKE + 8, n=need) == hdq.ERR_SHAPE
    for bad in ((0, 100, 4096), (64, 0, 4096), (64, 100, 40), ((1 << 20) + 1, 100, 64)):
        assert L.hdq_w4_linear_workspace_bytes(*bad) == 0, bad
    assert lin(x=None) == hdq.ERR_INVALID and lin(y=None) == hdq.ERR_INVALID and lin(w=None) == hdq.ERR_INVALID
    assert lin(t=2) == hdq.ERR_UNSUPPORTED
    assert lin(M=-1) == hdq.ERR_SHAPE and lin(M=(1 << 20) + 1) == hdq.ERR_SHAPE
    assert lin(x=FAKE + 2) == hdq.ERR_SHAPE and lin(y=FAKE + 1) == hdq.ERR_SHAPE and lin(y=FAKE + 2, t=0) == hdq.ERR_SHAPE
    assert lin(M=0) == hdq.OK and lin(M=0, x=None, y=None) == hdq.OK
    for w in (T(0, 128, 64, FAKE, FAKE, None), T(100, 96, 64, FAKE, FAKE, None), T(100, 128, 16, FAKE, FAKE, None),
              T(100, 128, 64, FAKE + 8, FAKE, None), T(100, 128, 64, FAKE, FAKE + 4, None), T(100, 128, 64, FAKE, FAKE, FAKE + 2),
              T(100, 128, 64, FAKE, FAKE + 8, None), T(100, 128, 64, FAKE, FAKE, FAKE + 8)):
        assert lin(w=w) == hdq.ERR_SHAPE and L.hdq_w4_quantize(FAKE, w, None) == hdq.ERR_SHAPE
        zero = FAKE if w.zero else None
        assert L.hdq_w4_pack(FAKE, FAKE, zero, w, None) == hdq.ERR_SHAPE
    for w in (T(100, 128, 64, None, FAKE, None), T(100, 128, 64, FAKE, None, None)):
        assert lin(w=w) == hdq.ERR_INVALID
    assert L.hdq_w4_pack(FAKE, FAKE, FAKE, ok, None) == hdq.ERR_INVALID          # zero points without a place
    assert L.hdq_w4_pack(None, FAKE, None, ok, None) == hdq.ERR_INVALID
    assert L.hdq_w4_pack(FAKE + 2, FAKE, None, ok, None) == hdq.ERR_SHAPE
    assert L.hdq_w4_quantize(None, ok, None) == hdq.ERR_INVALID and L.hdq_w4_quantize(FAKE + 8, ok, None) == hdq.ERR_SHAPE
    for bad in ((10, 100, 128), (10, 128, 48)):
        with pytest.raises(ValueError):
            hdq.W4Weights(*bad, device="cpu")
    codes, scale = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.bfloat16)
    for args in ((codes, scale), (codes.int(), scale), (codes, scale[:, :0]), (codes, scale.float()), (codes, scale[:3]),
                 (codes, scale, scale), (codes, scale.repeat(1, 100)), (codes[:, :0], scale)):
        with pytest.raises(ValueError):           # wrong operands, and (the first) not on a GPU
            hdq.w4_pack(*args)


@pytest.mark.parametrize("dim", [2, 6, 64, 512])
def test_rope_turns(hdq, dim):
    j = torch.arange(0, dim, 2, dtype=torch.float64)
    plain = 10000.0 ** (-j / dim) / (2 * math.pi)
    same = lambda a, b: bool(((a - b).abs() <= 4 * 2.0 ** -52 * b).all())      # pow, a division, a blend
    assert same(hdq.rope_turns(dim), plain)
    assert same(hdq.rope_turns(dim, scaling=hdq.ROPE_SCALE_LINEAR, factor=8.0), plain / 8)
    assert same(hdq.rope_turns(dim, 5e5), 5e5 ** (-j / dim) / (2 * math.pi))
    r = hdq.rope_turns(dim, scaling=hdq.ROPE_SCALE_RAMP, factor=16.0, length=4096.0, ramp=(1.0, 32.0))
    g = ((4096 * plain - 1) / 31).clamp(0, 1)
    assert bool(((r - (plain * g + plain / 16 * (1 - g))).abs() <= 16 * 2.0 ** -52 * plain).all())
    if dim > 2:
        b = hdq.rope_turns(dim, scaling=hdq.ROPE_SCALE_BASE, factor=8.0)
        assert abs(float(b[0] / plain[0]) - 1) < 1e-15 and abs(float(b[-1] * 8 / plain[-1]) - 1) < 1e-12


def test_rope_turns_refusals(hdq):
    out = (ctypes.c_double * 256)()
    f = lambda dim=8, base=1e4, kind=0, factor=2.0, length=10.0, slow=1.0, fast=2.0, o=out: hdq.lib.hdq_rope_turns(
        dim, base, kind, factor, length, slow, fast, o)
    assert f() == hdq.OK and f(o=None) == hdq.ERR_INVALID
    for dim in (0, -2, 7, 514):
        assert f(dim=dim) == hdq.ERR_SHAPE
    assert f(dim=2, kind=2) == hdq.ERR_SHAPE
    for kw in (dict(kind=4), dict(kind=-1), dict(base=0.0), dict(base=math.inf), dict(base=math.nan), dict(kind=1, factor=0.5),
               dict(kind=1, factor=math.nan), dict(kind=2, factor=math.inf), dict(kind=3, length=0.0), dict(kind=3, slow=2.0),
               dict(kind=3, slow=-1.0), dict(kind=3, fast=math.inf), dict(kind=3, length=math.nan)):
        assert f(**kw) == hdq.ERR_INVALID, kw
    with pytest.raises(hdq.HdqError):
        hdq.rope_turns(7)


def heads(hdq, data=FAKE, dtype=1, n=4, b=4096, t=256, h=64):
    return hdq.HeadsDesc(data, dtype, n, b, t, h)


def rope(hdq, layout=0, dim=64, axes=1, dims=(64, 0, 0), scale=1.0, turns=FAKE, pos=FAKE, st=(0, 0, 1)):
    return hdq.RopeDesc(layout, dim, axes, (ctypes.c_int32 * 3)(*dims), scale, turns, pos, *st)


def test_qk_norm_rope_refusals(hdq):
    H = lambda **kw: heads(hdq, **kw)
    P = lambda **kw: rope(hdq, **kw)

    def f(q=H(), k=H(), b=2, t=16, dim=64, norm=None, rope=None, qo=H(), ko=H()):
        return hdq.lib.hdq_qk_norm_rope(q, k, b, t, dim, norm, rope, qo, ko, None)
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(q=H(data=None)), dict(ko=H(data=None))):
        assert f(**kw) == hdq.ERR_INVALID, kw
    for kw in (dict(q=H(dtype=2)), dict(q=H(dtype=0)), dict(ko=H(dtype=0)), dict(qo=H(dtype=7))):
        assert f(**kw) == hdq.ERR_UNSUPPORTED, kw
    for kw in (dict(dim=0), dict(dim=513), dict(b=-1), dict(t=-1), dict(b=1 << 16, t=1 << 15), dict(q=H(n=0)), dict(qo=H(n=5)),
               dict(ko=H(n=3)), dict(q=H(n=(1 << 20) + 1)), dict(q=H(n=1 << 20), qo=H(n=1 << 20)), dict(q=H(b=-1)), dict(q=H(t=-64)),
               dict(q=H(h=1 << 41)), dict(qo=H(h=32)), dict(qo=H(t=0)), dict(qo=H(b=0)), dict(q=H(data=FAKE + 1))):
        assert f(**kw) == hdq.ERR_SHAPE, kw
    # strides of an output's single elements do not count
    assert f(b=0) == hdq.OK and f(t=0, q=H(data=None)) == hdq.OK

    N = hdq.HeadNormDesc
    for kind, eps in ((3, 1e-6), (-1, 1e-6), (1, -1e-6), (2, math.nan), (2, math.inf)):
        assert f(norm=N(kind, eps, None, None, None, None)) == hdq.ERR_INVALID
    assert f(norm=N(1, 0.0, FAKE + 2, None, None, None)) == hdq.ERR_SHAPE
    for kw in (dict(layout=2), dict(turns=None), dict(pos=None), dict(scale=math.nan), dict(scale=math.inf)):
        assert f(rope=P(**kw)) == hdq.ERR_INVALID, kw
    for kw in (dict(dim=66, dims=(66, 0, 0)), dict(dim=-2, dims=(-2, 0, 0)), dict(dim=7, dims=(7, 0, 0)), dict(axes=0), dict(axes=4),
               dict(dims=(62, 0, 0)), dict(axes=2, dims=(33, 31, 0)), dict(axes=2, dims=(68, -4, 0)), dict(turns=FAKE + 4),
               dict(pos=FAKE + 4), dict(st=(0, -1, 1))):
        assert f(rope=P(**kw)) == hdq.ERR_SHAPE, kw


def cache(hdq, fmt=1, group=64, had=64, n=4, dim=64, slots=100, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE):
    return hdq.KvCacheDesc(fmt, group, had, n, dim, slots, kc, ks, vc, vs)


def test_cache_refusals(hdq):
    H = lambda **kw: heads(hdq, **kw)
    C = lambda **kw: cache(hdq, **kw)

    def write(q=H(), k=H(), v=H(), b=2, t=16, norm=None, rope=None, qo=H(), slots=FAKE, c=C()):
        return hdq.lib.hdq_qkv_to_cache(q, k, v, b, t, norm, rope, qo, slots, c, None)

    def read(c=C(), slots=FAKE, n=5, ko=FAKE, vo=FAKE, t=1):
        return hdq.lib.hdq_cache_read(c, slots, n, ko, vo, t, None)
    for f in (write, read):
        assert f(c=None) == hdq.ERR_INVALID and f(slots=None) == hdq.ERR_INVALID
        for kw in (dict(kc=None), dict(ks=None), dict(vc=None), dict(vs=None)):
            assert f(c=C(**kw)) == hdq.ERR_INVALID, kw
        assert f(c=C(fmt=3)) == hdq.ERR_UNSUPPORTED
        for kw in (dict(group=48), dict(group=4), dict(group=128), dict(group=0), dict(had=3), dict(had=256), dict(had=0),
                   dict(dim=60, group=60, had=4), dict(dim=520, group=520, had=8), dict(dim=72, group=72, had=16), dict(n=0),
                   dict(n=(1 << 19) + 1), dict(slots=-1), dict(slots=1 << 40), dict(kc=FAKE + 4), dict(vs=FAKE + 2)):
            assert f(c=C(**kw)) == hdq.ERR_SHAPE, kw
        assert f(slots=FAKE + 4) == hdq.ERR_SHAPE
    for kw in (dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(v=H(data=None))):
        assert write(**kw) == hdq.ERR_INVALID, kw
    for kw in (dict(v=H(dtype=0)), dict(q=H(dtype=0)), dict(k=H(dtype=2))):
        assert write(**kw) == hdq.ERR_UNSUPPORTED, kw
    for kw in (dict(k=H(n=3)), dict(v=H(n=5)), dict(qo=H(n=5)), dict(b=-1), dict(qo=H(h=8)), dict(b=1 << 16, t=1 << 16)):
        assert write(**kw) == hdq.ERR_SHAPE, kw
    assert write(b=0, slots=None) == hdq.OK and read(n=0, slots=None, ko=None, vo=None) == hdq.OK
    for kw in (dict(ko=None), dict(vo=None)):
        assert read(**kw) == hdq.ERR_INVALID
    for kw in (dict(n=-1), dict(n=1 << 31), dict(ko=FAKE + 8), dict(vo=FAKE + 2)):
        assert read(**kw) == hdq.ERR_SHAPE
    assert read(t=2) == hdq.ERR_UNSUPPORTED


def test_binding_refusals(hdq):
    x = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    r = hdq.Rope(64, turns=hdq.rope_turns(64))
    pos = torch.arange(5)
    with pytest.raises(ValueError):
        hdq.rope(x, pos, r)                       # not on a GPU
    for bad in (x.half(), x[..., ::2], x[0]):
        with pytest.raises(ValueError):
            hdq.rope(bad, pos, r)
    for args in ((63,), ((2, 2, 2, 2),), ((),), (64, 7), (0,)):
        with pytest.raises(ValueError):
            hdq.Rope(*args, turns=torch.zeros(1, dtype=torch.float64))
    with pytest.raises(ValueError):
        hdq.Rope(64, turns=torch.zeros(32))
    dev = torch.device("cpu")
    r3 = hdq.Rope((16, 24, 24), turns=torch.cat([hdq.rope_turns(d) for d in (16, 24, 24)]))
    desc = lambda rope, p: hdq.RopeDesc.from_buffer_copy(rope.desc(p, 2, 5, dev))
    d = desc(r3, torch.zeros(3, 2, 5, dtype=torch.int64))
    assert list(d.axis_dim) == [16, 24, 24] and (d.layout, d.dim, d.axes, d.scale) == (hdq.ROPE_INTERLEAVED, 64, 3, 1.0)
    assert d.turns == r3.turns.data_ptr()
    d = desc(r3, torch.zeros(3, 5, dtype=torch.int64))
    assert (d.pos_axis_stride, d.pos_batch_stride, d.pos_token_stride) == (5, 0, 1)
    d = desc(r, torch.zeros(5, 2, dtype=torch.int64).t())
    assert (d.pos_batch_stride, d.pos_token_stride) == (1, 2)
    for packed, cls in ((hdq._HEADS, hdq.HeadsDesc), (hdq._NORM, hdq.HeadNormDesc), (hdq._ROPE, hdq.RopeDesc)):
        assert packed.size == ctypes.sizeof(cls)
    h = hdq.HeadsDesc.from_buffer_copy(hdq._heads(x[:, 1:3], "x", 2, 64, dev))
    assert (h.data, h.dtype, h.heads, h.batch_stride, h.token_stride, h.head_stride) == (x[:, 1:].data_ptr(), 1, 2, 0, 256, 64)
    n = hdq.HeadNormDesc.from_buffer_copy(hdq._head_norm(2, 0.5, 64, dev, None, r.turns[:0].new_zeros(64).float(), None, None))
    assert (n.kind, n.eps, n.q_weight, n.k_bias) == (2, 0.5, None, None) and n.q_bias
    for p in (pos.int(), torch.zeros(4, dtype=torch.int64), torch.zeros(2, 5, 1, dtype=torch.int64)):
        with pytest.raises(ValueError):
            r.desc(p, 2, 5, dev)
    for kw in (dict(fmt=3), dict(group=48), dict(group=0), dict(dim=60)):
        with pytest.raises(ValueError):
            hdq.KvCache(10, 2, **dict(dict(dim=64, device="cpu"), **kw))
    c = hdq.KvCache(10, 4, 64, device="cpu")
    assert c.k_codes.shape == (10, 4, 64) and c.v_scale.shape == (10, 4, 1)
    k, slots = x, torch.arange(5)
    for args in ((c, None, k, k, slots), (c, None, k, None, slots), (c, None, k[:, :3], k[:, :3], slots), (c, None, k, k[:4], slots)):
        with pytest.raises(ValueError):
            hdq.qkv_to_cache(*args)
    for s in (slots.int(), torch.arange(10)[::2], slots):
        with pytest.raises(ValueError):
            hdq.cache_read(c, s)
