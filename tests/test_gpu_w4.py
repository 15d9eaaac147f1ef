"""The 4-bit group-scaled layer on the GPU against float64; packing and
quantization bit for bit; and one serving step through all of it."""
import math

import pytest
import torch

import heads_ref as R
from test_gpu_heads import BF, DEV, F32, make, plan, reference

pytestmark = pytest.mark.gpu
from bit_quantized_video_amd import hdq  # noqa: E402


def check(y, x, codes, scale, zero, group):
    ref, tol = R.w4_linear(x, codes, scale, zero, group)
    assert R.close(y, ref, tol)
    if float(ref.norm()) > 0:
        # the bounds above are worst cases; sums of differences from 24 or so lose a dozen float32 roundings
        assert float((y.cpu().double() - ref).norm() / ref.norm()) <= R.HALF[y.dtype] + 64 * R.U


@pytest.mark.parametrize("M,N,K,group", [
    (1, 1, 32, 32), (1, 5760, 1920, 128), (1, 16, 128, 128), (2, 17, 96, 32), (1, 100, 160, 32), (3, 15, 64, 64), (13, 1921, 4096, 32),
    (16, 33, 192, 64), (17, 48, 1024, 128), (31, 64, 12288, 128), (33, 257, 320, 64), (64, 130, 4096, 128), (48, 1, 2048, 32),
    (65, 95, 256, 64), (130, 31, 384, 128), (1, 40000, 512, 64), (5, 3, 8192, 64), (300, 1000, 128, 32)])
@pytest.mark.parametrize("zero", [False, True])
def test_linear(M, N, K, group, zero):
    codes, scale, z = R.w4_random(N, K, group, zero, M + N)
    x = make((M, K), BF, 1)
    w = hdq.w4_pack(codes.to(DEV), scale.to(DEV), z.to(DEV) if zero else None)
    for code, dt in ((hdq.DTYPE_BF16, BF), (hdq.DTYPE_F32, F32)):
        y = hdq.w4_linear(x.to(DEV), w, y_dtype=code)
        assert y.dtype == dt and y.shape == (M, N)
        check(y, x, codes, scale, z, group)
    assert torch.equal(hdq.w4_linear(x.to(DEV), w), hdq.w4_linear(x.to(DEV), w))


@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (33, 160, 32), (16, 128, 128), (50, 192, 64), (200, 1920, 128)])
@pytest.mark.parametrize("zero", [False, True])
def test_pack_and_quantize(N, K, group, zero):
    codes, scale, z = R.w4_random(N, K, group, zero, 2)
    got = hdq.w4_pack(codes.to(DEV), scale.to(DEV), z.to(DEV) if zero else None)
    for have, want in zip((got.codes, got.scale, got.zero), R.w4_pack(codes, scale, z, group)):
        assert have is None and want is None or torch.equal(have.cpu(), want)
    w = make((N, K), BF, 3, 0.02)
    w[0, :group] = 0
    if N > 20:
        w[3, :group] = w[3, :group].abs() + 0.01          # one sign alone
        w[5, 0], w[7, group - 1], w[9, :group] = math.nan, math.inf, 1e-38
        w[11, 0], w[11, 1] = 3e38, -3e38
    q = hdq.w4_quantize(w.to(DEV), group, zero)
    for have, want in zip((q.codes, q.scale, q.zero), R.w4_pack(*R.w4_quantize(w, group, zero), group)):
        if want is not None:
            assert torch.equal(torch.nan_to_num(have.cpu().float(), 7.0), torch.nan_to_num(want.float(), 7.0))


def test_large_zero_points():
    """Zero points past 15 (checkpoints that store z + 1) are taken as they are."""
    codes, scale, z = R.w4_random(40, 256, 64, True, 4)
    z = (z.int() * 17).to(torch.uint8)
    x = make((2, 256), BF, 5)
    w = hdq.w4_pack(codes.to(DEV), scale.to(DEV), z.to(DEV))
    check(hdq.w4_linear(x.to(DEV), w, y_dtype=hdq.DTYPE_F32), x, codes, scale, z, 64)


def test_non_finite():
    """NaN and infinities stay in their token (x) or row (scales); padding rows and columns hold none."""
    codes, scale, _ = R.w4_random(37, 160, 32, False, 6)
    x = make((18, 160), BF, 7)
    x[3, 5], x[17, 159] = math.nan, math.inf
    scale[20, 1] = math.nan
    y = hdq.w4_linear(x.to(DEV), hdq.w4_pack(codes.to(DEV), scale.to(DEV))).cpu()
    ok = torch.ones(18, 37, dtype=torch.bool)
    ok[3], ok[17], ok[:, 20] = False, False, False
    assert bool(torch.isfinite(y[ok]).all()) and bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[:, 20]).all())
    assert not bool(torch.isfinite(y[17]).any())


def test_output_and_empty():
    codes, scale, _ = R.w4_random(37, 128, 64, False, 8)
    w = hdq.w4_pack(codes.to(DEV), scale.to(DEV))
    x = make((5, 128), BF, 9).to(DEV)
    room = torch.full((7 * 37 + 1,), 7.0, dtype=BF, device=DEV)
    y = room[1:1 + 5 * 37].view(5, 37)                   # element-aligned, nothing written around it
    assert hdq.w4_linear(x, w, y=y) is y and torch.equal(y, hdq.w4_linear(x, w))
    assert float(room[0]) == 7.0 and bool((room[1 + 5 * 37:] == 7.0).all())
    assert hdq.w4_linear(x[:0], w).shape == (0, 37)
    for bad in (dict(y=torch.empty(5, 38, dtype=BF, device=DEV)), dict(y=torch.empty(5, 37, device=DEV))):
        with pytest.raises(ValueError):
            hdq.w4_linear(x, w, **bad)
    with pytest.raises(ValueError):
        hdq.w4_linear(x[:, :64].contiguous(), w)


def test_weights_past_32_bits():
    """More than 2^32 bytes of codes: the last rows, decoded from the packed bytes."""
    N, K, group = 16 * 4100 + 3, 128 * 1100, 128
    w = hdq.W4Weights(N, K, group, device=DEV)
    assert w.codes.numel() > 1 << 32
    w.codes.zero_()
    w.scale.fill_(0.01)
    tail = 1100 * 1024
    w.codes[-tail:] = torch.randint(0, 256, (tail,), device=DEV, dtype=torch.uint8)
    x = make((1, K), BF, 10)
    y = hdq.w4_linear(x.to(DEV), w, y_dtype=hdq.DTYPE_F32).cpu()
    t = w.codes[-tail:].cpu().view(1100, 4, 16, 4, 4)[:, :, :3].long()    # [tile k][quarter][row][word][byte], the last tile's three rows
    t = sum(t[..., i] << (8 * i) for i in range(4))
    t = (t >> 3) | ((t & 7) << 29)
    u = torch.stack([(t >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15 for e in range(8)], -1).to(torch.uint8)
    u = u.permute(2, 0, 3, 1, 4).reshape(3, K)
    codes, scale = u[:, 0::2] | (u[:, 1::2] << 4), torch.full((3, K // group), 0.01, dtype=BF)
    check(y[:, -3:], x, codes, scale, None, group)
    # zero codes are -8
    want = -8 * float(scale[0, 0]) * x.double().sum()
    bound = 24 * (group + 10 + K / group) * R.U * float(scale[0, 0]) * float(x.double().abs().sum())
    assert float((y[:, :-3].double() - want).abs().max()) <= bound


def test_stream_and_graph():
    codes, scale, z = R.w4_random(300, 512, 64, True, 11)
    w = hdq.w4_pack(codes.to(DEV), scale.to(DEV), z.to(DEV))
    x = make((4, 512), BF, 12).to(DEV)
    want = hdq.w4_linear(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = hdq.w4_linear(x, w, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = hdq.w4_linear(x, w)
    for i in range(3):
        x.copy_(make(x.shape, BF, 50 + i))
        want = hdq.w4_linear(x, w)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("T", [1, 5])
def test_serving_step(T):
    """A projection in 4 bits, its queries and keys normed and rotated, keys and
    values into the cache, the history read back: against the same chain in
    float64 from each stage's own output."""
    H, Hk, D, K, past = 6, 2, 64, 384, 20
    codes, scale, _ = R.w4_random((H + 2 * Hk) * D, K, 128, False, 13)
    w = hdq.w4_pack(codes.to(DEV), scale.to(DEV))
    x = make((T, K), BF, 14)
    qkv = hdq.w4_linear(x.to(DEV), w).view(1, T, H + 2 * Hk, D)
    check(qkv.view(T, -1), x, codes, scale, None, 128)
    c = hdq.KvCache(past + T, Hk, D, hdq.CACHE_INT8, 32, 64, device=DEV)
    pos = torch.arange(past, past + T, device=DEV)
    turns, r = plan((D,), True)
    q = hdq.qkv_to_cache(c, qkv[:, :, :H], qkv[:, :, H:H + Hk], qkv[:, :, H + Hk:], pos, hdq.HEAD_NORM_RMS, positions=pos, rope=r)
    host, p = qkv.cpu(), pos.cpu().view(1, 1, T)
    assert R.close(q, *reference(host[:, :, :H], "rms", None, None, 1e-6, (D,), True, turns, p, 1.0))
    kr, kt = reference(host[:, :, H:H + Hk], "rms", None, None, 1e-6, (D,), True, turns, p, 1.0)
    k, v = hdq.cache_read(c, torch.arange(past + T, device=DEV), y_dtype=hdq.DTYPE_F32)
    assert not bool(k[:past].any()) and not bool(v[:past].any())
    for y, ref, tol in ((k, kr, kt), (v, host[:, :, H + Hk:].double(), torch.zeros_like(kt))):
        # a code is off by half a step in the rotated domain: in the 2-norm of a head at most sqrt(D) / 2 steps of the
        # largest group's, a step at most the rotated maximum / 127, that at most the head's 2-norm
        err = (y[past:].cpu().double() - ref[0]).norm(dim=-1)
        assert bool((err <= ref[0].norm(dim=-1) * (math.sqrt(D) / 2 / 127 + 2.0 ** -18) + tol[0].norm(dim=-1)).all())


@pytest.mark.parametrize("M,N,K,group", [
    (1, 20, 32640, 128), (1, 20, 32672, 32),      # the last row of tokens that LDS takes, the first it does not
    (9, 33, 3584, 64), (9, 33, 3616, 32), (16, 40, 1920, 64), (16, 40, 2048, 128), (8, 17, 4064, 32), (8, 17, 4096, 64),
    (4, 70001, 128, 64), (13, 66000, 256, 32),    # several tiles of rows a wave
    (7, 13000, 1920, 64), (16, 12300, 1920, 128), (3, 12305, 2080, 32), (2, 12289, 96, 32), (5, 26000, 640, 128),  # waves that share K
    (17, 100, 96, 32), (32, 1000, 2080, 32), (33, 70, 1920, 64), (64, 257, 1120, 32), (47, 4100, 640, 128),
    (16, 12288, 1920, 64), (1, 12288, 2560, 128), (1, 4096, 8192, 64), (12, 256, 8192, 128), (13, 256, 8192, 128),
    (200, 12289, 160, 32), (70, 33000, 64, 64),   # more than a workgroup a CU
    (2, 500, 20480, 64), (33, 16, 8192, 128), (64, 2050, 1920, 32), (200, 129, 512, 64)])
@pytest.mark.parametrize("zero", [False, True])
def test_edges_of_the_forms(M, N, K, group, zero):
    codes, scale, z = R.w4_random(N, K, group, zero, 3 * M + N)
    x = make((M, K), BF, 21)
    w = hdq.w4_pack(codes.to(DEV), scale.to(DEV), z.to(DEV) if zero else None)
    check(hdq.w4_linear(x.to(DEV), w, y_dtype=hdq.DTYPE_F32), x, codes, scale, z, group)


def test_scratch_and_streams():
    """The caller's scratch, whatever it held; calls that overlap on two streams."""
    M, N, K = 40, 300, 8192                       # K split over workgroups
    codes, scale, _ = R.w4_random(N, K, 64, False, 31)
    w = hdq.w4_pack(codes.to(DEV), scale.to(DEV))
    xs = [make((M, K), BF, 32 + i).to(DEV) for i in range(2)]
    want = [hdq.w4_linear(x, w) for x in xs]
    need = hdq.w4_linear_workspace_bytes(M, N, K)
    assert need > 0
    for size in (need, need + 4096, 16):          # too small: one of its own
        ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
        assert all(torch.equal(hdq.w4_linear(x, w, ws=ws), y) for x, y in zip(xs, want))
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(8):
        for x, s, g in zip(xs, streams, got):
            g.append(hdq.w4_linear(x, w, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    # two graphs that share the caller's scratch, replayed one after the other
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    graphs = []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = hdq.w4_linear(x, w, ws=ws)
        graphs.append((g, y))
    for i in (0, 1, 1, 0):
        ws.fill_(77)
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[i][1], want[i])
