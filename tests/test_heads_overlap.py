"""CPU checks: outputs of the head entry points whose elements would be one, or
that lie on another operand, are refused before any launch."""
import pytest

FAKE = 0x100000   # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def hdq():
    from bit_quantized_video_amd import hdq as H
    return H


def view(hdq, at=0, dtype=1, n=6, b=0, t=384, h=64):
    return hdq.HeadsDesc(FAKE + at * (1 << 24), dtype, n, b, t, h)


# (batch, length, heads, batch stride, token stride, head stride) with heads of 64
COINCIDE = [(1, 2, 6, 0, 64, 64), (1, 5, 6, 0, 128, 64), (1, 16, 6, 0, 383, 64), (2, 16, 6, 64, 384, 64), (2, 16, 6, 16 * 384 - 1, 384, 64),
            (2, 16, 6, 384, 768, 64 * 3), (4, 1, 6, 320, 0, 64), (3, 16, 1, 64 * 8, 64, 0), (1, 16, 6, 0, 64, 64 * 15), (1, 2, 1, 0, 63, 0),
            (1, 2, 6, 0, 384, 63), (2, 1, 1, 0, 0, 0), (3, 1 << 28, 2, 1 << 40, 1 << 20, 64)]
APART = [(1, 2, 6, 0, 384, 64), (1, 1, 6, 0, 0, 64), (1, 16, 1, 0, 64, 0), (2, 16, 6, 16 * 384, 384, 64), (2, 16, 6, 384, 768, 64),
         (2, 16, 6, 16 * 64, 64, 2 * 16 * 64), (2, 16, 6, 64, 128, 16 * 128), (1, 1, 1, 0, 0, 0), (1, 16, 6, 7, 400, 66),
         (2, 2, 2, 1 << 40, 1 << 39, 1 << 38), (1 << 20, 1 << 10, 6, 1 << 39, 384, 64)]


def status(hdq, shape, cached):
    """The refusal of an output of this shape, or that of the argument checked after it (a dtype of its own)."""
    B, T, H, b, t, h = shape
    q, out = view(hdq, 0, n=H, b=1 << 20, t=1 << 10, h=64), view(hdq, 1, n=H, b=b, t=t, h=h)
    if cached:
        c = hdq.KvCacheDesc(1, 64, 1, 2, 64, 100, FAKE, FAKE, FAKE, FAKE)
        k, v = view(hdq, 2, n=2), view(hdq, 3, n=2, dtype=0)
        return hdq.lib.hdq_qkv_to_cache(q, k, v, B, T, None, None, out, FAKE, c, None)
    k, ko = view(hdq, 2, n=2, dtype=0), view(hdq, 3, n=2, b=1 << 40, t=1 << 10, h=64)
    return hdq.lib.hdq_qk_norm_rope(q, k, B, T, 64, None, None, out, ko, None)


@pytest.mark.parametrize("cached", [False, True])
def test_elements_that_coincide(hdq, cached):
    for shape in COINCIDE:
        assert status(hdq, shape, cached) == hdq.ERR_SHAPE, shape


@pytest.mark.parametrize("cached", [False, True])
def test_views_that_lie_apart(hdq, cached):
    """They pass this check and meet the next one, of the types."""
    for shape in APART:
        if cached or shape[0] * shape[1] < 1 << 10:
            assert status(hdq, shape, cached) == hdq.ERR_UNSUPPORTED, shape


def test_inputs_may_coincide(hdq):
    """An expanded input is refused for nothing."""
    q, out = view(hdq, 0, n=6, b=0, t=0, h=0), view(hdq, 1, dtype=7)
    assert hdq.lib.hdq_qk_norm_rope(q, None, 2, 16, 64, None, None, out, None, None) == hdq.ERR_UNSUPPORTED


def test_outputs_on_other_operands(hdq):
    V = lambda *a, **kw: view(hdq, *a, **kw)

    def f(q, qo, k=None, ko=None, T=16):
        return hdq.lib.hdq_qk_norm_rope(q, k, 1, T, 64, None, None, qo, ko, None)
    # at its own input with other strides or another type
    assert f(V(0), V(0, t=448)) == hdq.ERR_SHAPE and f(V(0), V(0, t=64, h=64 * 16)) == hdq.ERR_SHAPE
    assert f(V(0), V(0, dtype=0)) == hdq.ERR_SHAPE
    assert f(V(0), V(1), V(2), V(2, t=448)) == hdq.ERR_SHAPE and f(V(0), V(1, dtype=0), V(2), V(2, dtype=0)) == hdq.ERR_SHAPE
    # at the other input, or the other output
    for qo, ko in ((2, 3), (1, 0), (1, 1), (2, 0)):
        assert f(V(0), V(qo), V(2), V(ko)) == hdq.ERR_INVALID, (qo, ko)
    c = hdq.KvCacheDesc(1, 64, 1, 2, 64, 100, FAKE, FAKE, FAKE, FAKE)
    for at, st in ((1, hdq.ERR_INVALID), (2, hdq.ERR_INVALID)):
        got = hdq.lib.hdq_qkv_to_cache(V(0), V(1, n=2), V(2, n=2), 1, 16, None, None, V(at), FAKE, c, None)
        assert got == st, at
    got = hdq.lib.hdq_qkv_to_cache(V(0), V(1, n=2), V(2, n=2), 1, 16, None, None, V(0, t=448), FAKE, c, None)
    assert got == hdq.ERR_SHAPE
