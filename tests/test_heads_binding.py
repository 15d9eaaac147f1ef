"""CPU checks of the head bindings' own refusals: types of outputs."""
import pytest
import torch


@pytest.fixture(scope="module")
def hdq():
    from bit_quantized_video_amd import hdq as H
    return H


def test_output_types(hdq, monkeypatch):
    """A y_dtype that heads cannot have, or that is not the given output's, is
    refused; the call itself is left out."""
    calls = []
    ok = lambda *a: calls.append(a) or hdq.OK
    monkeypatch.setattr(hdq, "_launch", lambda dev, stream, call: call(None))
    monkeypatch.setattr(hdq, "_qk_norm_rope", ok)
    monkeypatch.setattr(hdq, "_qkv_to_cache", ok)
    x = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    f32 = torch.zeros(5, 4, 64)
    c, slots = hdq.KvCache(10, 4, 64, device="cpu"), torch.arange(5)
    for kw in (dict(y_dtype=hdq.DTYPE_I32), dict(y_dtype=7), dict(y_dtype=hdq.DTYPE_F32, q_out=x), dict(y_dtype=hdq.DTYPE_BF16, q_out=f32)):
        with pytest.raises(ValueError):
            hdq.qk_norm_rope(x, **kw)
        with pytest.raises(ValueError):
            hdq.qkv_to_cache(c, x, x, x, slots, **kw)
    with pytest.raises(ValueError):
        hdq.qk_norm_rope(x, x, q_out=f32, k_out=torch.zeros_like(x), y_dtype=hdq.DTYPE_F32)
    assert not calls
    for kw, dt in ((dict(), torch.bfloat16), (dict(y_dtype=hdq.DTYPE_BF16), torch.bfloat16), (dict(y_dtype=hdq.DTYPE_F32), torch.float32),
                   (dict(y_dtype=hdq.DTYPE_F32, q_out=f32), torch.float32), (dict(q_out=f32), torch.float32)):
        assert hdq.qk_norm_rope(x, **kw).dtype is dt and hdq.qkv_to_cache(c, x, x, x, slots, **kw).dtype is dt
    assert len(calls) == 10
