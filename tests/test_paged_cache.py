"""PagedCache without a GPU: what it refuses, with the engine's call replaced by one that records that it was made."""
import types

import pytest
import torch

VOCAB = 64


@pytest.fixture
def calls(monkeypatch):
    from autoregressive_decode_persistent_gb300 import adp
    got = []
    monkeypatch.setattr(adp, "adp_paged_forward", lambda *a: got.append(a))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(synchronize=lambda: None))
    return got


def _model(kv_dtype="f16"):
    return types.SimpleNamespace(device=torch.device("cpu"), handle=None,
                                 cfg=dict(n_layers=2, n_kv_heads=2, head_dim=64, vocab=VOCAB, kv_dtype=kv_dtype))


def _refused(cache, calls, logits):
    from autoregressive_decode_persistent_gb300 import adp
    with pytest.raises(adp.AdpError) as e:
        cache.forward([[0], [1]], [[1], [2, 3]], [1, 2], logits)
    assert e.value.code == adp.ADP_ERR_INVALID_ARG and not calls


def test_logits_that_the_engine_cannot_write_are_refused(calls):
    from autoregressive_decode_persistent_gb300.model import PagedCache
    cache = PagedCache(_model(), 2)
    room = torch.zeros(2 * VOCAB + 64)
    first = (-room.data_ptr() // 4) % 4  # the first element at a multiple of 16 bytes
    for i in range(5):
        logits = room[first + i:first + i + 2 * VOCAB].view(2, VOCAB)
        if i % 4:
            _refused(cache, calls, logits)
        else:
            assert cache.forward([[0], [1]], [[1], [2, 3]], [1, 2], logits) is logits and calls.pop()
    _refused(cache, calls, torch.empty((2, VOCAB), device="meta"))  # on another device
    _refused(cache, calls, torch.zeros((2, VOCAB), dtype=torch.float16))
    _refused(cache, calls, torch.zeros((2, VOCAB + 1))[:, :VOCAB])
    _refused(cache, calls, torch.zeros((3, VOCAB)))


@pytest.mark.parametrize("kv_dtype,own,other", [("f16", torch.float16, torch.bfloat16), ("bf16", torch.bfloat16, torch.float16)])
def test_pages_of_a_type_that_the_engine_would_misread_are_refused(kv_dtype, own, other):
    """The engine takes what is not e4m3 for the model's own 16-bit type: half a pool's bytes, or another type's bits."""
    from autoregressive_decode_persistent_gb300 import adp
    from autoregressive_decode_persistent_gb300.model import PagedCache
    for dtype in (other, torch.float8_e5m2, torch.uint8, torch.int16, torch.float32):
        with pytest.raises(adp.AdpError) as e:
            PagedCache(_model(kv_dtype), 2, 16, dtype)
        assert e.value.code == adp.ADP_ERR_UNSUPPORTED_CONFIG
    for dtype in (None, own, torch.float8_e4m3fn):
        cache = PagedCache(_model(kv_dtype), 2, 16, dtype)
        assert cache.k.dtype == cache.v.dtype == (dtype or own)
        assert (cache.k_scale is None) == (dtype != torch.float8_e4m3fn)
