"""The tensor calls where the extension module of their checks could not be built: attention of single tokens runs all the same, the
calls that need the module say so."""
import random
import sys

import pytest
import torch

from test_gpu_paged import BF16, E4M3, F16, check_attention, paged, run


@pytest.fixture
def alone(monkeypatch):
    """ops.py on a machine that has libadp.so alone."""
    import autoregressive_decode_persistent_gb300 as package
    from autoregressive_decode_persistent_gb300 import build, ops
    build.build()
    monkeypatch.delattr(package, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, package.__name__ + "._binding", None)
    monkeypatch.setattr(ops, "_binding", None)
    monkeypatch.setattr(ops, "_missing", None, raising=False)
    return ops


def test_calls_that_need_the_module_say_so(alone):
    x = torch.zeros(1)
    for call in (lambda: alone.paged_kv_append(*[x] * 10), lambda: alone.paged_chunk_attention(*[x] * 6)):
        with pytest.raises(RuntimeError, match=r"build\.build\(\)"):
            call()


def test_tensors_off_the_gpu_are_refused(alone):
    from autoregressive_decode_persistent_gb300 import adp
    pages, table, lens = torch.zeros(2, 1, 16, 64, dtype=F16), torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for kw in ({}, dict(window=3), dict(window=0), dict(sinks=1), dict(window=3, sinks=-1)):
        with pytest.raises(adp.AdpError):
            alone.paged_attention(torch.zeros(1, 1, 64, dtype=F16), pages, pages, table, lens, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,q_dtype", [(F16, F16), (BF16, BF16), (E4M3, BF16)])
def test_attention_of_single_tokens_runs_alike(alone, monkeypatch, dtype, q_dtype):
    from autoregressive_decode_persistent_gb300 import adp
    rng = random.Random(3)
    c, q = run([6000, 0] + [rng.randint(0, 300) for _ in range(20)], (8, 2), 64, 16, dtype, q_dtype, seed=2)
    calls = [dict(), dict(scale=0.3), dict(window=50, sinks=4), dict(window=10 ** 12, sinks=3), dict(window=5000)]
    got = [paged(alone, q, c, **kw) for kw in calls]
    out, status = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = alone._paged("test", c.k, c.v, c.table, c.len_t, *(c.scales.get(n) for n in ("k_scale", "v_scale")), 0)
    ws = torch.empty(adp.adp_paged_attention_workspace(kv, 8), dtype=torch.uint8, device="cuda")
    assert paged(alone, q, c, out=out, workspace=ws, status=status) is out
    for kw in (dict(window=0), dict(sinks=2), dict(out=out[1:]), dict(scale=float("nan")), dict(workspace=out)):
        with pytest.raises(adp.AdpError):
            paged(alone, q, c, **kw)
    check_attention(got[0], q, c)
    check_attention(got[2], q, c, skip={(b, p) for b, n in enumerate(c.lens) for p in range(4, n - 50)})
    monkeypatch.undo()
    assert int(status) == 0 and torch.equal(out, got[0])
    for kw, o in zip(calls, got):  # with the module
        assert torch.equal(paged(alone, q, c, **kw), o)


@pytest.mark.gpu
def test_a_workspace_that_is_too_small_is_refused(alone):
    from autoregressive_decode_persistent_gb300 import adp
    c, q = run([6000, 10], (8, 2), 128, 16, F16, seed=22)
    kv = alone._paged("test", c.k, c.v, c.table, c.len_t, None, None, 0)
    need = adp.adp_paged_window_attention_workspace(kv, 8, 5000, 4)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    check_attention(paged(alone, q, c, workspace=ws, window=5000, sinks=4), q, c, skip={(0, p) for p in range(4, 1000)})
    with pytest.raises(adp.AdpError):
        paged(alone, q, c, workspace=ws[:need - 1], window=5000, sinks=4)
