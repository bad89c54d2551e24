"""Appending to a paged cache and attention with a window, without a GPU: what they refuse."""
import pytest

from test_paged import BAD_KV, FAKE, _kv, adp  # noqa: F401


def _rope(adp, **kw):
    f = dict(cos=FAKE, sin=FAKE, n_positions=100, rotated=128, q_gain=FAKE, k_gain=FAKE, gain_dtype=0, eps=1e-5)
    f.update(kw)
    return adp.Rope(*[f[n] for n, _ in adp.Rope._fields_])


APPEND = dict(q=FAKE, k=FAKE, v=FAKE, rows_dtype=1, n_heads=20, q_stride=2560, k_stride=512, v_stride=512, cu_rows=FAKE, n_rows=5,
              out=FAKE, out_dtype=1, out_stride=2560, dev_status=None)
WINDOW = dict(q=FAKE, q_dtype=0, n_heads=20, q_stride=2560, scale=0.1, window=64, sinks=4, out=FAKE, out_stride=2560, workspace=FAKE,
              workspace_bytes=1 << 40, dev_status=None)


@pytest.mark.parametrize("change,code", BAD_KV)
def test_a_wrong_cache_is_refused(adp, change, code):
    kv = _kv(adp, **change)
    for call in (lambda: adp.adp_paged_kv_append(kv, _rope(adp), **APPEND), lambda: adp.adp_paged_window_attention(kv, **WINDOW),
                 lambda: adp.adp_paged_window_attention_workspace(kv, 20, 64, 4)):
        with pytest.raises(adp.AdpError) as e:
            call()
        assert e.value.code == code


@pytest.mark.parametrize("change,code", [
    (dict(rows_dtype=2), -2), (dict(out_dtype=2), -2), (dict(n_heads=4097), -2), (dict(n_heads=-1), -1), (dict(n_rows=-1), -1),
    (dict(cu_rows=None), -1), (dict(cu_rows=FAKE + 2), -1), (dict(dev_status=FAKE + 1), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(q=None), -1), (dict(out=None), -1), (dict(q=FAKE + 8), -1), (dict(k=FAKE + 4), -1), (dict(v=FAKE + 8), -1), (dict(out=FAKE + 2), -1),
    (dict(q_stride=2552), -1), (dict(q_stride=2564), -1), (dict(k_stride=511), -1), (dict(v_stride=516), -1), (dict(out_stride=2559), -1),
    (dict(out_stride=2562, out_dtype=3), -1)])
def test_wrong_rows_to_append_are_refused(adp, change, code):
    with pytest.raises(adp.AdpError) as e:
        adp.adp_paged_kv_append(_kv(adp), _rope(adp), **dict(APPEND, **change))
    assert e.value.code == code


@pytest.mark.parametrize("change,code", [
    (dict(cos=None), -1), (dict(sin=None), -1), (dict(cos=FAKE + 8), -1), (dict(sin=FAKE + 4), -1), (dict(n_positions=-1), -1),
    (dict(rotated=0), -2), (dict(rotated=24), -2), (dict(rotated=144), -2), (dict(rotated=-16), -1), (dict(q_gain=FAKE + 8), -1),
    (dict(k_gain=FAKE + 2), -1), (dict(gain_dtype=2), -2), (dict(eps=-1e-5), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1)])
def test_a_wrong_rotation_is_refused(adp, change, code):
    with pytest.raises(adp.AdpError) as e:
        adp.adp_paged_kv_append(_kv(adp), _rope(adp, **change), **APPEND)
    assert e.value.code == code


def test_no_rows_and_no_sequences_are_no_work(adp):
    adp.adp_paged_kv_append(_kv(adp), _rope(adp), **dict(APPEND, n_rows=0, q=None, k=None, v=None, out=None))
    adp.adp_paged_kv_append(_kv(adp, n_seqs=0), _rope(adp, q_gain=None, k_gain=None, gain_dtype=9), **dict(APPEND, k=None))
    adp.adp_paged_window_attention(_kv(adp, n_seqs=0), **dict(WINDOW, q=None, out=None, workspace=None, workspace_bytes=0))


@pytest.mark.parametrize("change,code", [
    (dict(window=0), -1), (dict(window=-3), -1), (dict(sinks=-1), -1), (dict(n_heads=18), -1), (dict(n_heads=4100), -2), (dict(q_dtype=3), -2),
    (dict(q_dtype=1), -2), (dict(q=None), -1), (dict(out=FAKE + 2), -1), (dict(q_stride=2552), -1), (dict(scale=float("inf")), -1),
    (dict(dev_status=FAKE + 3), -1)])
def test_wrong_window_arguments_are_refused(adp, change, code):
    with pytest.raises(adp.AdpError) as e:
        adp.adp_paged_window_attention(_kv(adp), **dict(WINDOW, **change))
    assert e.value.code == code


def test_tensors_off_the_gpu_are_refused():
    import torch
    from autoregressive_decode_persistent_gb300 import adp, ops
    pages, table, lens = torch.zeros(2, 1, 16, 64, dtype=torch.float16), torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    rows, cu, angles = torch.zeros(1, 1, 64, dtype=torch.float16), torch.tensor([0, 1], dtype=torch.int32), torch.zeros(5, 32)
    with pytest.raises(adp.AdpError):
        ops.paged_attention(rows, pages, pages, table, lens, window=3)
    with pytest.raises(adp.AdpError):
        ops.paged_kv_append(pages, pages, table, lens, cu, rows, rows, rows, angles, angles)


@pytest.mark.parametrize("which", range(6))
def test_what_is_no_tensor_is_refused(which):
    import torch
    from autoregressive_decode_persistent_gb300 import adp, ops
    for bad in (None, 3, [1.0]):
        args = [torch.zeros(1)] * 6
        args[which] = bad
        with pytest.raises((adp.AdpError, TypeError, AttributeError)):
            ops.paged_chunk_attention(*args)


# ---------------------------------------------------------------- chunks of rows over the pages

CHUNK = dict(q=FAKE, q_dtype=0, n_heads=20, q_stride=2560, cu_rows=FAKE, n_rows=50, scale=0.1, window=0, sinks=0, out=FAKE, out_stride=2560,
             workspace=FAKE, workspace_bytes=1 << 40, dev_status=None)


@pytest.mark.parametrize("change,code", BAD_KV)
def test_a_wrong_cache_is_refused_by_chunk_attention(adp, change, code):
    kv = _kv(adp, **change)
    for call in (lambda: adp.adp_paged_chunk_attention(kv, **CHUNK), lambda: adp.adp_paged_chunk_attention_workspace(kv, 20, 50, 0, 0)):
        with pytest.raises(adp.AdpError) as e:
            call()
        assert e.value.code == code


@pytest.mark.parametrize("change,code", [
    (dict(n_heads=0), -1), (dict(n_heads=18), -1), (dict(n_heads=516), -2), (dict(q_dtype=3), -2), (dict(q_dtype=1), -2), (dict(q=None), -1),
    (dict(out=None), -1), (dict(q=FAKE + 8), -1), (dict(out=FAKE + 2), -1), (dict(q_stride=2552), -1), (dict(out_stride=2564), -1),
    (dict(cu_rows=None), -1), (dict(cu_rows=FAKE + 2), -1), (dict(n_rows=-1), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(dev_status=FAKE + 3), -1)])
def test_wrong_chunk_arguments_are_refused(adp, change, code):
    with pytest.raises(adp.AdpError) as e:
        adp.adp_paged_chunk_attention(_kv(adp), **dict(CHUNK, **change))
    assert e.value.code == code


def test_no_rows_of_chunks_are_no_work(adp):
    adp.adp_paged_chunk_attention(_kv(adp), **dict(CHUNK, n_rows=0, q=None, out=None, workspace=None, workspace_bytes=0))
    adp.adp_paged_chunk_attention(_kv(adp, n_seqs=0), **dict(CHUNK, q=None, out=None, workspace=None, workspace_bytes=0))
    with pytest.raises(adp.AdpError) as e:
        adp.adp_paged_chunk_attention(_kv(adp, n_seqs=8193), **CHUNK)
    assert e.value.code == adp.ADP_ERR_UNSUPPORTED_CONFIG


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    import ctypes
    import os
    import subprocess
    from test_paged import ROOT
    d = tmp_path_factory.mktemp("chunk_lines")
    src, lib = d / "lines.cpp", d / "lines.so"
    src.write_text('#include "%s"\nusing namespace adp;\nextern "C" {\n'
                   "void t_span(int32_t f, int32_t l, int32_t w, int32_t s, int32_t* o) { ChunkSpan c = chunk_span(f, l, w, s);\n"
                   " o[0] = c.head; o[1] = c.gap; o[2] = c.n; o[3] = c.low; }\n"
                   "int32_t t_block(int32_t f, int32_t l, int32_t w, int32_t s, int32_t i) { return chunk_block(chunk_span(f, l, w, s), i); }\n"
                   "int32_t t_cut(int32_t n, int64_t d) { return chunk_cut(n, d); }\n"
                   "int32_t t_parts(int64_t t, int64_t n, int32_t c) { return chunk_parts(t, n, c); }\n}\n"
                   % os.path.join(ROOT, "autoregressive_decode_persistent_gb300", "csrc", "paged_chunk.h"))
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    L.t_cut.argtypes = [ctypes.c_int32, ctypes.c_int64]
    L.t_parts.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32]
    return L


def test_the_line_holds_every_block_that_a_row_sees_once(lines):
    import ctypes
    import random
    rng = random.Random(1)
    for _ in range(4000):
        first = rng.choice([rng.randint(-200, 0), rng.randint(0, 3000)])
        last = first + rng.randint(0, 300)
        window = rng.choice([2 ** 31 - 1, 1, rng.randint(1, 3000)])
        sinks = rng.choice([0, 1, rng.randint(0, 400), 2 ** 31 - 1])
        o = (ctypes.c_int32 * 4)()
        lines.t_span(first, last, window, sinks, o)
        blocks = [lines.t_block(first, last, window, sinks, i) for i in range(o[2])]
        assert blocks == sorted(set(blocks))
        seen = set()
        for p in range(max(first, 0), last + 1):
            low = max(0, p - window + 1)
            seen |= set(range(low // 64, p // 64 + 1)) | set(range(0, -(-min(sinks, low) // 64)))
        assert seen <= set(blocks)
        assert len(blocks) <= len(seen) + 1 or window < 64  # (a block more at most)
        assert (o[2] == 0) == (last < 0)


def test_cuts_leave_whole_pieces_or_parts_of_some_blocks(lines):
    for n in (0, 1, 3, 7, 8, 9, 20, 1000):
        at = [lines.t_cut(n, d) for d in range(n + 5)]
        assert at == sorted(at) and at[0] == 0 and all(j in (0, n) or 4 <= j <= n - 4 for j in at)
    for total, items, ctas in ((0, 0, 152), (5, 1, 152), (100, 2, 152), (10 ** 12, 10, 152), (500, 400, 152), (40, 1, 1)):
        p = lines.t_parts(total, items, ctas)
        assert 1 <= p <= ctas and p >= min(items, ctas)
