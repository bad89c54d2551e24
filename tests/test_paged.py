"""The paged operators without a GPU: what they refuse, and their index arithmetic."""
import ctypes
import itertools
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # a 16-byte aligned address that no refused call reads


@pytest.fixture(scope="module")
def adp():
    from autoregressive_decode_persistent_gb300 import adp, build
    build.build()
    return adp


def _kv(adp, **kw):
    f = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, table=FAKE, lens=FAKE, page_stride=4 * 16 * 128,
             scale_stride=4 * 16, n_pages=10, page_size=16, n_kv_heads=4, head_dim=128, dtype=adp.ADP_F16, n_seqs=3,
             table_width=7)
    f.update(kw)
    return adp.PagedKV(*[f[n] for n, _ in adp.PagedKV._fields_])


BAD_KV = [(dict(k=None), -1), (dict(v=None), -1), (dict(table=None), -1), (dict(lens=None), -1), (dict(n_seqs=-1), -1),
          (dict(n_pages=0), -1), (dict(table_width=0), -1), (dict(n_kv_heads=0), -1), (dict(page_size=0), -1),
          (dict(k=FAKE + 8), -1), (dict(v=FAKE + 2), -1), (dict(table=FAKE + 2), -1), (dict(lens=FAKE + 1), -1),
          (dict(page_stride=4 * 16 * 128 - 8), -1), (dict(page_stride=4 * 16 * 128 + 4), -1),
          (dict(dtype=2, k_scale=None), -1), (dict(dtype=2, v_scale=None), -1), (dict(dtype=2, scale_stride=63), -1),
          (dict(dtype=2, k_scale=FAKE + 2), -1), (dict(dtype=3), -2), (dict(dtype=4), -2), (dict(head_dim=96), -2),
          (dict(head_dim=256, page_stride=1 << 20), -2), (dict(page_size=24, page_stride=1 << 20), -2),
          (dict(page_size=2048, page_stride=1 << 20), -2), (dict(n_kv_heads=1025, page_stride=1 << 30), -2),
          (dict(table_width=1 << 27), -2)]


@pytest.mark.parametrize("change,code", BAD_KV)
def test_a_wrong_cache_is_refused_by_every_operator(adp, change, code):
    kv = _kv(adp, **change)
    calls = [lambda: adp.adp_paged_kv_write(kv, FAKE, FAKE, adp.ADP_F16, 512, 512, FAKE, 5),
             lambda: adp.adp_paged_kv_read(kv, FAKE, FAKE, adp.ADP_F16, 512, 512, FAKE, 5),
             lambda: adp.adp_paged_attention(kv, FAKE, adp.ADP_F16, 20, 20 * 128, 0.1, FAKE, 20 * 128, FAKE, 1 << 40),
             lambda: adp.adp_paged_attention_workspace(kv, 20)]
    for call in calls:
        with pytest.raises(adp.AdpError) as e:
            call()
        assert e.value.code == code


@pytest.mark.parametrize("change,code", [
    (dict(rows_dtype=2), -2), (dict(rows_dtype=9), -2), (dict(n_rows=-1), -1), (dict(cu_rows=None), -1),
    (dict(cu_rows=FAKE + 2), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(k=FAKE + 4), -1), (dict(v=FAKE + 8), -1),
    (dict(k_stride=511), -1), (dict(v_stride=500), -1), (dict(k_stride=516), -1), (dict(v_stride=513), -1),
    (dict(dev_status=FAKE + 1), -1)])
def test_wrong_rows_are_refused(adp, change, code):
    a = dict(k=FAKE, v=FAKE, rows_dtype=adp.ADP_BF16, k_stride=512, v_stride=512, cu_rows=FAKE, n_rows=5, dev_status=None)
    a.update(change)
    for call in (adp.adp_paged_kv_write, adp.adp_paged_kv_read):
        with pytest.raises(adp.AdpError) as e:
            call(_kv(adp), **a)
        assert e.value.code == code


def test_no_rows_and_no_sequences_are_no_work(adp):
    for call in (adp.adp_paged_kv_write, adp.adp_paged_kv_read):
        call(_kv(adp), None, None, adp.ADP_F32, 0, 0, FAKE, 0)
        call(_kv(adp, n_seqs=0), None, None, adp.ADP_F32, 0, 0, FAKE, 0)
    adp.adp_paged_attention(_kv(adp, n_seqs=0), None, adp.ADP_F16, 20, 2560, 0.1, None, 2560, None, 0)


@pytest.mark.parametrize("change,code", [
    (dict(n_heads=0), -1), (dict(n_heads=18), -1), (dict(n_heads=4100), -2), (dict(q_dtype=3), -2), (dict(q_dtype=1), -2),
    (dict(q=None), -1), (dict(out=None), -1), (dict(q=FAKE + 8), -1), (dict(out=FAKE + 2), -1), (dict(q_stride=2552), -1),
    (dict(out_stride=2564), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(dev_status=FAKE + 3), -1)])
def test_wrong_attention_arguments_are_refused(adp, change, code):
    a = dict(q=FAKE, q_dtype=adp.ADP_F16, n_heads=20, q_stride=2560, scale=0.1, out=FAKE, out_stride=2560, workspace=FAKE,
             workspace_bytes=1 << 40, dev_status=None)
    a.update(change)
    with pytest.raises(adp.AdpError) as e:
        adp.adp_paged_attention(_kv(adp), **a)
    assert e.value.code == code


def test_too_many_sequences_for_one_attention_call_are_refused(adp):
    with pytest.raises(adp.AdpError) as e:
        adp.adp_paged_attention(_kv(adp, n_seqs=8193), FAKE, 0, 20, 2560, 0.1, FAKE, 2560, FAKE, 1 << 40)
    assert e.value.code == adp.ADP_ERR_UNSUPPORTED_CONFIG


def test_tensors_off_the_gpu_are_refused():
    import torch
    from autoregressive_decode_persistent_gb300 import adp, ops
    pages, table, lens = torch.zeros(2, 1, 16, 64, dtype=torch.float16), torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(adp.AdpError):
        ops.paged_attention(torch.zeros(1, 1, 64, dtype=torch.float16), pages, pages, table, lens)


# ---------------------------------------------------------------- index arithmetic (csrc/paged.h) on the host

@pytest.fixture(scope="module")
def index(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged_index")
    src = d / "index.cpp"
    src.write_text('#include "%s"\nusing namespace adp;\nextern "C" {\n'
                   "int32_t t_length(int32_t l, int32_t w, int lg) { return paged_length(l, w, lg); }\n"
                   "int64_t t_position(int32_t l, int32_t n, int32_t i) { return paged_position(l, n, i); }\n"
                   "int32_t t_page(const int32_t* t, int32_t w, int32_t n, int lg, int64_t p) { return paged_page(t, w, n, lg, p); }\n"
                   "int64_t t_begin(int64_t t, int32_t n, int32_t i) { return split_begin(t, n, i); }\n"
                   "int32_t t_owner(int64_t t, int32_t n, int64_t u) { return split_owner(t, n, u); }\n"
                   "int32_t t_parts(int64_t t, int32_t n) { return split_parts(t, n); }\n}\n"
                   % os.path.join(ROOT, "autoregressive_decode_persistent_gb300", "csrc", "paged.h"))
    lib = d / "index.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    i32, i64, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    for name, res, args in [("t_length", i32, [i32, i32, i32]), ("t_position", i64, [i32, i32, i32]),
                            ("t_page", i32, [p, i32, i32, i32, i64]), ("t_begin", i64, [i64, i32, i32]),
                            ("t_owner", i32, [i64, i32, i64]), ("t_parts", i32, [i64, i32])]:
        getattr(L, name).restype, getattr(L, name).argtypes = res, args
    return L


def test_no_page_number_or_length_leads_outside_the_pool(index):
    rng = random.Random(1)
    for lg, width, n_pages in itertools.product((0, 3, 4, 10), (1, 5), (1, 9)):
        entries = [rng.choice([-1, -2 ** 31, 2 ** 31 - 1, n_pages, 0, n_pages - 1]) for _ in range(width)]
        row = np.array(entries, dtype=np.int32)
        cap = width << lg
        for pos in [-2 ** 33, -1, 0, 1, cap - 1, cap, cap + 1, 2 ** 31, 2 ** 40] + [rng.randrange(cap) for _ in range(20)]:
            got = index.t_page(row.ctypes.data, width, n_pages, lg, pos)
            want = entries[pos >> lg] if 0 <= pos < cap else -1
            assert got == (want if 0 <= want < n_pages else -1)
        for n in (-2 ** 31, -1, 0, 1, cap, cap + 1, 2 ** 31 - 1):
            assert index.t_length(n, width, lg) == min(max(n, 0), cap)


def test_positions_of_packed_rows(index):
    assert [index.t_position(10, 7, i) for i in (4, 5, 6)] == [7, 8, 9]
    assert index.t_position(2, 7, 3) == -2                              # fewer positions than rows
    assert index.t_position(-2 ** 31, 2 ** 31 - 1, 0) == -2 ** 32 + 1  # no 32-bit overflow


def test_the_split_covers_every_unit_once_and_owners_agree(index):
    rng = random.Random(2)
    for _ in range(300):
        total = rng.choice([1, 2, 7, 8, 9, 151, 1217, rng.randrange(1, 10 ** 6), rng.randrange(1, 2 ** 40)])
        parts = index.t_parts(total, rng.choice([1, 2, 152, 304]))
        edges = [index.t_begin(total, parts, i) for i in range(parts + 1)]
        assert edges[0] == 0 and edges[-1] == total
        assert all(b > a for a, b in zip(edges, edges[1:]))  # no part is empty
        for i in range(parts):
            for u in {edges[i], edges[i + 1] - 1, rng.randrange(edges[i], edges[i + 1])}:
                assert index.t_owner(total, parts, u) == i


def test_rows_that_no_offsets_hold(tmp_path):
    """paged_holds (csrc/paged.h) against the sets of rows that the offsets name."""
    src, lib = tmp_path / "holds.cpp", tmp_path / "holds.so"
    src.write_text('#include "%s"\nextern "C" int t_holds(int32_t b, int32_t f, int32_t n, int32_t i) '
                   "{ return adp::paged_holds(b, f, n, i); }\n"
                   % os.path.join(ROOT, "autoregressive_decode_persistent_gb300", "csrc", "paged.h"))
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    for cu in ([0, 3, 3, 7], [0, 50, 20, 60], [5, 10, 20, 20], [-5, 10, 12, 14], [0, -5, 4, 9], [0, 2 ** 31 - 1, -2 ** 31, 3]):
        for b in range(3):
            rows = range(cu[b], cu[b + 1]) if cu[b] >= 0 and (b > 0 or cu[0] == 0) else ()
            for i in list(range(70)) + [2 ** 31 - 2, 2 ** 31 - 1]:
                assert bool(L.t_holds(b, cu[b], cu[b + 1], i)) == (i in rows)


def test_shapes_that_name_no_rows_are_refused():
    import torch
    from autoregressive_decode_persistent_gb300 import adp, ops
    pages, table, lens = torch.zeros(2, 1, 16, 64, dtype=torch.float16), torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    cu, rows = torch.tensor([0, 1], dtype=torch.int32), torch.zeros(1, 1, 64, dtype=torch.float16)
    for bad, n, more in ((pages[0], 1, {}), (pages[0, 0, 0, 0], 1, {}), (pages, -1, {}), (pages, 1, dict(dtype=torch.int32)),
                         (pages, 1, dict(out=(rows,))), (pages, 1, dict(out=(rows, rows, rows))), (pages, 2, dict(out=(rows, rows))),
                         (pages, 1, dict(out=(rows[0, 0, 0], rows))), (pages, 1, dict(out=(rows, rows), dtype=torch.float32))):
        with pytest.raises(adp.AdpError) as e:
            ops.paged_kv_read(bad, bad, table, lens, cu, n, **more)
        assert e.value.code == adp.ADP_ERR_INVALID_ARG


@pytest.mark.parametrize("head_dim,dtype,unit", [(128, 0, 16), (64, 0, 32), (128, 2, 32), (64, 2, 64)])
def test_tables_whose_units_do_not_fit_32_bits_are_refused(adp, head_dim, dtype, unit):
    """32 sequences' units (`unit` positions each) are added in 32 bits."""
    most = 2 ** 31 - 1024 - 1  # positions that a table may name at all
    for n_seqs, width in ((1, 2 ** 21 - 2), (31, 2 ** 20), (32, 2 ** 20 - 1), (32, 2 ** 20), (32, 2 ** 20 + 1), (8192, 2 ** 21 - 2)):
        assert width * 1024 <= most
        kv = _kv(adp, n_seqs=n_seqs, table_width=width, page_size=1024, head_dim=head_dim, dtype=dtype,
                 page_stride=4 * 1024 * head_dim, scale_stride=4 * 1024)
        code = 0
        try:
            adp.adp_paged_attention_workspace(kv, 20)
        except adp.AdpError as e:
            code = e.code
        fits = min(n_seqs, 32) * -(-width * 1024 // unit) < 2 ** 31
        assert code in ((0, adp.ADP_ERR_CUDA) if fits else (adp.ADP_ERR_UNSUPPORTED_CONFIG,))  # (CUDA: no GPU here)
