"""Attention of one new token per sequence with a sliding window and first positions that stay visible, against plain 64-bit
computations, through ops.paged_attention."""
import random

import pytest
import torch

from test_gpu_paged import BF16, E4M3, F16, NAN, TYPES, check_attention, ops, paged, run  # noqa: F401

pytestmark = pytest.mark.gpu


def unseen(lens, window, sinks):
    return {(b, p) for b, n in enumerate(lens) for p in range(sinks, n - window)}


def wide_table(c, width=20000):
    t = torch.full((len(c.lens), width), -1, dtype=torch.int32, device="cuda")
    t[:, :c.table.shape[1]] = c.table
    return t


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("heads,page,lens,window,sinks", [
    ((4, 2), 16, [77], 20, 0), ((20, 4), 16, [513, 0, 1, 15, 16, 17, 33, 200], 16, 4), ((8, 8), 32, [1, 2, 31, 32, 65, 300], 1, 0),
    ((8, 1), 64, [0, 0, 700, 0], 64, 64), ((14, 2), 8, [9, 100, 3, 64], 33, 17), ((24, 2), 128, [129, 40, 900], 100, 130),
    ((16, 1), 1, [5, 20, 90], 7, 2), ((34, 2), 4, [30, 31, 200], 65, 1), ((4, 2), 16, [400, 90], 2 ** 31 - 1, 2 ** 31 - 1),
    ((4, 1), 16, [1500, 64, 65], 500, 1000)])
def test_matches_64_bits(ops, hd, dtype, q_dtype, heads, page, lens, window, sinks):
    c, q = run(lens, heads, hd, page, dtype, q_dtype, seed=hd + page)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for table in (c.table, wide_table(c, 3000)):
        out = ops.paged_attention(q, c.k, c.v, table, c.len_t, window=window, sinks=sinks, status=status, **c.scales)
        check_attention(out, q, c, skip=unseen(lens, window, sinks))
        assert torch.equal(out, ops.paged_attention(q, c.k, c.v, table, c.len_t, window=window, sinks=sinks, **c.scales))
    assert int(status) == 0


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
def test_windows_that_are_split_and_joined(ops, dtype, q_dtype):
    rng = random.Random(5)
    for lens, window, sinks in (([9000], 5000, 0), ([9000, 7, 0, 5500], 3000, 100), ([rng.randint(0, 300) for _ in range(200)], 70, 9)):
        c, q = run(lens, (8, 2), 64, 16, dtype, q_dtype, seed=len(lens))
        out = paged(ops, q, c, window=window, sinks=sinks)
        check_attention(out, q, c, skip=unseen(lens, window, sinks))
        assert torch.equal(out, paged(ops, q, c, window=window, sinks=sinks))


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("page", [4, 16, 64])
def test_what_is_not_seen_is_neither_read_nor_looked_up(ops, dtype, q_dtype, page):
    """Pages of which nothing is seen have no number any more, and the other cells that are not seen hold NaN."""
    lens, window, sinks = [300, 1000, 129], 40, 6
    c, q = run(lens, (8, 2), 128, page, dtype, q_dtype, seed=3)
    gone = unseen(lens, window, sinks)
    for b, n in enumerate(lens):
        for at in range(-(-n // page)):
            cells = [p for p in range(at * page, (at + 1) * page) if p < n]
            if all((b, p) in gone for p in cells):
                c.table[b, at] = -7
            else:
                for p in cells:
                    if (b, p) in gone:
                        i = int(c.table[b, at]), slice(None), p % page
                        if dtype == E4M3:
                            c.scales["k_scale"][i] = c.scales["v_scale"][i] = NAN
                        else:
                            c.k[i] = c.v[i] = NAN
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for table in (c.table, wide_table(c)):
        out = ops.paged_attention(q, c.k, c.v, table, c.len_t, window=window, sinks=sinks, status=status, **c.scales)
        check_attention(out, q, c, skip=gone)
    assert int(status) == 0
    c.table[1, 999 // page] = -7  # a page that is seen
    ops.paged_attention(q, c.k, c.v, c.table, c.len_t, window=window, sinks=sinks, status=status, **c.scales)
    assert int(status) == -1


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
def test_a_window_as_long_as_the_context_is_none(ops, dtype, q_dtype):
    c, q = run([500, 31, 0, 64], (8, 2), 128, 16, dtype, q_dtype, seed=4)
    want = paged(ops, q, c)
    for window, sinks in ((500, 0), (10 ** 12, 3), (500, 10 ** 12)):
        assert torch.equal(paged(ops, q, c, window=window, sinks=sinks), want)


def test_captured_graphs_with_changing_lengths(ops):
    lens, window, sinks = [300, 10], 50, 5
    c, q = run(lens, (8, 2), 64, 16, BF16, seed=11)
    graphs, outs = [], []
    for table in (c.table, wide_table(c)):
        for w in (window, 5000):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append((ops.paged_attention(q, c.k, c.v, table, c.len_t, window=w, sinks=sinks), w))
            graphs.append((g, table))
    for lens in ([300, 10], [51, 0], [299, 5]):
        c.len_t.copy_(torch.tensor(lens, dtype=torch.int32))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out, w in outs:
            check_attention(out, q, c, lens=lens, skip=unseen(lens, w, sinks))


def test_workspace_and_refusals(ops):
    from autoregressive_decode_persistent_gb300 import adp
    c, q = run([6000, 10], (8, 2), 128, 16, F16, seed=22)
    kv = ops._paged("test", c.k, c.v, c.table, c.len_t, None, None, 0)
    assert adp.adp_paged_window_attention_workspace(kv, 8, 64, 4) == 0  # short windows: a cluster each
    need = adp.adp_paged_window_attention_workspace(kv, 8, 5000, 4)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    check_attention(paged(ops, q, c, workspace=ws, window=5000, sinks=4), q, c, skip=unseen(c.lens, 5000, 4))
    for kw in (dict(workspace=ws[:need - 1], window=5000, sinks=4), dict(window=0), dict(window=-1), dict(window=5, sinks=-1), dict(sinks=3)):
        with pytest.raises(adp.AdpError):
            paged(ops, q, c, **kw)
