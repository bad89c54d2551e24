"""Chunk attention of more sequences than a warp has lanes, some of them cut over several CTAs, and lengths beyond the table."""
import random

import pytest
import torch

from test_gpu_paged import E4M3, F16, TYPES, ops  # noqa: F401
from test_gpu_paged_chunk import Chunk, wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("n,heads,hd,page", [(33, (8, 2), 64, 16), (65, (4, 1), 128, 64), (100, (16, 4), 64, 8), (40, (2, 2), 64, 16)])
def test_long_sequences_among_more_than_32_are_cut_and_joined(ops, dtype, q_dtype, n, heads, hd, page):  # noqa: F811
    from autoregressive_decode_persistent_gb300 import adp
    rng = random.Random(n)
    new = [rng.choice([0, 0, 1, 2, 5, 8]) for _ in range(n)]
    old = [rng.choice([0, rng.randint(0, 90)]) for _ in range(n)]
    for b, m, o in ((31, 8, 3000), (32, 1, 4500), (33, 3, 2100), (n - 1, 7, 3600)):
        if b < n:
            new[b], old[b] = m, o
    x = Chunk(new, old, heads, hd, page, dtype, q_dtype, seed=n)
    c = x.c
    kv = ops._paged("test", c.k, c.v, c.table, c.len_t, *(c.scales.get(s) for s in ("k_scale", "v_scale")), 0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for window, sinks in ((None, 0), (1500, 70)):
        assert adp.adp_paged_chunk_attention_workspace(kv, heads[0], x.n, window or 0, sinks) > 0
        out = x.call(ops, window=window, sinks=sinks, status=status)
        x.check(out, window=window, sinks=sinks)
        assert torch.equal(out, x.call(ops, window=window, sinks=sinks))
        x.check(x.call(ops, table=wide(x), window=window, sinks=sinks, status=status), window=window, sinks=sinks)
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_prompts_and_single_tokens_of_many_sequences(ops, dtype):  # noqa: F811
    """Pieces of two tiles and of one, cut, on both sides of the 32nd and the 64th sequence."""
    rng = random.Random(9)
    new, old = [rng.choice([0, 1, 1, 30]) for _ in range(70)], [rng.randint(0, 60) for _ in range(70)]
    for b, m, o in ((0, 200, 0), (31, 300, 900), (32, 1, 3000), (63, 40, 2500), (64, 150, 1700), (69, 1, 2000)):
        new[b], old[b] = m, o
    x = Chunk(new, old, (8, 2), 64, 16, dtype, F16, seed=3)
    out = x.call(ops)
    x.check(out)
    assert torch.equal(out, x.call(ops))


@pytest.mark.parametrize("dtype", [F16, E4M3])
@pytest.mark.parametrize("page", [4, 8, 16, 64])
def test_lengths_beyond_the_table_are_cut_to_it_and_reported(ops, page, dtype):  # noqa: F811
    x = Chunk([2 * page, 3], [2 * page, 4 * page - 3], (4, 2), 64, page, dtype, F16, seed=8)
    assert x.c.table.shape[1] == 4  # (both sequences fill it)
    want = x.call(ops)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for b in (0, 1):
        for beyond in (4 * page + 1, 2 ** 31 - 1):
            x.c.len_t[b] = beyond
            out = x.call(ops, status=status)
            assert int(status) == -3 and torch.equal(out, want)
            x.check(out)
            status.zero_()
        x.c.len_t[b] = 4 * page
    x.call(ops, status=status)
    assert int(status) == 0
