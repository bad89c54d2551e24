"""Attention of every sequence's last rows over the pages, against plain 64-bit computations, through ops.paged_chunk_attention."""
import math
import random

import pytest
import torch

from test_gpu_paged import BF16, E4M3, F16, NAN, TYPES, Cache, half_step, ops, raw  # noqa: F401

pytestmark = pytest.mark.gpu


class Chunk:
    """A cache whose sequences hold new[b] + old[b] positions, and queries for the new ones (and `pad` more rows)."""

    def __init__(self, new, old, heads, hd, page, dtype, q_dtype=None, seed=0, pad=0, spare=3):
        self.new, self.old, self.pad = new, old, pad
        self.lens = [a + b for a, b in zip(new, old)]
        self.c = Cache(self.lens, heads[1], hd, page, dtype, seed + 7, q_dtype=q_dtype, spare=spare)
        g = torch.Generator().manual_seed(seed)
        self.n = sum(new)
        self.q = (torch.randn(self.n + pad, heads[0], hd, generator=g) * 1.5).to(self.c.q_dtype).cuda()
        self.cu = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32).cuda()

    def call(self, ops, **kw):
        c = self.c
        a = dict(table=c.table, lens=c.len_t, cu=self.cu, q=self.q)
        a.update({k: kw.pop(k) for k in list(kw) if k in a})
        return ops.paged_chunk_attention(a["q"], c.k, c.v, a["table"], a["lens"], a["cu"], **c.scales, **kw)

    def check(self, out, q=None, window=None, sinks=0, scale=None, skip=(), new=None, lens=None):
        """Every row within the tolerance; skip: (sequence, position) without a page."""
        c, q = self.c, self.q if q is None else q
        hq, hd = q.shape[1:]
        group, scale = hq // c.hkv, hd ** -0.5 if scale is None else scale
        p_type = F16 if c.dtype == E4M3 else c.dtype
        new, lens = new or self.new, lens or self.lens
        at = 0
        for b, (m, n) in enumerate(zip(new, lens)):
            if m == 0:
                continue
            pos = torch.arange(n - m, n, device="cuda")
            key = torch.arange(n, device="cuda")
            seen = key[None] <= pos[:, None]
            if window:
                seen &= (key[None] > pos[:, None] - window) | (key[None] < sinks)
            for s, p in skip:
                if s == b and p < n:
                    seen[:, p] = False
            k, v = (x[b][:n].cuda().transpose(0, 1).repeat_interleave(group, 0) for x in c.kv)  # [hq, n, hd]
            k, v = torch.nan_to_num(k, 0.0), torch.nan_to_num(v, 0.0)
            qb = q[at:at + m].double().transpose(0, 1)
            got = out[at:at + m].double().transpose(0, 1)
            some = seen.any(1)
            assert (got[:, ~some] == 0).all()
            assert torch.isfinite(got).all()
            s = (qb @ k.transpose(1, 2) * scale).masked_fill(~seen, -math.inf)
            p = torch.softmax(s, 2)
            p[:, ~some] = 0
            o, a = p @ v, p @ v.abs()
            # out rounded once; every probability rounded once (relative to a maximum that may be stale by 2^8, which fp16 has
            # room for: 2^-25 of a weight of 1 is half its least step; over e4m3 pages the product with the value scale, at
            # most twice the largest |v|), off by its score's fp32 error (and that of q brought to fp16 beside e4m3
            # codes, 2^-25 of its largest) in numerator and sum, by exp2's, and by the fp32 sums over the keys
            ds = qb.abs() @ k.abs().transpose(1, 2) * (hd + 8) * 2.0 ** -24
            if c.dtype == E4M3:
                ds = ds + qb.abs().amax(2)[..., None] * k.abs().sum(2)[:, None] * 2.0 ** -24
            ds = (ds * abs(scale)).masked_fill(~seen, 0).amax(2)[..., None]
            tol = half_step(c.q_dtype) * o.abs() + a * (half_step(p_type) + 2 * ds + 2.0 ** -19 + n * 2.0 ** -24)
            tol = tol + n * 2.0 ** -25 * 2 * v.abs().amax() * (p_type == F16) + 1e-30
            err = (got - o).abs()
            assert (err <= tol)[:, some].all(), (b, float((err / tol)[:, some].max()))
            at += m


def wide(x, width=3000):
    t = torch.full((len(x.lens), width), -1, dtype=torch.int32, device="cuda")
    t[:, :x.c.table.shape[1]] = x.c.table
    return t


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("heads,page,new,old,window,sinks", [
    ((4, 2), 16, [16], [61], None, 0), ((1, 1), 16, [1], [0], None, 0), ((2, 1), 8, [1, 0, 2, 127, 128, 129], [0, 5, 0, 1, 0, 63], None, 0),
    ((20, 4), 16, [50, 300, 7, 1], [0, 33, 1000, 64], None, 0), ((8, 8), 32, [257, 0], [0, 9], None, 0),
    ((32, 8), 64, [64, 65, 33, 1, 1], [200, 0, 400, 63, 700], None, 0), ((14, 2), 128, [40, 9], [90, 40], None, 0),
    ((128, 1), 16, [5], [130], None, 0), ((4, 4), 1, [3, 70], [10, 0], None, 0), ((24, 2), 4, [30], [41], None, 0),
    ((4, 2), 16, [16], [61], 20, 0), ((20, 4), 16, [300, 1, 40], [500, 700, 0], 100, 4), ((8, 8), 8, [257], [300], 1, 0),
    ((8, 1), 64, [130, 70], [900, 0], 64, 64), ((6, 2), 32, [5, 1, 200], [1000, 77, 400], 200, 130),
    ((4, 1), 2, [9, 60], [200, 30], 33, 17), ((4, 2), 16, [100], [400], 2 ** 31 - 1, 2 ** 31 - 1)])
def test_matches_64_bits(ops, hd, dtype, q_dtype, heads, page, new, old, window, sinks):
    x = Chunk(new, old, heads, hd, page, dtype, q_dtype, seed=hd + page, pad=2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(x.q, 7.0)
    x.call(ops, window=window, sinks=sinks, out=out, status=status)
    assert int(status) == 0
    x.check(out, window=window, sinks=sinks)
    assert (out[x.n:] == 7).all()  # rows behind the last sequence are left as they were
    assert torch.equal(out[:x.n], x.call(ops, window=window, sinks=sinks)[:x.n])
    x.check(x.call(ops, table=wide(x), window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("new,old,window,sinks", [
    ([8], [6000], None, 0), ([1], [9000], None, 0), ([8, 1, 3, 0, 5], [3000, 2500, 7, 90, 0], None, 0), ([700], [3000], None, 0),
    ([3, 150], [6000, 3000], 2500, 100), ([2500], [0], None, 0)])
def test_long_contexts_are_split_and_joined(ops, dtype, q_dtype, new, old, window, sinks):
    for heads, hd, page in (((8, 2), 64, 16), ((4, 4), 128, 64)):
        x = Chunk(new, old, heads, hd, page, dtype, q_dtype, seed=len(new))
        out = x.call(ops, window=window, sinks=sinks)
        x.check(out, window=window, sinks=sinks)
        assert torch.equal(out, x.call(ops, window=window, sinks=sinks))  # the same bits again


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
def test_more_work_than_the_gpu_holds_at_once(ops, dtype, q_dtype):
    """Several pieces of work in a row on every SM, with sequences and tiles that see nothing among them."""
    rng = random.Random(4)
    for new, old in (([500, 0, 33, 300, 200], [100, 40, 600, 0, 1]), ([rng.choice([0, 1, 1, 5, 70]) for _ in range(75)], [rng.randint(0, 200) for _ in range(75)])):
        x = Chunk(new, old, (64, 16), 64, 16, dtype, q_dtype, seed=10)
        out = x.call(ops)
        x.check(out)
        assert torch.equal(out, x.call(ops))


def test_many_sequences(ops):
    """1,100 short sequences: more than one scan of a warp holds."""
    rng = random.Random(8)
    new, old = [rng.randint(0, 3) for _ in range(1100)], [rng.randint(0, 6) for _ in range(1100)]
    x = Chunk(new, old, (4, 2), 64, 4, F16, seed=12)
    x.check(x.call(ops))


def test_scales_negative_zero_and_large_and_growing_scores(ops):
    for dtype, q_dtype in TYPES:
        x = Chunk([150], [100], (4, 2), 64, 16, dtype, q_dtype, seed=1)
        for scale in (0.0, -0.3, 2.0):
            x.check(x.call(ops, scale=scale), scale=scale)
        for scale in (3e38, -3e38):
            q = x.q * 0
            x.check(x.call(ops, q=q, scale=scale), q=q, scale=scale)
    x = Chunk([150], [100], (4, 2), 64, 16, BF16, seed=1)
    for p in range(250):  # later keys' scores grow: O is rescaled
        at = int(x.c.table[0, p // 16]), slice(None), p % 16
        x.c.k[at] = (x.c.k[at].float() * (0.1 + p / 6)).to(BF16)
        x.c.kv[0][0][p] = x.c.k[at].double().cpu()
    x.check(x.call(ops))


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("page", [4, 16, 64])
def test_what_no_row_sees_is_neither_read_nor_looked_up(ops, dtype, q_dtype, page):
    """Pages of which no row sees anything have no number any more, and the other cells that no row sees hold NaN."""
    new, old, window, sinks = [30, 1, 3], [300, 999, 126], 40, 6
    x = Chunk(new, old, (8, 2), 128, page, dtype, q_dtype, seed=3)
    c = x.c
    for b, (m, n) in enumerate(zip(new, x.lens)):
        gone = set(range(sinks, n - m + 1 - window))
        for at in range(-(-n // page)):
            cells = [p for p in range(at * page, (at + 1) * page) if p < n]
            if all(p in gone for p in cells):
                c.table[b, at] = -7
            else:
                for p in cells:
                    if p in gone:
                        i = int(c.table[b, at]), slice(None), p % page
                        if dtype == E4M3:
                            c.scales["k_scale"][i] = c.scales["v_scale"][i] = NAN
                        else:
                            c.k[i] = c.v[i] = NAN
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for table in (c.table, wide(x)):
        x.check(x.call(ops, table=table, window=window, sinks=sinks, status=status), window=window, sinks=sinks)
    assert int(status) == 0


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("value", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("heads,new,old,window,sinks", [((4, 2), [150, 40], [50, 0], None, 0), ((4, 2), [150, 40], [50, 0], 70, 5),
                                                       ((4, 2), [3, 2], [100, 20], 60, 3)])
def test_what_a_row_does_not_see_does_not_reach_it(ops, dtype, q_dtype, value, heads, new, old, window, sinks):
    """Non-finite keys and values: the rows that do not see them, and other sequences, are as if they were zeros; the rows that see
    them are not finite (in the channel of v, or everywhere for k and for e4m3's scales)."""
    for at in (0, 5, old[0], old[0] + new[0] - 2):
        x = Chunk(new, old, heads, 64, 16, dtype, q_dtype, seed=4)
        c = x.c
        i = int(c.table[0, at // 16]), 1, at % 16
        for which in ("v", "k"):
            zeros = {}
            pool = getattr(c, which)
            if dtype == E4M3:
                was = c.scales[which + "_scale"][i].clone()
                clean = x.call(ops, window=window, sinks=sinks)
                c.scales[which + "_scale"][i] = value
                out = x.call(ops, window=window, sinks=sinks)
                c.scales[which + "_scale"][i] = was
            else:
                was = pool[i].clone()
                clean = x.call(ops, window=window, sinks=sinks)
                pool[i][7] = value if which == "v" else NAN
                out = x.call(ops, window=window, sinks=sinks)
                pool[i] = was
            pos = torch.arange(old[0], old[0] + new[0])
            sees = pos >= at
            if window:
                sees &= (pos < at + window) | (at < sinks)
            blind = torch.ones(x.n, 4, 64, dtype=torch.bool)
            if which == "v" and dtype != E4M3:
                blind[:new[0], 2:, 7] = ~sees[:, None]
            else:
                blind[:new[0], 2:] = ~sees[:, None, None]
            blind = blind.cuda()
            assert torch.equal(out[blind], clean[blind]), (at, which)
            if which == "k" and dtype == E4M3 and not math.isnan(value):
                continue  # (a key of infinities may score -infinity: weight 0)
            assert not torch.isfinite(out[~blind]).any(), (at, which)
            if which == "v" and dtype != E4M3 and not math.isnan(value):
                assert (out[~blind] == value).all()


def test_strided_queries_outputs_and_interleaved_pages(ops):
    x = Chunk([50, 3, 0, 7], [30, 33, 5, 0], (8, 2), 128, 16, BF16, seed=9)
    c = x.c
    fused = torch.full((60, 20, 128), NAN, dtype=BF16, device="cuda")
    fused[:, 5:13] = x.q
    both = torch.full((c.k.shape[0], 3, 2, 16, 128), NAN, dtype=BF16, device="cuda")  # K, something else and V by page
    both[:, 0], both[:, 2] = c.k, c.v
    out = torch.full((60, 12, 128), 5.0, dtype=BF16, device="cuda")
    got = ops.paged_chunk_attention(fused[:, 5:13], both[:, 0], both[:, 2], c.table, c.len_t, x.cu, out=out[:, 2:10])
    x.check(got)
    assert (out[:, :2] == 5).all() and (out[:, 10:] == 5).all()


@pytest.mark.parametrize("q_dtype,hd", [(F16, 64), (BF16, 128)])
@pytest.mark.parametrize("page", [1, 4, 16, 64])
def test_codes_and_scales_side_by_side_at_odd_addresses(ops, page, q_dtype, hd):
    """K's and V's codes of a page one after the other; their scales an odd number of floats apart, from an odd one on."""
    x = Chunk([50, 3, 0, 7], [130, 33, 5, 0], (8, 2), hd, page, E4M3, q_dtype, seed=9)
    c = x.c
    n = c.k.shape[0]
    codes = torch.full((n, 2, 2, page, hd), NAN, device="cuda").to(E4M3)
    raw(codes)[:, 0], raw(codes)[:, 1] = raw(c.k), raw(c.v)
    step = 4 * page + 3
    floats = torch.full((n * step + 1,), NAN, device="cuda")
    k_scale, v_scale = (floats.as_strided((n, 2, page), (step, page, 1), at) for at in (1, 1 + 2 * page))
    k_scale.copy_(c.scales["k_scale"])
    v_scale.copy_(c.scales["v_scale"])
    got = ops.paged_chunk_attention(x.q, codes[:, 0], codes[:, 1], c.table, c.len_t, x.cu, k_scale=k_scale, v_scale=v_scale)
    x.check(got)
    assert torch.equal(got, x.call(ops))


def test_two_threads(ops):
    """Calls of two threads of the host, each on its own stream."""
    import threading
    cases = [Chunk([7, 90], [700, 20], (8, 2), 64, 16, F16, seed=s) for s in (31, 32)]
    want, got = [x.call(ops) for x in cases], [None, None]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            results = [cases[i].call(ops) for _ in range(30)]
            torch.cuda.current_stream().synchronize()
        got[i] = all(torch.equal(r, want[i]) for r in results)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert got == [True, True]


@pytest.mark.parametrize("page", [4, 8, 16])
@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_bad_pages_lengths_and_offsets_are_reported(ops, page, dtype):
    x = Chunk([70, 20], [30, 0], (4, 2), 64, page, dtype, F16, seed=8)
    c = x.c
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = int(c.table[0, 2])
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        status.zero_()
        c.table[0, 2] = bad
        x.check(x.call(ops, status=status), skip={(0, p) for p in range(2 * page, 3 * page)})
        assert int(status) == -1
    c.table[0, 2] = good
    x = Chunk([2 * page, 20], [4 * page - 2 * page, 0], (4, 2), 64, page, dtype, F16, seed=8)
    fits = x.c.table.shape[1] * page  # the longest sequence that the table holds
    status.zero_()
    if fits == 4 * page:
        x.c.len_t[0] = 2 ** 31 - 1
        x.check(x.call(ops, status=status))
        assert int(status) == -3
    status.zero_()
    x.c.len_t[0] = -5  # no positions: its rows give zeros
    out = x.call(ops, status=status)
    assert int(status) == -1 and (out[:2 * page] == 0).all()
    status.zero_()
    x.c.len_t[0] = page  # more rows than positions: the first ones give zeros
    out = x.call(ops, status=status)
    assert int(status) == -1 and (out[:page] == 0).all() and torch.isfinite(out).all() and (out[page:] != 0).any(-1).all()
    n = x.n
    for cu in ([0, n + 30, n], [-5, 10, n], [0, 2 ** 31 - 1, -2 ** 31], [n, 10, 0], [3, 10, n]):
        x = Chunk([2 * page, 20], [2 * page, 0], (4, 2), 64, page, dtype, F16, seed=8)
        status.zero_()
        x.call(ops, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), status=status)
        assert int(status) == -1


def test_offsets_past_32_bits(ops):
    """A pool of 5 GB whose used pages lie at its end."""
    page, hkv, hd = 64, 8, 128
    n_pages = 5 * 2 ** 30 // (page * hkv * hd * 2) + 3
    pools = [torch.zeros(n_pages, hkv, page, hd, dtype=F16, device="cuda") for _ in range(2)]
    x = Chunk([20], [80], (8, 8), hd, page, F16, seed=10)
    for pool, src in zip(pools, (x.c.k, x.c.v)):
        pool[n_pages - 2], pool[n_pages - 1] = src[x.c.table[0, 0]], src[x.c.table[0, 1]]
    table = torch.tensor([[n_pages - 2, n_pages - 1]], dtype=torch.int32, device="cuda")
    x.check(ops.paged_chunk_attention(x.q, *pools, table, x.c.len_t, x.cu))
    codes = [torch.zeros(2 * n_pages, hkv, page, hd, dtype=E4M3, device="cuda") for _ in range(2)]
    scales = [torch.zeros(2 * n_pages, hkv, page, device="cuda") for _ in range(2)]
    x = Chunk([20], [80], (8, 8), hd, page, E4M3, F16, seed=10)
    for pool, src in ((codes[0], x.c.k), (codes[1], x.c.v), (scales[0], x.c.scales["k_scale"]), (scales[1], x.c.scales["v_scale"])):
        for i in (0, 1):
            p = pool[2 * n_pages - 2 + i]
            (p.view(torch.uint8) if p.dtype == E4M3 else p).copy_(src[x.c.table[0, i]].view(torch.uint8) if p.dtype == E4M3 else src[x.c.table[0, i]])
    table = torch.tensor([[2 * n_pages - 2, 2 * n_pages - 1]], dtype=torch.int32, device="cuda")
    x.check(ops.paged_chunk_attention(x.q, *codes, table, x.c.len_t, x.cu, k_scale=scales[0], v_scale=scales[1]))


@pytest.mark.parametrize("dtype,q_dtype", [(BF16, BF16), (E4M3, F16)])
def test_another_stream_and_captured_graphs_with_changing_lengths(ops, dtype, q_dtype):
    x = Chunk([130, 70], [900, 20], (8, 2), 64, 16, dtype, q_dtype, seed=6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = x.call(ops)
    torch.cuda.current_stream().wait_stream(s)
    x.check(out)
    graphs = []
    for _ in range(2):  # graphs of one cache: each has a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = x.call(ops)
        graphs.append((g, out))
    for new, lens in (([130, 70], [1030, 90]), ([1, 199], [20, 90]), ([200, 0], [220, 0]), ([130, 3], [900, 3])):
        if new[1] > lens[1]:
            continue
        x.cu.copy_(torch.tensor([0, new[0], new[0] + new[1]], dtype=torch.int32))
        x.c.len_t.copy_(torch.tensor(lens, dtype=torch.int32))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            x.check(out, new=new, lens=lens)


def test_calls_at_once_and_the_result_in_the_queries_place(ops):
    xs = [Chunk([300, 5, 1], [500, 3000, 4000], (16, 4), 128, 16, dtype, BF16, seed=13) for dtype in (BF16, E4M3)]
    want = [x.call(ops) for x in xs]
    for x, w in zip(xs, want):
        x.check(w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s, x, w in zip(streams, xs, want):
            with torch.cuda.stream(s):
                got.append((x.call(ops), w))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in got)
    over = xs[0].q.clone()
    xs[0].call(ops, q=over, out=over)
    assert torch.equal(over, want[0])


@pytest.mark.parametrize("dtype,q_dtype", [(F16, F16), (E4M3, F16), (E4M3, BF16)])
@pytest.mark.parametrize("new", [3, 300])
def test_a_dominating_key_leaves_the_others_their_weights(ops, dtype, q_dtype, new):
    """Key 0 outweighs every other one by 2^25 and its V is 0: the result is the others' share alone, whose fp16 weights must not
    vanish beside it."""
    n, hd, bits = 4096, 64, 25
    x = Chunk([new], [n - new], (4, 1), hd, 16, dtype, q_dtype, seed=20)
    c = x.c
    g = torch.Generator().manual_seed(41)
    v = (torch.rand(n, 1, hd, generator=g) + 0.5).to(dtype)
    k = torch.zeros(n, 1, hd).to(dtype)
    k.view(torch.uint8 if dtype == E4M3 else torch.int16)[0, 0, 0] = torch.ones(1).to(dtype).view(torch.uint8 if dtype == E4M3 else torch.int16)[0]
    raw(v)[0] = 0
    for pool, y in ((c.k, k), (c.v, v)):
        for p0 in range(0, n, 16):
            raw(pool)[int(c.table[0, p0 // 16])] = raw(y)[p0:p0 + 16].transpose(0, 1).cuda()
    for s in c.scales.values():
        s.fill_(1.0)
    q = torch.zeros_like(x.q)
    q[:, :, 0] = float(bits)  # (exact in every type; exponents of base 2)
    out = x.call(ops, q=q, scale=math.log(2)).double()
    s = torch.einsum("ihd,jd->hij", q.double(), k[:, 0].cuda().double()) * math.log(2)
    seen = torch.arange(n, device="cuda")[None] <= torch.arange(n - new, n, device="cuda")[:, None]
    p = torch.softmax(s.masked_fill(~seen, -math.inf), 2)
    vd = v[:, 0].cuda().double()
    o = torch.einsum("hij,jd->ihd", p, vd)
    # as in check (V is positive), but fp16's least half step 2^-25 is one of weights that are held 2^7 times larger
    ds = bits * math.log(2) * (hd + 8) * 2.0 ** -24
    tol = o * (half_step(q_dtype) + half_step(F16) + 2 * ds + 2.0 ** -19 + n * 2.0 ** -24) + 2.0 ** -32 * vd.sum(0) + torch.finfo(q_dtype).smallest_normal * half_step(q_dtype)
    assert ((out - o).abs() <= tol).all(), float(((out - o).abs() / tol).max())


@pytest.mark.parametrize("q_dtype", [F16, BF16])
def test_value_scales_at_both_ends_of_fp32(ops, q_dtype):
    """Positions of zeros (the least scale), of tiny and of huge scales in one sequence: the result is the huge ones' sum, or
    the tiny ones' where there are no others, and always finite; one that hardly counts takes no bits from the others."""
    n = 96
    for scales in ([2.0 ** -126] * 96, [2.0 ** -100] * 96, [2.0 ** -126] * 64 + [1.0] * 32, [2.0 ** 100] * 32 + [2.0 ** -100] * 64,
                   [2.0 ** (5 * (i % 40) - 100) for i in range(96)]):
        x = Chunk([5], [n - 5], (4, 1), 64, 16, E4M3, q_dtype, seed=43)
        c = x.c
        for p, f in enumerate(scales):
            at = int(c.table[0, p // 16]), 0, p % 16
            c.kv[1][0][p] *= f / float(c.scales["v_scale"][at])
            c.scales["v_scale"][at] = f
        out = x.call(ops).double().cpu()
        k, v, sc = c.kv[0][0][:, 0], c.kv[1][0][:, 0], torch.tensor(scales, dtype=torch.float64)
        for i in range(5):
            m = n - 4 + i
            q = x.q[i].double().cpu()
            p = torch.softmax(q @ k[:m].T * 64 ** -0.5, 1)
            o, a = p @ v[:m], p @ v[:m].abs()
            ds = ((q.abs() @ k[:m].abs().T) * 72 * 2.0 ** -24 + q.abs().amax(1)[:, None] * k[:m].abs().sum(1) * 2.0 ** -24).amax(1) * 64 ** -0.5
            largest = (p * sc[:m]).amax(1)[:, None]
            tol = half_step(q_dtype) * o.abs() + a * (half_step(F16) + 2 * ds[:, None] + 2.0 ** -19 + n * 2.0 ** -24)
            tol = tol + n * 448 * 2.0 ** -32 * largest + torch.finfo(q_dtype).smallest_normal * half_step(q_dtype) * 2
            big = o.abs() > torch.finfo(q_dtype).max  # (what the result's type cannot hold becomes an infinity)
            assert torch.isinf(out[i][big]).all()
            assert ((out[i] - o).abs() <= tol)[~big].all(), (scales[0], i, float(((out[i] - o).abs() / tol)[~big].max()))


def test_workspace_and_refusals(ops):
    from autoregressive_decode_persistent_gb300 import adp
    x = Chunk([6, 10], [6000, 0], (8, 2), 128, 16, F16, seed=22)
    c = x.c
    kv = ops._paged("test", c.k, c.v, c.table, c.len_t, None, None, 0)
    need = adp.adp_paged_chunk_attention_workspace(kv, 8, 16, 0, 0)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # its contents do not matter
    x.check(x.call(ops, workspace=ws))
    for kw in (dict(workspace=ws[:need - 1]), dict(workspace=ws.float()), dict(window=0), dict(window=-1), dict(window=5, sinks=-1), dict(sinks=3),
               dict(q=x.q.float()), dict(q=x.q[:, :7]), dict(q=x.q[0]), dict(q=x.q[:, :, :64]), dict(q=x.q.to(BF16)), dict(cu=x.cu[:2]), dict(cu=x.cu.long()),
               dict(out=x.q[:15]), dict(scale=NAN), dict(scale=math.inf)):
        with pytest.raises(adp.AdpError):
            x.call(ops, **kw)
    small = Chunk([6, 10], [300, 0], (8, 2), 128, 16, F16, seed=22)
    kv = ops._paged("test", small.c.k, small.c.v, small.c.table, small.c.len_t, None, None, 0)
    assert adp.adp_paged_chunk_attention_workspace(kv, 8, 16, 0, 0) == 0
    none = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert ops.paged_chunk_attention(x.q[:0], c.k, c.v, none, cu[:0], cu).shape == (0, 8, 128)
    assert ops.paged_chunk_attention(x.q[:0], c.k, c.v, c.table, c.len_t, torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 8, 128)


@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_a_server_in_small(ops, dtype):
    """A run of the operators together: prompts appended and attended in chunks beside other requests' single tokens, with a
    window, and a last step of single tokens alone."""
    hq, hkv, hd, window, sinks, eps = 8, 2, 64, 50, 4, 1e-5
    prompts = [120, 33, 64]
    c = Cache(prompts, hkv, hd, 16, dtype, 5, q_dtype=F16)
    g = torch.Generator().manual_seed(2)
    rows = [torch.randn(n, hq + 2 * hkv, hd, generator=g).to(F16).cuda() for n in prompts]
    at = torch.arange(128, dtype=torch.float64)[:, None] * 1e4 ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64) / hd)
    cos, sin = torch.cos(at).float().cuda(), torch.sin(at).float().cuda()
    gain = (1 + torch.randn(hd, generator=g) / 8).to(F16).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    done, results, turned = [0, 0, 0], [[], [], []], [[], [], []]
    for step in ([70, 32, 0], [1, 1, 40], [48, 0, 23], [1, 0, 1]):
        qkv = torch.cat([r[d:d + m] for r, d, m in zip(rows, done, step)])
        done = [d + m for d, m in zip(done, step)]
        lens, cu = torch.tensor(done, **i32), torch.tensor([0] + step, device="cuda").cumsum(0).to(torch.int32)
        q = ops.paged_kv_append(c.k, c.v, c.table, lens, cu, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], cos, sin, q_gain=gain,
                                k_gain=gain, eps=eps, **c.scales)
        out = ops.paged_chunk_attention(q, c.k, c.v, c.table, lens, cu, window=window, sinks=sinks, **c.scales)
        if max(step) == 1:  # single tokens: the other operator agrees
            some = [b for b in range(3) if step[b]]
            one = ops.paged_attention(q, c.k, c.v, c.table[some].contiguous(), lens[some].contiguous(), window=window, sinks=sinks, **c.scales)
            x = Chunk.__new__(Chunk)
            kr, vr = ops.paged_kv_read(c.k, c.v, c.table, lens, torch.tensor([0] + done, device="cuda").cumsum(0).to(torch.int32), sum(done), dtype=torch.float32, **c.scales)
            ends = [0, done[0], done[0] + done[1], sum(done)]
            c.kv = [[y[ends[b]:ends[b + 1]].double() for b in range(3)] for y in (kr, vr)]
            x.c, x.new, x.lens, x.q = c, step, done, q
            x.check(out, window=window, sinks=sinks)
            x.check(one, window=window, sinks=sinks)
        for b in range(3):
            lo, hi = int(cu[b]), int(cu[b + 1])
            results[b].append(out[lo:hi])
            turned[b].append(q[lo:hi])
    # all prompts in one call over the same cache
    x = Chunk.__new__(Chunk)
    x.c, x.new, x.lens, x.q = c, prompts, prompts, torch.cat([torch.cat(t) for t in turned])
    assert done == [120, 33, 64]
    whole = ops.paged_chunk_attention(x.q, c.k, c.v, c.table, torch.tensor(prompts, **i32), torch.tensor([0] + prompts, device="cuda").cumsum(0).to(torch.int32), window=window, sinks=sinks, **c.scales)
    x.check(whole, window=window, sinks=sinks)
    x.check(torch.cat([torch.cat(r) for r in results]), window=window, sinks=sinks)
