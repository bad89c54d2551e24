"""The paged KV cache operators against plain 64-bit computations, through the tensor wrappers of ops.py."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN = float("nan")


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "a CUDA GPU is required"
    from autoregressive_decode_persistent_gb300 import build, ops
    build.build()
    return ops


def half_step(t):
    return torch.finfo(t).eps / 2


def raw(t):
    """The bits of a pool, in a type that CPU and GPU can index and compare."""
    return t.view(torch.uint8 if t.dtype == E4M3 else torch.int16)


class Cache:
    """A pool with NaN in every cell that no sequence holds, and the values its sequences hold, on the CPU."""

    def __init__(self, lens, hkv, hd, page, dtype, seed, spare=3, q_dtype=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.page, self.lens, self.hd, self.hkv, self.dtype, self.q_dtype = page, lens, hd, hkv, dtype, q_dtype or dtype
        n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=g).tolist()
        table = torch.full((len(lens), max(1, max(need, default=1))), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            for i in range(n):
                table[b, i] = order.pop()
        self.kv, pools, scales = [], [], []
        for _ in range(2):
            pool = torch.full((n_pages, hkv, page, hd), NAN).to(dtype)
            scale = torch.full((n_pages, hkv, page), NAN)
            held = []
            for b, n in enumerate(lens):
                x = torch.randn(n, hkv, hd, generator=g) * (1 + 2 * torch.rand(n, hkv, 1, generator=g))
                if dtype == E4M3:
                    s = x.abs().amax(-1) / 448
                    codes = (x / s[..., None]).to(E4M3)
                    held.append(codes.double() * s.double()[..., None])
                else:
                    s, codes = torch.ones(n, hkv), x.to(dtype)
                    held.append(codes.double())
                for p in range(n):
                    at = int(table[b, p // page])
                    raw(pool)[at, :, p % page] = raw(codes)[p]
                    scale[at, :, p % page] = s[p]
            self.kv.append(held)
            pools.append(pool.cuda())
            scales.append(scale.cuda())
        self.k, self.v = pools
        self.scales = dict(k_scale=scales[0], v_scale=scales[1]) if dtype == E4M3 else {}
        self.table, self.len_t = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def attend64(q, k, v, scale):
    """One sequence in 64 bits: out, and what the tolerance needs: sum p |v|, and the scores' error bound in fp32."""
    hq, hd = q.shape
    g = hq // k.shape[1]
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.einsum("hd,nhd->hn", q, k) * scale
    p = torch.softmax(s, 1)
    o = torch.einsum("hn,nhd->hd", p, v)
    # fp32 sums of head_dim products, the scales, and q brought to fp16 beside e4m3 codes (2^-25 of its largest)
    ds = (torch.einsum("hd,nhd->hn", q.abs(), k.abs()) * (hd + 8) * 2.0 ** -24
          + q.abs().amax(1)[:, None] * k.abs().sum(2).T * 2.0 ** -24).amax(1) * abs(scale)
    return o, torch.einsum("hn,nhd->hd", p, v.abs()), ds, v.abs().amax()


def check_attention(out, q, cache, lens=None, scale=None, skip=()):
    scale = cache.hd ** -0.5 if scale is None else scale
    p_type = F16 if cache.dtype == E4M3 else cache.dtype
    out, q = out.double().cpu(), q.double().cpu()
    assert torch.isfinite(out).all()
    for b, n in enumerate(lens or cache.lens):
        keep = [p for p in range(n) if (b, p) not in skip]
        if not keep:
            assert (out[b] == 0).all(), b
            continue
        o, a, ds, vmax = attend64(q[b], cache.kv[0][b][keep], cache.kv[1][b][keep], scale)
        # out rounded once; every probability rounded once (fp16 below 2^-14: half its least step, times at most
        # twice the largest |v|), off by its score's error (numerator and sum) and exp2's; fp32 sums over n
        tol = half_step(cache.q_dtype) * o.abs() + a * (half_step(p_type) + 2 * ds[:, None] + 2.0 ** -19 + n * 2.0 ** -24)
        tol = tol + n * 2.0 ** -25 * 2 * vmax * (p_type == F16) + 1e-30
        err = (out[b] - o).abs()
        assert (err <= tol).all(), (b, n, float((err / tol).max()))


def run(lens, heads, hd, page, dtype, q_dtype=None, seed=0):
    cache = Cache(lens, heads[1], hd, page, dtype, seed + 7, q_dtype=q_dtype)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(len(lens), heads[0], hd, generator=g) * 1.5).to(cache.q_dtype).cuda()
    return cache, q


def paged(ops, q, c, **kw):
    return ops.paged_attention(q, c.k, c.v, c.table, c.len_t, **c.scales, **kw)


TYPES = [(F16, F16), (BF16, BF16), (E4M3, F16), (E4M3, BF16)]


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("heads,page,lens", [
    ((4, 2), 16, [77]), ((20, 4), 16, [513, 0, 1, 15, 16, 17, 33]), ((8, 8), 32, [1, 2, 31, 32, 65]),
    ((8, 1), 64, [0, 0, 200, 0]), ((14, 2), 8, [9, 100, 3]), ((24, 2), 128, [129, 40]), ((16, 1), 1, [5, 20]),
    ((20, 1), 16, [50, 7]), ((34, 2), 4, [30, 31])])
def test_attention_matches_64_bits(ops, hd, dtype, q_dtype, heads, page, lens):
    c, q = run(lens, heads, hd, page, dtype, q_dtype, seed=hd + page)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_attention(paged(ops, q, c, status=status), q, c)
    assert int(status) == 0


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
def test_long_and_ragged_contexts_are_split_and_joined(ops, dtype, q_dtype):
    rng = random.Random(5)
    for lens in ([6000], [3001, 5, 0, 2500], [rng.randint(0, 40) for _ in range(200)], [1] * 70 + [2000]):
        c, q = run(lens, (8, 2), 64, 16, dtype, q_dtype, seed=len(lens))
        out = paged(ops, q, c)
        check_attention(out, q, c)
        assert torch.equal(out, paged(ops, q, c))  # the same bits again
        wide = torch.full((len(lens), 20000), -1, dtype=torch.int32, device="cuda")  # (the even split at any length)
        wide[:, :c.table.shape[1]] = c.table
        out = ops.paged_attention(q, c.k, c.v, wide, c.len_t, **c.scales)
        check_attention(out, q, c)
        assert torch.equal(out, ops.paged_attention(q, c.k, c.v, wide, c.len_t, **c.scales))


def test_more_sequences_than_one_scan_of_a_warp_holds(ops):
    lens = [(i * 7) % 5 for i in range(1100)]  # (more segments than can be resident: the even split)
    c, q = run(lens, (2, 1), 64, 4, F16, seed=1)
    check_attention(paged(ops, q, c), q, c)


def test_scales_negative_zero_and_large(ops):
    for scale in (0.0, -0.2, 3.0):
        c, q = run([70, 3], (4, 2), 64, 16, BF16, seed=3)
        check_attention(paged(ops, q, c, scale=scale), q, c, scale=scale)


def test_values_of_very_different_scale_in_an_e4m3_cache(ops):
    """The value scales of one sequence differ by 2^40: the small ones' share is below half a step of the large
    ones' sum, and no intermediate leaves fp16's range."""
    c, q = run([64], (4, 1), 128, 16, E4M3, BF16, seed=4)
    f = torch.ones(64, dtype=torch.float64)
    f[:40] = 2.0 ** -30
    f[50] = 2.0 ** 10
    for p in range(64):
        c.scales["v_scale"][c.table[0, p // 16], 0, p % 16] *= float(f[p])
    c.kv[1][0] *= f[:, None, None]
    check_attention(paged(ops, q, c), q, c)


def test_large_scores_and_infinities_in_k(ops):
    c, q = run([40], (2, 1), 64, 16, BF16, seed=6)
    check_attention(paged(ops, q * 64, c), q * 64, c)
    # a key of -inf in one channel, of the sign that q has: its score is -inf, its weight 0
    q = q.abs() + 0.1
    c.k[c.table[0, 0], 0, 3, 5] = -math.inf
    check_attention(paged(ops, q, c), q, c, skip={(0, 3)})
    c.k[c.table[0, 0], 0, 3, 5] = NAN
    assert torch.isnan(paged(ops, q, c)).all()


@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_bad_pages_and_lengths_are_left_out_and_reported(ops, page, dtype):
    c, q = run([100, 20], (4, 2), 64, page, dtype, F16, seed=8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        status.zero_()
        c.table[0, 2] = bad
        out = paged(ops, q, c, status=status)
        check_attention(out, q, c, skip={(0, p) for p in range(2 * page, 3 * page)})
        assert int(status) == -1
    c, q = run([4 * page, 20], (4, 2), 64, page, dtype, F16, seed=8)
    status.zero_()
    c.len_t[0] = 2 ** 31 - 1
    check_attention(paged(ops, q, c, status=status), q, c)
    assert int(status) == -3
    c.len_t[0] = -5
    check_attention(paged(ops, q, c, status=status), q, c, lens=[0, 20])
    assert int(status) == -1


def test_strided_queries_outputs_and_interleaved_pages(ops):
    c, q = run([50, 33, 0, 7], (8, 2), 128, 16, BF16, seed=9)
    fused = torch.full((4, 20, 128), NAN, dtype=BF16, device="cuda")
    fused[:, 5:13] = q
    both = torch.full((c.k.shape[0], 3, 2, 16, 128), NAN, dtype=BF16, device="cuda")  # K, something else and V by page
    both[:, 0], both[:, 2] = c.k, c.v
    out = torch.full((4, 12, 128), 5.0, dtype=BF16, device="cuda")
    got = ops.paged_attention(fused[:, 5:13], both[:, 0], both[:, 2], c.table, c.len_t, out=out[:, 2:10])
    check_attention(got, q, c)
    assert (out[:, :2] == 5).all() and (out[:, 10:] == 5).all()


def test_offsets_past_32_bits(ops):
    """A pool of 5 GB whose used pages lie at its end."""
    page, hkv, hd = 64, 8, 128
    n_pages = 5 * 2 ** 30 // (page * hkv * hd * 2) + 3
    pools = [torch.zeros(n_pages, hkv, page, hd, dtype=F16, device="cuda") for _ in range(2)]
    c, q = run([100], (8, 8), hd, page, F16, seed=10)
    for pool, src in zip(pools, (c.k, c.v)):
        pool[n_pages - 2], pool[n_pages - 1] = src[c.table[0, 0]], src[c.table[0, 1]]
    table = torch.tensor([[n_pages - 2, n_pages - 1]], dtype=torch.int32, device="cuda")
    check_attention(ops.paged_attention(q, *pools, table, c.len_t), q, c)
    cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    k, v = ops.paged_kv_read(*pools, table, c.len_t, cu, 100)
    assert torch.equal(k.double().cpu(), c.kv[0][0]) and torch.equal(v.double().cpu(), c.kv[1][0])
    ops.paged_kv_write(*pools, table, c.len_t, cu, v, k)
    assert torch.equal(pools[0][n_pages - 1, :, :36].transpose(0, 1), v[64:])


def test_another_stream_and_captured_graphs_with_changing_lengths(ops):
    c, q = run([300, 10], (8, 2), 64, 16, F16, seed=11)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = paged(ops, q, c)
    torch.cuda.current_stream().wait_stream(s)
    check_attention(out, q, c)
    wide = torch.full((2, 20000), -1, dtype=torch.int32, device="cuda")  # (the even split, with its second launch)
    wide[:, :c.table.shape[1]] = c.table
    graphs, outs = [], []
    for i in range(4):  # graphs of one cache: each has a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(paged(ops, q, c) if i < 2 else ops.paged_attention(q, c.k, c.v, wide, c.len_t))
        graphs.append(g)
    for lens in ([300, 10], [17, 0], [299, 5]):
        c.len_t.copy_(torch.tensor(lens, dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            check_attention(out, q, c, lens=lens)


# ---------------------------------------------------------------- writing and reading

def e4m3_nearest(y):
    """The e4m3 value nearest to each fp64 y, |y| <= 448, ties to even."""
    step = torch.exp2((torch.frexp(y)[1].double().clamp(min=-5) - 4))
    return torch.round(y / step) * step


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [F16, BF16, F32])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
@pytest.mark.parametrize("hkv,page,new,old", [(4, 16, [1, 1, 1, 1], [1000, 0, 15, 16]), (1, 1, [5], [0]),
                                              (2, 8, [0, 17, 0, 9], [3, 4, 0, 0]), (3, 64, [130], [1]),
                                              (8, 16, [1] * 40, list(range(40)))])
def test_rows_written_and_read_back(ops, hd, rows, dtype, hkv, page, new, old):
    lens = [a + b for a, b in zip(new, old)]
    c = Cache(lens, hkv, hd, page, dtype, 3)
    g = torch.Generator().manual_seed(hd)
    n, pad = sum(new), 3
    k, v = ((torch.randn(n + pad, hkv, hd, generator=g) * 2).to(rows) for _ in range(2))
    k[0, 0] = 0  # a row of zeros
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    before = [c.k.clone(), c.v.clone()]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.paged_kv_write(c.k, c.v, c.table, c.len_t, cu, k.cuda(), v.cuda(), status=status, **c.scales)
    assert int(status) == 0
    at = [(b, p) for b in range(len(new)) for p in range(old[b], lens[b])]
    page_of = torch.tensor([int(c.table[b, p // page]) for b, p in at])
    slot = torch.tensor([p % page for b, p in at])
    written = torch.zeros(c.k.shape[0], page, dtype=torch.bool)
    written[page_of, slot] = True
    for x, pool, was, name in ((k[:n], c.k, before[0], "k_scale"), (v[:n], c.v, before[1], "v_scale")):
        got = pool.cpu().double()[page_of, :, slot]
        if dtype == E4M3:
            s = c.scales[name].cpu()[page_of, :, slot]
            want_s = (x.float().abs().amax(-1) / 448).clamp(min=2.0 ** -126)  # fp32 division, rounded to nearest
            assert torch.equal(s, want_s)
            assert torch.equal(got, e4m3_nearest((x.float() / want_s[..., None]).double()))
        else:
            assert torch.equal(got, x.to(dtype).double())
        same = (raw(pool) == raw(was)).all(-1).cpu()  # [pages, heads, page]
        assert same.transpose(1, 2)[~written].all()  # nothing else changed
    out = tuple(torch.full((n + pad, hkv, hd), 7.0, dtype=rows, device="cuda") for _ in range(2))
    ops.paged_kv_read(c.k, c.v, c.table, c.len_t, cu, n + pad, out=out, status=status, **c.scales)
    assert int(status) == 0
    for pool, got, name in ((c.k, out[0], "k_scale"), (c.v, out[1], "v_scale")):
        want = pool.cpu().float()[page_of, :, slot]
        if dtype == E4M3:
            want = want * c.scales[name].cpu()[page_of, :, slot][..., None]
        assert torch.equal(got[:n].cpu(), want.to(rows))
        assert (got[n:] == 7).all()  # rows behind the last sequence are left as they were


def test_rows_that_are_slices_of_a_fused_projection(ops):
    c = Cache([40], 2, 128, 16, BF16, 5)
    qkv = torch.randn(40, 8, 128, device="cuda").to(BF16)
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    ops.paged_kv_write(c.k, c.v, c.table, c.len_t, cu, qkv[:, 4:6], qkv[:, 6:8])
    back = torch.zeros(40, 6, 128, dtype=BF16, device="cuda")
    ops.paged_kv_read(c.k, c.v, c.table, c.len_t, cu, 40, out=(back[:, :2], back[:, 3:5]))
    assert torch.equal(back[:, :2], qkv[:, 4:6]) and torch.equal(back[:, 3:5], qkv[:, 6:8])
    assert (back[:, 2] == 0).all() and (back[:, 5] == 0).all()


@pytest.mark.parametrize("value", [math.inf, -math.inf, NAN])
def test_a_quantised_row_with_a_non_finite_value_reads_back_as_nan(ops, value):
    c = Cache([4], 2, 64, 16, E4M3, 6)
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    k, v = torch.randn(2, 4, 2, 64, device="cuda")
    k[2, 1, 30] = value
    ops.paged_kv_write(c.k, c.v, c.table, c.len_t, cu, k, v, **c.scales)
    kr, vr = ops.paged_kv_read(c.k, c.v, c.table, c.len_t, cu, 4, dtype=F32, **c.scales)
    bad = torch.isnan(kr).cpu()
    assert bad[2, 1].all() and bad.sum() == 64 and torch.isfinite(vr).all()


def test_tiny_and_huge_rows_quantise_without_overflow(ops):
    c = Cache([3], 1, 64, 16, E4M3, 6)
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    k = torch.randn(3, 1, 64)
    k[0] = (k[0].double() * (1e-42 / float(k[0].abs().max()))).float()
    k[1] *= 3e38 / k[1].abs().max()
    ops.paged_kv_write(c.k, c.v, c.table, c.len_t, cu, k.cuda(), k.cuda(), **c.scales)
    kr, _ = ops.paged_kv_read(c.k, c.v, c.table, c.len_t, cu, 3, dtype=F32, **c.scales)
    top = k.double().abs().amax(-1, keepdim=True)
    # half a step of the code (2^-4 of the value, at least half of e4m3's least step 2^-9), and fp32's roundings
    tol = k.double().abs() * (2.0 ** -4 + 2.0 ** -20) + torch.clamp(top / 448, min=2.0 ** -126) * 2.0 ** -10 * 1.001 + 2.0 ** -148
    assert ((kr.double().cpu() - k.double()).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_rows_without_a_page_are_reported(ops, dtype):
    c = Cache([20, 5], 1, 64, 8, dtype, 7)
    cu = torch.tensor([0, 20, 25], dtype=torch.int32, device="cuda")
    x = torch.randn(25, 1, 64, device="cuda")
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.table[0, 1] = bad
        ops.paged_kv_write(c.k, c.v, c.table, c.len_t, cu, x, x, status=status, **c.scales)
        assert int(status) == -1
        status.zero_()
        k, v = ops.paged_kv_read(c.k, c.v, c.table, c.len_t, cu, 25, dtype=F32, status=status, **c.scales)
        assert int(status) == -1
        assert (k[8:16] == 0).all() and (v[8:16] == 0).all() and (k[:8] != 0).any() and (k[16:] != 0).any()
    # more rows than positions, and a length behind the table
    for lens in ([3, 5], [1000, 5], [-1, 5], [2 ** 31 - 1, 5]):
        c = Cache([20, 5], 1, 64, 8, dtype, 7)
        c.len_t.copy_(torch.tensor(lens, dtype=torch.int32))
        was = raw(c.k).clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.paged_kv_write(c.k, c.v, c.table, c.len_t, cu, x, x, status=status, **c.scales)
        assert int(status) == -1
        changed = (raw(c.k) != was).any(-1)[:, 0].sum(1).tolist()  # cells by page
        first, second = [int(p) for p in c.table[0].tolist()], int(c.table[1, 0])
        assert changed[second] == 5
        assert [changed[p] for p in first] == ([3, 0, 0] if lens[0] == 3 else [0, 0, 0])


def test_written_then_attended(ops):
    """A run of them together: prompts written, a step's rows appended, the caches read back and attended."""
    for dtype in (F16, E4M3):
        lens, hkv, hd = [37, 5, 64], 2, 128
        c = Cache(lens, hkv, hd, 16, dtype, 12, q_dtype=F16)
        g = torch.Generator().manual_seed(1)
        k, v = ((torch.randn(sum(lens), hkv, hd, generator=g)).to(F16).cuda() for _ in range(2))
        first = [n - 1 for n in lens]
        cu = torch.tensor([0] + lens).cumsum(0).tolist()
        old = torch.cat([torch.arange(cu[b], cu[b + 1] - 1) for b in range(3)])
        last = torch.tensor([cu[b + 1] - 1 for b in range(3)])
        i32 = dict(dtype=torch.int32, device="cuda")
        ops.paged_kv_write(c.k, c.v, c.table, torch.tensor(first, **i32),
                           torch.tensor([0] + first, device="cuda").cumsum(0).to(torch.int32), k[old], v[old], **c.scales)
        ops.paged_kv_write(c.k, c.v, c.table, c.len_t, torch.arange(4, **i32), k[last], v[last], **c.scales)
        kr, vr = ops.paged_kv_read(c.k, c.v, c.table, c.len_t, torch.tensor(cu, **i32), sum(lens), dtype=F32, **c.scales)
        c.kv = [[x[cu[b]:cu[b + 1]].double().cpu() for b in range(3)] for x in (kr, vr)]
        if dtype == F16:
            assert torch.equal(kr, k.float()) and torch.equal(vr, v.float())
        q = torch.randn(3, 8, hd, generator=g).to(F16).cuda()
        check_attention(paged(ops, q, c), q, c)


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
@pytest.mark.parametrize("hd", [64, 128])
def test_segments_of_a_cluster_and_of_the_even_split_agree(ops, dtype, q_dtype, hd):
    """The same sequences with a table just wide enough (a cluster for each) and with a very wide one (the even split)."""
    lens = [1, 16, 17, 31, 0, 33, 64, 65, 200, 500]
    c, q = run(lens, (8, 2), hd, 16, dtype, q_dtype, seed=21)
    check_attention(paged(ops, q, c), q, c)
    wide = torch.full((len(lens), 20000), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_attention(ops.paged_attention(q, c.k, c.v, wide, c.len_t, status=status, **c.scales), q, c)
    assert int(status) == 0


def test_the_workspace_that_is_asked_for(ops):
    from autoregressive_decode_persistent_gb300 import adp
    c, q = run([6000, 10], (8, 2), 128, 16, F16, seed=22)
    kv = ops._paged("test", c.k, c.v, c.table, c.len_t, None, None, 0)
    need = adp.adp_paged_attention_workspace(kv, 8)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # its contents do not matter
    check_attention(paged(ops, q, c, workspace=ws), q, c)
    with pytest.raises(adp.AdpError):
        paged(ops, q, c, workspace=ws[:need - 1])
    c, q = run([300, 10], (8, 2), 128, 16, F16, seed=22)
    kv = ops._paged("test", c.k, c.v, c.table, c.len_t, None, None, 0)
    assert adp.adp_paged_attention_workspace(kv, 8) == 0


def test_calls_at_once_on_two_streams(ops):
    """Two caches attended at the same time, each call with a workspace of its own, many times over."""
    pairs = []
    for seed in (31, 32):
        c, q = run([6000, 300, 5], (8, 2), 64, 16, F16, seed=seed)  # (long enough for the even split)
        pairs.append((c, q, paged(ops, q, c), torch.cuda.Stream()))
        check_attention(pairs[-1][2], q, c)
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        for c, q, _, s in pairs:
            with torch.cuda.stream(s):
                got.append((paged(ops, q, c), c))
    torch.cuda.synchronize()
    for out, c in got:
        want = next(w for cc, _, w, _ in pairs if cc is c)
        assert torch.equal(out, want)


def test_no_sequences_and_no_rows(ops):
    c = Cache([5], 2, 64, 16, F16, 1)
    none = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    no_lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 4, 64, dtype=F16, device="cuda")
    assert ops.paged_attention(q, c.k, c.v, none, no_lens).shape == (0, 4, 64)
    rows = torch.zeros(0, 2, 64, dtype=F16, device="cuda")
    ops.paged_kv_write(c.k, c.v, none, no_lens, cu, rows, rows)
    k, v = ops.paged_kv_read(c.k, c.v, none, no_lens, cu, 0)
    assert k.shape == v.shape == (0, 2, 64)


def test_the_result_in_the_queries_place(ops):
    for lens in ([40, 3], [6000, 20]):
        c, q = run(lens, (8, 2), 64, 16, F16, seed=33)
        want = paged(ops, q, c)
        got = q.clone()
        paged(ops, got, c, out=got)
        assert torch.equal(got, want)


WRONG_OFFSETS = [  # offsets of two sequences, rows, and by row: (sequence, rows behind it) or None; rows not named are padding
    ([0, 50, 20], 30, {**{i: (0, 50 - i) for i in range(20)}, **dict.fromkeys(range(20, 30))}),
    ([5, 10, 20], 20, {**dict.fromkeys(range(10)), **{i: (1, 20 - i) for i in range(10, 20)}}),
    ([-5, 10, 20], 20, {**dict.fromkeys(range(10)), **{i: (1, 20 - i) for i in range(10, 20)}}),
    ([0, -5, 20], 20, dict.fromkeys(range(20))),
    ([0, 2 ** 31 - 1, -2 ** 31], 20, dict.fromkeys(range(20))),
    ([20, 10, 0], 20, dict.fromkeys(range(10)))]


@pytest.mark.parametrize("dtype", [F16, E4M3])
@pytest.mark.parametrize("cu,n_rows,where", WRONG_OFFSETS)
def test_row_offsets_that_are_wrong_are_reported(ops, dtype, cu, n_rows, where):
    """Rows that no sequence's offsets hold are not written (read: zeros), whatever the tables hold behind the lengths."""
    lens, page = [60, 40], 8
    c = Cache(lens, 1, 64, page, dtype, 7)
    stale = next(p for p in range(c.k.shape[0]) if p not in c.table.flatten().tolist())
    c.table[c.table < 0] = stale  # entries behind the lengths name a page of somebody else's
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    was = [raw(c.k).clone(), raw(c.v).clone()]
    x = torch.randn(n_rows, 1, 64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.paged_kv_write(c.k, c.v, c.table, c.len_t, offsets, x, x, status=status, **c.scales)
    assert int(status) == -1
    at = {i: (s, lens[s] - n) for i, (s, n) in ((i, w) for i, w in where.items() if w)}
    cells = torch.zeros(c.k.shape[0], page, dtype=torch.bool)
    for s, p in at.values():
        cells[int(c.table[s, p // page]), p % page] = True
    for pool, before in zip((c.k, c.v), was):
        changed = (raw(pool) != before).any(-1)[:, 0].cpu()
        assert torch.equal(changed, cells)
    status.zero_()
    out = tuple(torch.full((n_rows, 1, 64), 7.0, device="cuda") for _ in range(2))
    ops.paged_kv_read(c.k, c.v, c.table, c.len_t, offsets, n_rows, out=out, status=status, **c.scales)
    assert int(status) == -1
    for got, pool, name in ((out[0], c.k, "k_scale"), (out[1], c.v, "v_scale")):
        for i in range(n_rows):
            if i not in where:
                assert (got[i] == 7).all()
            elif i not in at:
                assert (got[i] == 0).all()
            else:
                s, p = at[i]
                cell = int(c.table[s, p // page]), 0, p % page
                want = pool[cell[0]].cpu().float()[0, p % page]
                if dtype == E4M3:
                    want = want * c.scales[name][cell].cpu()
                assert torch.equal(got[i, 0].cpu(), want)


def test_a_descending_pair_among_many_row_offsets(ops):
    """40 sequences (more than one comparison of a warp), two of whose offsets descend: no row lands behind a length."""
    lens, page = [9] * 40, 4
    c = Cache(lens, 1, 64, page, F16, 8, spare=2)
    behind = (torch.arange(c.table.shape[1] * page)[None] >= 9).expand(40, -1)  # positions behind the lengths
    cu = list(range(0, 3 * 41, 3))
    cu[20], cu[21] = cu[21], cu[20]
    x = torch.ones(120, 1, 64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.paged_kv_write(c.k, c.v, c.table, c.len_t, torch.tensor(cu, dtype=torch.int32, device="cuda"), x, x, status=status)
    assert int(status) == -1
    one = (c.k == 1).all(-1)[:, 0].cpu()  # [pages, slots]
    for b in range(40):
        for p in range(c.table.shape[1] * page):
            if behind[b, p]:
                assert not one[int(c.table[b, p // page]), p % page], (b, p)


@pytest.mark.parametrize("heads", [(4, 1), (16, 1)])
@pytest.mark.parametrize("wide", [False, True])
def test_a_dominating_position_leaves_the_others_their_weights(ops, heads, wide):
    """Position 0 outweighs every other one by 2^25.5 and its V is 0: the result is the others' share alone, whose fp16
    weights must not vanish beside it."""
    n, hd, bits = 4096, 64, 25.5
    c = Cache([n], 1, hd, 16, F16, 40)
    g = torch.Generator().manual_seed(41)
    held = [torch.zeros(n, 1, hd), torch.rand(n, 1, hd, generator=g) + 0.5]
    held[0][0, 0, 0] = 1.0
    held[1][0] = 0.0
    for pool, x in zip((c.k, c.v), held):
        x = x.to(F16).cuda()
        for p0 in range(0, n, 16):
            pool[int(c.table[0, p0 // 16])] = x[p0:p0 + 16].transpose(0, 1)
    k, v = (x.to(F16).double() for x in held)
    q = torch.zeros(1, heads[0], hd)
    q[:, :, 0] = bits * math.log(2)
    q = q.to(F16).cuda()
    table = c.table
    if wide:  # (the even split)
        table = torch.full((1, 20000), -1, dtype=torch.int32, device="cuda")
        table[:, :c.table.shape[1]] = c.table
    out = ops.paged_attention(q, c.k, c.v, table, c.len_t, scale=1.0)[0].double().cpu()
    o, a, ds, _ = attend64(q[0].double().cpu(), k, v, 1.0)
    # as in check_attention, but fp16's least half step 2^-25 is one of weights that are held 2^7 times larger
    tol = half_step(F16) * o.abs() + a * (half_step(F16) + 2 * ds[:, None] + 2.0 ** -19 + n * 2.0 ** -24)
    tol = tol + 2.0 ** -32 * v.abs().sum((0, 1))
    assert ((out - o).abs() <= tol).all(), float(((out - o).abs() / tol).max())


@pytest.mark.parametrize("q_dtype", [F16, BF16])
@pytest.mark.parametrize("heads,hd,wide", [((4, 1), 128, False), ((16, 1), 64, True), ((8, 2), 64, False)])
def test_a_large_value_scale_that_hardly_counts_leaves_the_others_theirs(ops, q_dtype, heads, hd, wide):
    """One position's V scale is 2^26 times the others', and its score so low that it weighs next to nothing: the others'
    values keep their bits.  Another one's V is all zeros, at the least scale there is, and weighs the most."""
    n = 200
    c, q = run([n], heads, hd, 16, E4M3, q_dtype, seed=42)
    hkv, group = heads[1], heads[0] // heads[1]
    q = (q.float() + 1.0).to(q_dtype)  # (every query has a good part along the vector of ones)
    at = lambda p: (int(c.table[0, p // 16]), slice(None), p % 16)
    for p, sign, f in ((70, -1.0, 2.0 ** 26), (130, 1.0, None)):
        c.k.view(torch.uint8)[at(p)] = torch.full((hkv, hd), sign, device="cuda").to(E4M3).view(torch.uint8)
        c.scales["k_scale"][at(p)] = (60.0 if sign < 0 else 20.0) / hd ** 0.5
        c.kv[0][0][p] = sign * float(c.scales["k_scale"][at(p)][0])
        if f is None:
            c.v.view(torch.uint8)[at(p)] = 0
            c.scales["v_scale"][at(p)] = 2.0 ** -126
            c.kv[1][0][p] = 0
        else:
            c.scales["v_scale"][at(p)] *= f
            c.kv[1][0][p] *= f
    table = c.table
    if wide:  # (the even split)
        table = torch.full((1, 20000), -1, dtype=torch.int32, device="cuda")
        table[:, :c.table.shape[1]] = c.table
    out = ops.paged_attention(q, c.k, c.v, table, c.len_t, **c.scales)[0].double().cpu()
    qd, k, v = q[0].double().cpu(), c.kv[0][0], c.kv[1][0]
    o, a, ds, _ = attend64(qd, k, v, hd ** -0.5)
    s = torch.einsum("hd,nhd->hn", qd, k.repeat_interleave(group, 1)) * hd ** -0.5
    p = torch.softmax(s, 1)
    assert float(p[:, 70].max()) < 2.0 ** -60 and float(p[:, 130].min()) > 0.1
    # as in check_attention; fp16's least half step is one of the products weight x value scale, held so that the largest of
    # them is 2^7 at least, times codes of at most 448
    largest = (p * c.scales["v_scale"].double().cpu()[c.table[0].long().cpu()].transpose(1, 2).reshape(-1, hkv)[:n].T
               .repeat_interleave(group, 0)).amax(1)
    tol = half_step(q_dtype) * o.abs() + a * (half_step(F16) + 2 * ds[:, None] + 2.0 ** -19 + n * 2.0 ** -24)
    tol = tol + (n * 448 * 2.0 ** -32 * largest)[:, None] + torch.finfo(q_dtype).smallest_normal * half_step(q_dtype)
    assert ((out - o).abs() <= tol).all(), float(((out - o).abs() / tol).max())


@pytest.mark.parametrize("q_dtype", [F16, BF16])
def test_value_scales_at_both_ends_of_fp32(ops, q_dtype):
    """Positions of zeros (the least scale), of tiny and of huge scales in one sequence, in units of their own and
    mixed: the result is the huge ones' sum, or the tiny ones' where there are no others, and always finite."""
    n = 96
    for scales in ([2.0 ** -126] * 96, [2.0 ** -100] * 96, [2.0 ** -126] * 64 + [1.0] * 32, [2.0 ** 100] * 32 + [2.0 ** -100] * 64,
                   [2.0 ** (5 * (i % 40) - 100) for i in range(96)]):
        c, q = run([n], (4, 1), 64, 16, E4M3, q_dtype, seed=43)
        for p, f in enumerate(scales):
            was = float(c.scales["v_scale"][c.table[0, p // 16], 0, p % 16])
            c.scales["v_scale"][c.table[0, p // 16], 0, p % 16] = f
            c.kv[1][0][p] *= f / was
        out = paged(ops, q, c)[0].double().cpu()
        o, a, ds, _ = attend64(q[0].double().cpu(), c.kv[0][0], c.kv[1][0], 64 ** -0.5)
        p = torch.softmax(torch.einsum("hd,nd->hn", q[0].double().cpu(), c.kv[0][0][:, 0]) * 64 ** -0.5, 1)
        largest = (p * torch.tensor(scales, dtype=torch.float64)).amax(1)[:, None]
        tol = half_step(q_dtype) * o.abs() + a * (half_step(F16) + 2 * ds[:, None] + 2.0 ** -19 + n * 2.0 ** -24)
        tol = tol + n * 448 * 2.0 ** -32 * largest + torch.finfo(q_dtype).smallest_normal * half_step(q_dtype) * 2
        big = o.abs() > torch.finfo(q_dtype).max  # (what the result's type cannot hold becomes an infinity)
        assert torch.isinf(out[big]).all()
        assert ((out - o).abs() <= tol)[~big].all(), (scales[0], float(((out - o).abs() / tol)[~big].max()))


def test_ranks_and_empty_heads_are_refused(ops):
    from autoregressive_decode_persistent_gb300 import adp
    c = Cache([5], 2, 64, 16, F16, 1)
    cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    rows = torch.zeros(5, 2, 64, dtype=F16, device="cuda")
    none = torch.zeros(3, 2, 16, 0, dtype=F16, device="cuda")
    q = torch.zeros(1, 2, 0, dtype=F16, device="cuda")
    for call in (lambda: ops.paged_kv_write(c.k, c.v, c.table, c.len_t, cu, rows[0, 0, 0], rows),
                 lambda: ops.paged_kv_write(c.k, c.v, c.table, c.len_t, cu, rows[0], rows[0]),
                 lambda: ops.paged_kv_write(c.k, c.v, c.table, c.len_t, cu, rows, rows[:, :1]),
                 lambda: ops.paged_attention(rows[0], c.k, c.v, c.table, c.len_t),
                 lambda: ops.paged_attention(q, none, none, c.table, c.len_t),
                 lambda: ops.packed_attention(q, q, q, cu, cu),
                 lambda: ops.packed_attention(rows, rows[0], rows, cu, cu)):
        with pytest.raises(adp.AdpError) as e:
            call()
        assert e.value.code == adp.ADP_ERR_INVALID_ARG


@pytest.mark.parametrize("q_dtype", [F16, BF16])
def test_a_quantised_row_with_a_non_finite_value_makes_the_attention_nan(ops, q_dtype):
    c, q = run([40], (4, 2), 64, 16, E4M3, q_dtype, seed=45)
    x = torch.randn(1, 2, 64, device="cuda")
    for which in (0, 1):  # K, V of the last position, head 0
        k, v = x.clone(), x.clone()
        (k, v)[which][0, 0, 9] = math.inf
        ops.paged_kv_write(c.k, c.v, c.table, c.len_t, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), k, v, **c.scales)
        out = paged(ops, q, c)
        assert torch.isnan(out[0, :2]).all() and torch.isfinite(out[0, 2:]).all()


@pytest.mark.parametrize("dtype,q_dtype", TYPES)
def test_a_scale_near_the_largest_float(ops, dtype, q_dtype):
    """Scores of 0 stay 0 under any finite scale: the mean of the values."""
    for scale in (3e38, -3e38):
        c, q = run([33], (4, 2), 64, 16, dtype, q_dtype, seed=44)
        check_attention(paged(ops, q * 0, c, scale=scale), q * 0, c, scale=scale)
