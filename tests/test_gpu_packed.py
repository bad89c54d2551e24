"""Packed prompt attention against plain 64-bit computations, through the tensor wrapper of ops.py."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
NAN = float("nan")


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "a CUDA GPU is required"
    from autoregressive_decode_persistent_gb300 import build, ops
    build.build()
    return ops


def half_step(t):
    return torch.finfo(t).eps / 2


def cumulative(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def inputs(lq, lk, heads, hd, dtype, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(sum(lq) + pad, heads[0], hd, generator=g) * 1.5).to(dtype)
    k, v = (torch.randn(sum(lk) + pad, heads[1], hd, generator=g).to(dtype) for _ in range(2))
    return q.cuda(), k.cuda(), v.cuda()


def check(out, q, k, v, lq, lk, scale=None, rows=None):
    """Every query row (or the given ones) within the tolerance; they are computed in 64 bits on the GPU."""
    hq, hd = q.shape[1:]
    g = hq // k.shape[1]
    dtype, scale = q.dtype, hd ** -0.5 if scale is None else scale
    q0 = k0 = 0
    for b in range(len(lq)):
        for h in range(hq):
            qb = q[q0:q0 + lq[b], h].double()
            kb, vb = k[k0:k0 + lk[b], h // g].double(), v[k0:k0 + lk[b], h // g].double()
            seen = torch.arange(lk[b], device="cuda")[None] <= torch.arange(lq[b], device="cuda")[:, None] + lk[b] - lq[b]
            got = out[q0:q0 + lq[b], h].double()
            some = seen.any(1)
            assert (got[~some] == 0).all()
            if not some.any():
                continue
            s = (qb @ kb.T * scale).masked_fill(~seen, -math.inf)
            p = torch.softmax(s, 1)
            p[~some] = 0
            o, a = p @ vb, p @ vb.abs()
            # out rounded once, every probability rounded once (relative to a maximum that may be stale by 2^8, which
            # fp16 has room for below: 2^-25 of a weight of 1 is half its least step), off by its score's fp32 error
            # in numerator and sum, by exp2's, and by the fp32 sums over the keys
            ds = (qb.abs() @ kb.abs().T * (hd + 8) * 2.0 ** -24 * abs(scale)).masked_fill(~seen, 0).amax(1)
            tol = half_step(dtype) * o.abs() + a * (half_step(dtype) + 2 * ds[:, None] + 2.0 ** -19 + lk[b] * 2.0 ** -24)
            tol = tol + lk[b] * 2.0 ** -25 * vb.abs().amax() * (dtype == F16) + 1e-30
            err = (got - o).abs()[some]
            assert torch.isfinite(got).all()
            assert (err <= tol[some]).all(), (b, h, float((err / tol[some]).max()))
        q0, k0 = q0 + lq[b], k0 + lk[b]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("heads,lq,lk", [
    ((4, 2), [16], [16]), ((1, 1), [1], [1]), ((2, 1), [1, 0, 2, 127, 128, 129], [1, 0, 2, 127, 128, 129]),
    ((20, 4), [50, 300, 7], [50, 300, 7]), ((8, 8), [257], [257]), ((32, 8), [64, 65, 33], [200, 65, 400]),
    ((14, 2), [40, 9], [9, 40]), ((6, 2), [130, 5], [0, 700]), ((128, 1), [5], [130]), ((12, 1), [1, 1, 1], [300, 1, 128])])
def test_matches_64_bits(ops, dtype, hd, heads, lq, lk):
    q, k, v = inputs(lq, lk, heads, hd, dtype, seed=hd + len(lq))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.packed_attention(q, k, v, cumulative(lq), cumulative(lk), status=status)
    check(out, q, k, v, lq, lk)
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_long_prompts_and_many_short_ones(ops, dtype):
    rng = random.Random(3)
    for lq, lk in (([2500], [2500]), ([700], [5000]), ([rng.randint(0, 90) for _ in range(75)],) * 2):
        q, k, v = inputs(lq, lk, (8, 2), 128, dtype, seed=9)
        out = ops.packed_attention(q, k, v, cumulative(lq), cumulative(lk))
        check(out, q, k, v, lq, lk)
        assert torch.equal(out, ops.packed_attention(q, k, v, cumulative(lq), cumulative(lk)))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hd", [64, 128])
def test_more_work_than_the_gpu_holds_at_once(ops, dtype, hd):
    """Several pieces of work in a row on every SM, in both orders (up to 32 sequences and more), with sequences and
    tiles that see nothing among them."""
    rng = random.Random(4)
    for lq, lk in (([1000, 0, 33, 700, 500], [1000, 40, 600, 300, 500]),
                   ([rng.randint(0, 90) for _ in range(75)], [rng.randint(0, 200) for _ in range(75)])):
        q, k, v = inputs(lq, lk, (64, 4), hd, dtype, seed=10)
        out = ops.packed_attention(q, k, v, cumulative(lq), cumulative(lk))
        check(out, q, k, v, lq, lk)
        assert torch.equal(out, ops.packed_attention(q, k, v, cumulative(lq), cumulative(lk)))


def test_scales_negative_zero_and_large_and_growing_scores(ops):
    lq = lk = [300]
    q, k, v = inputs(lq, lk, (4, 2), 64, BF16, seed=1)
    for scale in (0.0, -0.3, 2.0):
        check(ops.packed_attention(q, k, v, cumulative(lq), cumulative(lk), scale=scale), q, k, v, lq, lk, scale=scale)
    k = k * torch.linspace(0.1, 40, 300, device="cuda").to(BF16)[:, None, None]  # later keys' scores grow: O is rescaled
    check(ops.packed_attention(q, k, v, cumulative(lq), cumulative(lk)), q, k, v, lq, lk)


def test_padding_rows_and_strides(ops):
    lq, lk, pad = [40, 33], [40, 90], 9
    q, k, v = inputs(lq, lk, (8, 2), 128, F16, seed=2, pad=pad)
    q[73:], k[130:], v[130:] = NAN, NAN, NAN
    qkv = torch.full((q.shape[0], 24, 128), NAN, dtype=F16, device="cuda")
    qkv[:, 3:11] = q
    kv = torch.full((k.shape[0], 7, 128), NAN, dtype=F16, device="cuda")
    kv[:, :2], kv[:, 4:6] = k, v
    out = torch.full((q.shape[0], 10, 128), 3.0, dtype=F16, device="cuda")
    ops.packed_attention(qkv[:, 3:11], kv[:, :2], kv[:, 4:6], cumulative(lq), cumulative(lk), out=out[:, 1:9])
    check(out[:73, 1:9], q[:73], k[:130], v[:130], lq, lk)
    assert (out[73:] == 3).all() and (out[:, 0] == 3).all() and (out[:, 9] == 3).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("value", [NAN, math.inf, -math.inf])
def test_what_a_query_does_not_see_does_not_reach_it(ops, dtype, value):
    """Non-finite keys and values: the rows in front of them, and other sequences, are as if they were zeros; the rows
    that see them are not finite (in the channel of v, or everywhere for k)."""
    lq, lk = [200, 100, 60], [200, 130, 60]
    for at in (0, 5, 130, 199):  # in the first sequence
        q, k, v = inputs(lq, lk, (4, 2), 64, dtype, seed=4)
        kb, vb = k.clone(), v.clone()
        vb[at, 1, 7] = value
        out = ops.packed_attention(q, k, vb, cumulative(lq), cumulative(lk))
        blind = torch.ones(360, 4, 64, dtype=torch.bool, device="cuda")
        blind[at:200, 2:, 7] = False
        clean = ops.packed_attention(q, k, v, cumulative(lq), cumulative(lk))
        assert torch.equal(out[blind], clean[blind])
        assert not torch.isfinite(out[~blind]).any()
        if not math.isnan(value):
            assert (out[~blind] == value).all()
        kb[at, 1, 7] = NAN
        out = ops.packed_attention(q, kb, v, cumulative(lq), cumulative(lk))
        blind[at:200, 2:] = False
        assert torch.equal(out[blind], clean[blind])
        assert torch.isnan(out[~blind]).all()


def test_no_keys_at_all_and_offsets_that_are_wrong(ops):
    q, k, v = inputs([20], [0], (4, 2), 64, F16)
    out = ops.packed_attention(q, k, v, cumulative([20]), cumulative([0]))
    assert (out == 0).all()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = inputs([20], [20], (4, 2), 64, F16)
    for cu in ([0, 50, 20], [-5, 10, 20], [0, 2 ** 31 - 1, -2 ** 31], [20, 10, 0]):
        status.zero_()
        bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
        ops.packed_attention(q, k, v, bad, torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda"), status=status)
        assert int(status) == -1
        status.zero_()
        ops.packed_attention(q, k, v, torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda"), bad, status=status)
        assert int(status) == -1


def test_offsets_past_32_bits(ops):
    """Keys more than 4 GB into their tensor."""
    n = 5 * 2 ** 30 // (8 * 128 * 2)
    k = torch.zeros(n, 8, 128, dtype=F16, device="cuda")
    v = torch.zeros(n, 8, 128, dtype=F16, device="cuda")
    q, ks, vs = inputs([70], [70], (8, 8), 128, F16, seed=5)
    k[n - 70:], v[n - 70:] = ks, vs
    cu_k = torch.tensor([0, n - 70, n], dtype=torch.int32, device="cuda")
    cu_q = torch.tensor([0, 0, 70], dtype=torch.int32, device="cuda")
    check(ops.packed_attention(q, k, v, cu_q, cu_k), q, ks, vs, [70], [70])


def test_another_stream_and_a_captured_graph_with_changing_offsets(ops):
    lq, lk = [130, 70], [130, 90]
    q, k, v = inputs(lq, lk, (8, 2), 128, BF16, seed=6)
    cu_q, cu_k = cumulative(lq), cumulative(lk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = ops.packed_attention(q, k, v, cu_q, cu_k)
    torch.cuda.current_stream().wait_stream(s)
    check(out, q, k, v, lq, lk)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ops.packed_attention(q, k, v, cu_q, cu_k)
    for lq, lk in (([130, 70], [130, 90]), ([1, 199], [20, 200]), ([200, 0], [220, 0])):
        cu_q.copy_(cumulative(lq))
        cu_k.copy_(cumulative(lk))
        g.replay()
        torch.cuda.synchronize()
        check(out, q, k, v, lq, lk)


def test_prompts_attend_through_a_quantised_cache(ops):
    """A run of the operators together: a prompt's first part is attended and cached, its second part attends to the
    rows read back from the e4m3 pages."""
    hq, hkv, hd, n, cut = 8, 2, 128, 150, 90
    q, k, v = inputs([n], [n], (hq, hkv), hd, BF16, seed=7)
    i32 = dict(dtype=torch.int32, device="cuda")
    pages = [torch.zeros(12, hkv, 16, hd, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    scales = dict(k_scale=torch.zeros(12, hkv, 16, device="cuda"), v_scale=torch.zeros(12, hkv, 16, device="cuda"))
    table = torch.arange(11, 1, -1, **i32)[None].contiguous()
    ops.paged_kv_write(*pages, table, torch.tensor([cut], **i32), torch.tensor([0, cut], **i32), k[:cut], v[:cut], **scales)
    ops.paged_kv_write(*pages, table, torch.tensor([n], **i32), torch.tensor([0, n - cut], **i32), k[cut:], v[cut:], **scales)
    kr, vr = ops.paged_kv_read(*pages, table, torch.tensor([n], **i32), torch.tensor([0, n], **i32), n, dtype=BF16, **scales)
    # e4m3: half a step is 2^-4 of the value, at least half its least step of the row's scale; bf16 rounds once more
    for got, x in ((kr, k), (vr, v)):
        x = x.double()
        assert ((got.double() - x).abs() <= x.abs() * (2.0 ** -4 + 2.0 ** -8) * 1.01 + x.abs().amax(-1, keepdim=True) / 448 * 2.0 ** -9).all()
    out = ops.packed_attention(q[cut:], kr, vr, torch.tensor([0, n - cut], **i32), torch.tensor([0, n], **i32))
    check(out, q[cut:], kr, vr, [n - cut], [n])


def test_many_sequences(ops):
    """500 short sequences: more than are sorted by cost, and a grid that is mostly an upper bound."""
    rng = random.Random(8)
    lq = [rng.randint(0, 6) for _ in range(500)]
    lk = [n + rng.randint(0, 3) for n in lq]
    q, k, v = inputs(lq, lk, (4, 2), 64, F16, seed=12)
    out = torch.full_like(q, NAN)
    ops.packed_attention(q, k, v, cumulative(lq), cumulative(lk), out=out)
    check(out, q, k, v, lq, lk)


def test_calls_at_once_and_the_result_in_the_queries_place(ops):
    lq = [700, 90]
    q, k, v = inputs(lq, lq, (16, 4), 128, BF16, seed=13)
    cu = cumulative(lq)
    want = ops.packed_attention(q, k, v, cu, cu)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(ops.packed_attention(q, k, v, cu, cu))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)
    over = q.clone()
    ops.packed_attention(over, k, v, cu, cu, out=over)
    assert torch.equal(over, want)


@pytest.mark.parametrize("hd", [64, 128])
def test_a_dominating_key_leaves_the_others_their_weights(ops, hd):
    """Key 0 outweighs every other one by 2^25.5 and its V is 0: the result is the others' share alone, whose fp16 weights
    must not vanish beside it."""
    lq, lk, bits = [300], [4096], 25.5
    q, k, v = inputs(lq, lk, (4, 1), hd, F16, seed=20)
    q, k, v = torch.zeros_like(q), torch.zeros_like(k), v.abs() + 0.5
    q[:, :, 0] = bits * math.log(2)
    k[0, 0, 0] = 1.0
    v[0] = 0.0
    out = ops.packed_attention(q, k, v, cumulative(lq), cumulative(lk), scale=1.0).double()
    s = torch.einsum("ihd,jd->hij", q.double(), k[:, 0].double())
    seen = torch.arange(lk[0], device="cuda")[None] <= torch.arange(lq[0], device="cuda")[:, None] + lk[0] - lq[0]
    p = torch.softmax(s.masked_fill(~seen, -math.inf), 2)
    o = torch.einsum("hij,jd->ihd", p, v[:, 0].double())
    # as in check (V is positive), but fp16's least half step 2^-25 is one of weights that are held 2^7 times larger
    ds = bits * math.log(2) * (hd + 8) * 2.0 ** -24
    tol = o * (2 * half_step(F16) + 2 * ds + 2.0 ** -19 + lk[0] * 2.0 ** -24) + 2.0 ** -32 * v[:, 0].double().sum(0)
    assert ((out - o).abs() <= tol).all(), float(((out - o).abs() / tol).max())


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_scale_near_the_largest_float(ops, dtype):
    """Scores of 0 stay 0 under any finite scale: the mean of the values."""
    q, k, v = inputs([70], [70], (4, 2), 64, dtype, seed=21)
    for scale in (3e38, -3e38):
        check(ops.packed_attention(q * 0, k, v, cumulative([70]), cumulative([70]), scale=scale), q * 0, k, v, [70], [70], scale=scale)
