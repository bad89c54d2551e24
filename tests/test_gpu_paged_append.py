"""Rows normed, rotated and appended to a paged cache, against plain 64-bit computations, through ops.paged_kv_append."""
import math

import pytest
import torch

from test_gpu_paged import BF16, E4M3, F16, F32, NAN, Cache, check_attention, half_step, ops, raw  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 1e-5


def angles(n, rot, theta=1e4):
    at = torch.arange(n, dtype=torch.float64)[:, None] * theta ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    return torch.cos(at).float(), torch.sin(at).float()


def turned64(x, gain, cos, sin, eps=EPS):
    """Rows [n, heads, hd] in 64 bits, and the sum of the magnitudes that make each element."""
    x = x.double()
    if gain is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gain.double()
    r = cos.shape[1]
    c, s = cos.double()[:, None], sin.double()[:, None]
    a, b, rest = x[..., :r], x[..., r:2 * r], x[..., 2 * r:]
    return (torch.cat([a * c - b * s, b * c + a * s, rest], -1),
            torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs(), rest.abs()], -1))


def tolerance(y, size, out, hd):
    """Rounded once to `out`; before that in fp32: a sum of hd squares (half of its relative error reaches the root), the root
    and two products, two products and their sum."""
    least = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}[out]
    return half_step(out) * y.abs() * 1.001 + size * (hd / 2 + 16) * 2.0 ** -24 + least


class Setup:
    def __init__(self, new, old, hq, hkv, hd, page, dtype, rows, rot, norm, seed=0, pad=2):
        self.lens = [a + b for a, b in zip(new, old)]
        self.c = Cache(self.lens, hkv, hd, page, dtype, seed + 3)
        g = torch.Generator().manual_seed(seed)
        self.n, self.new, self.old, self.pad = sum(new), new, old, pad
        self.q, self.k, self.v = ((torch.randn(self.n + pad, h, hd, generator=g) * 2).to(rows) for h in (hq, hkv, hkv))
        self.cu = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32).cuda()
        self.cos, self.sin = angles(max(self.lens + [1]), rot)
        self.gains = [(1 + torch.randn(hd, generator=g) / 4).to(rows) if norm else None for _ in range(2)]
        self.pos = torch.tensor([p for a, b in zip(new, old) for p in range(b, a + b)], dtype=torch.long)
        self.at = [(b, p) for b in range(len(new)) for p in range(old[b], self.lens[b])]
        self.page_of = torch.tensor([int(self.c.table[b, p // page]) for b, p in self.at], dtype=torch.long)
        self.slot = self.pos % page

    def call(self, ops, **kw):
        c = self.c
        up = lambda t: None if t is None else t.cuda()
        return ops.paged_kv_append(c.k, c.v, c.table, c.len_t, self.cu, up(self.q), up(self.k), up(self.v), self.cos.cuda(),
                                   self.sin.cuda(), q_gain=up(self.gains[0]), k_gain=up(self.gains[1]), eps=EPS, **c.scales, **kw)

    def check(self, out, out_dtype, was):
        hd, n, c = self.q.shape[2], self.n, self.c
        cos, sin = self.cos[self.pos], self.sin[self.pos]
        y, size = turned64(self.q[:n], self.gains[0], cos, sin)
        assert ((out[:n].double().cpu() - y).abs() <= tolerance(y, size, out_dtype, hd)).all()
        y, size = turned64(self.k[:n], self.gains[1], cos, sin)
        got = c.k.cpu().double()[self.page_of, :, self.slot]
        v = raw(c.v).cpu()[self.page_of, :, self.slot].view(c.dtype)
        if c.dtype == E4M3:
            s = c.scales["k_scale"].cpu().double()[self.page_of, :, self.slot]
            slack = size.amax(-1) * (hd / 2 + 18) * 2.0 ** -24 / 448 + 2.0 ** -149
            assert ((s - (y.abs().amax(-1) / 448).clamp(min=2.0 ** -126)).abs() <= slack).all()
            # half a step of the code: 2^-4 of its value, 2^-10 of the scale at least
            tol = torch.maximum(y.abs() * 2.0 ** -4, s[..., None] * 2.0 ** -10) * 1.001 + size * (hd / 2 + 20) * 2.0 ** -24
            assert ((got * s[..., None] - y).abs() <= tol).all()
            want = (self.v[:n].float().abs().amax(-1) / 448).clamp(min=2.0 ** -126)
            assert torch.equal(c.scales["v_scale"].cpu()[self.page_of, :, self.slot], want)
            assert torch.equal(raw(v), raw((self.v[:n].float() / want[..., None]).to(E4M3)))
        else:
            assert ((got - y).abs() <= tolerance(y, size, c.dtype, hd)).all()
            assert torch.equal(v, self.v[:n].float().to(c.dtype))
        written = torch.zeros(c.k.shape[0], c.page, dtype=torch.bool)
        written[self.page_of, self.slot] = True
        for pool, before in zip((c.k, c.v), was):
            same = (raw(pool) == raw(before)).all(-1).cpu()
            assert same.transpose(1, 2)[~written].all()  # nothing else changed

    def pools(self):
        return [self.c.k.clone(), self.c.v.clone()]


@pytest.mark.parametrize("rows", [F16, BF16, F32])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
@pytest.mark.parametrize("hq,hkv,hd,page,rot,norm,new,old", [
    (20, 4, 128, 16, 128, False, [1, 1, 1, 1], [1000, 0, 15, 16]), (1, 1, 64, 1, 64, True, [5], [0]),
    (4, 2, 64, 8, 32, True, [0, 17, 0, 9], [3, 4, 0, 0]), (7, 3, 128, 64, 16, True, [130], [1]),
    (32, 8, 128, 16, 64, False, [1] * 40, list(range(40))), (5, 1, 64, 16, 48, False, [33, 2], [0, 100])])
def test_appended_rows_match_64_bits(ops, rows, dtype, hq, hkv, hd, page, rot, norm, new, old):
    s = Setup(new, old, hq, hkv, hd, page, dtype, rows, rot, norm, seed=hd)
    was, status = s.pools(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((s.n + s.pad, hq, hd), 7.0, dtype=rows, device="cuda")
    assert s.call(ops, out=out, status=status) is out
    assert int(status) == 0 and (out[s.n:] == 7).all()  # rows behind the last sequence are left as they were
    s.check(out, rows, was)
    was = s.pools()
    again = s.call(ops)
    assert torch.equal(again[:s.n], out[:s.n]) and all(torch.equal(raw(a), raw(b)) for a, b in zip(s.pools(), was))


@pytest.mark.parametrize("rows,to", [(F32, F16), (F32, BF16), (F16, F32), (BF16, F16)])
def test_queries_of_another_type(ops, rows, to):
    s = Setup([9, 30], [2, 0], 6, 2, 64, 16, BF16, rows, 64, True)
    out = torch.zeros(s.n + s.pad, 6, 64, dtype=to, device="cuda")
    was = s.pools()
    s.call(ops, out=out)
    s.check(out, to, was)


@pytest.mark.parametrize("which", [0, 1])
def test_one_norm_of_the_two(ops, which):
    s = Setup([12], [5], 4, 2, 128, 16, F16, F16, 128, True)
    s.gains[which] = None
    was = s.pools()
    s.check(s.call(ops), F16, was)


def test_many_rows_and_rows_in_parts_agree(ops):
    """The same rows in one call, a warp each, and in calls of a few, several warps each."""
    s = Setup([6000], [7], 12, 4, 128, 64, BF16, BF16, 128, True, pad=0)
    was = s.pools()
    out = s.call(ops)
    s.check(out, BF16, was)
    pools = s.pools()
    s.c.k.zero_(), s.c.v.zero_()
    up = lambda t: t.cuda()
    for r0, r1 in ((0, 3), (3, 40), (40, 6000)):
        part = ops.paged_kv_append(s.c.k, s.c.v, s.c.table, torch.tensor([7 + r1], dtype=torch.int32, device="cuda"),
                                   torch.tensor([0, r1 - r0], dtype=torch.int32, device="cuda"), up(s.q[r0:r1]), up(s.k[r0:r1]),
                                   up(s.v[r0:r1]), up(s.cos), up(s.sin), q_gain=up(s.gains[0]), k_gain=up(s.gains[1]), eps=EPS)
        assert torch.equal(part, out[r0:r1])
    for pool, whole in zip((s.c.k, s.c.v), pools):
        assert torch.equal(pool[s.page_of.cuda(), :, s.slot.cuda()], whole[s.page_of.cuda(), :, s.slot.cuda()])


def test_slices_of_a_fused_projection_and_the_result_in_the_queries_place(ops):
    s = Setup([40, 3], [1, 0], 4, 2, 128, 16, BF16, BF16, 128, False, pad=0)
    was = s.pools()
    want = s.call(ops)
    pools = s.pools()
    s.c.k.copy_(was[0]), s.c.v.copy_(was[1])
    qkv = torch.cat([s.q, s.k, s.v], 1).cuda()
    got = ops.paged_kv_append(s.c.k, s.c.v, s.c.table, s.c.len_t, s.cu, qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], s.cos.cuda(), s.sin.cuda(),
                              out=qkv[:, :4])
    assert torch.equal(got, want) and torch.equal(qkv[:, 4:].cpu(), torch.cat([s.k, s.v], 1))
    assert all(torch.equal(raw(a), raw(b)) for a, b in zip(s.pools(), pools))


def test_keys_and_values_only(ops):
    s = Setup([10], [3], 4, 2, 64, 16, F16, F16, 64, True)
    s.call(ops)
    pools = s.pools()
    s.c.k.zero_(), s.c.v.zero_()
    s.q = None
    assert s.call(ops) is None
    at = s.page_of.cuda(), slice(None), s.slot.cuda()  # (16-bit pages)
    assert torch.equal(s.c.k[at], pools[0][at]) and torch.equal(s.c.v[at], pools[1][at])


def test_elements_that_are_not_rotated_take_nothing_from_the_others(ops):
    s = Setup([6], [0], 2, 1, 64, 16, F16, F16, 32, False, pad=0)
    s.q[2, 1, 40], s.q[3, 0, 5] = math.inf, NAN
    out = s.call(ops).cpu()
    bad = torch.zeros(6, 2, 64, dtype=torch.bool)
    bad[2, 1, 40] = bad[3, 0, 5] = bad[3, 0, 21] = True  # (a rotated pair: 5 and 21)
    assert torch.equal(~torch.isfinite(out), bad)


@pytest.mark.parametrize("value", [math.inf, NAN])
def test_a_quantised_key_with_a_non_finite_value_reads_back_as_nan(ops, value):
    s = Setup([4], [0], 2, 2, 64, 16, E4M3, BF16, 64, False, pad=0)
    s.k[2, 1, 30] = value
    s.call(ops)
    kr, vr = ops.paged_kv_read(s.c.k, s.c.v, s.c.table, s.c.len_t, s.cu, 4, dtype=F32, **s.c.scales)
    bad = torch.isnan(kr).cpu()
    assert bad[2, 1].all() and bad.sum() == 64 and torch.isfinite(vr).all()


def test_rows_without_a_page_or_an_angle_are_reported_and_give_zeros(ops):
    s = Setup([20, 5], [0, 0], 2, 1, 64, 8, F16, F16, 64, False, pad=0)
    for bad in (-1, s.c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        good = int(s.c.table[0, 1])
        s.c.table[0, 1] = bad
        out = s.call(ops, status=status)
        s.c.table[0, 1] = good
        assert int(status) == -1
        assert (out[8:16] == 0).all() and (out[:8] != 0).any(-1).all() and (out[16:] != 0).any(-1).all()
    # positions behind the angles
    s = Setup([20, 5], [0, 0], 2, 1, 64, 8, F16, F16, 64, False, pad=0)
    was = s.pools()
    s.cos, s.sin = s.cos[:13], s.sin[:13]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.call(ops, status=status)
    assert int(status) == -3
    assert (out[13:20] == 0).all() and (out[:13] != 0).any(-1).all() and (out[20:] != 0).any(-1).all()
    rows = [int(s.page_of[i]) for i in range(13, 20)], [int(s.slot[i]) for i in range(13, 20)]
    for pool, before in zip((s.c.k, s.c.v), was):
        assert torch.equal(raw(pool)[rows[0], :, rows[1]], raw(before)[rows[0], :, rows[1]])
    # lengths and offsets that are wrong
    for lens, cu in (([3, 5], None), ([1000, 5], None), ([-1, 5], None), ([20, 5], [0, 50, 20]), ([20, 5], [5, 10, 25]), ([20, 5], [0, -5, 25])):
        s = Setup([20, 5], [0, 0], 2, 1, 64, 8, F16, F16, 64, False, pad=0)
        s.c.len_t.copy_(torch.tensor(lens, dtype=torch.int32))
        if cu:
            s.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        status.zero_()
        s.call(ops, status=status)
        assert int(status) == -1


def test_another_stream_and_a_captured_graph_with_changing_positions(ops):
    s = Setup([3, 40], [2, 0], 4, 2, 64, 16, E4M3, F16, 64, True, pad=0)
    want, pools = s.call(ops), s.pools()
    up = [t.cuda() for t in (s.q, s.k, s.v, s.cos, s.sin, *s.gains)]
    call = lambda: ops.paged_kv_append(s.c.k, s.c.v, s.c.table, s.c.len_t, s.cu, *up[:5], q_gain=up[5], k_gain=up[6], eps=EPS, **s.c.scales)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = call()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    s.c.len_t.copy_(torch.tensor([4, 39], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, want)
    s.c.len_t.copy_(torch.tensor([5, 40], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    at = s.page_of.cuda(), slice(None), s.slot.cuda()  # (the positions in front of them were written in between)
    assert all(torch.equal(raw(a)[at], raw(b)[at]) for a, b in zip(s.pools(), pools))


def test_offsets_past_32_bits(ops):
    page, hkv, hd = 64, 8, 128
    n_pages = 5 * 2 ** 30 // (page * hkv * hd * 2) + 3
    pools = [torch.zeros(n_pages, hkv, page, hd, dtype=F16, device="cuda") for _ in range(2)]
    s = Setup([100], [0], 8, hkv, hd, page, F16, F16, hd, False, pad=0)
    s.call(ops)
    table = torch.tensor([[n_pages - 2, n_pages - 1]], dtype=torch.int32, device="cuda")
    up = [t.cuda() for t in (s.q, s.k, s.v, s.cos, s.sin)]
    ops.paged_kv_append(*pools, table, s.c.len_t, s.cu, *up)
    for pool, src in zip(pools, (s.c.k, s.c.v)):
        assert torch.equal(pool[n_pages - 2], src[s.c.table[0, 0]]) and torch.equal(pool[n_pages - 1, :, :36], src[s.c.table[0, 1], :, :36])


def test_no_rows_and_no_sequences(ops):
    c = Cache([5], 2, 64, 16, F16, 1)
    cos, sin = (t.cuda() for t in angles(5, 64))
    none, no_lens = torch.zeros(0, 3, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    rows, q = torch.zeros(0, 2, 64, dtype=F16, device="cuda"), torch.zeros(0, 4, 64, dtype=F16, device="cuda")
    assert ops.paged_kv_append(c.k, c.v, none, no_lens, torch.zeros(1, dtype=torch.int32, device="cuda"), q, rows, rows, cos, sin).shape == q.shape
    assert ops.paged_kv_append(c.k, c.v, c.table, c.len_t, torch.zeros(2, dtype=torch.int32, device="cuda"), q, rows, rows, cos, sin).shape == q.shape


def test_refusals(ops):
    from autoregressive_decode_persistent_gb300 import adp
    s = Setup([5], [0], 4, 2, 64, 16, F16, F16, 64, True, pad=0)
    good = dict(q=s.q.cuda(), k=s.k.cuda(), v=s.v.cuda(), cos=s.cos.cuda(), sin=s.sin.cuda(), q_gain=s.gains[0].cuda(), k_gain=s.gains[1].cuda())
    cos = good["cos"]
    for change in (dict(cos=cos.double()), dict(sin=cos[:4]), dict(cos=s.cos), dict(cos=cos[:, :4], sin=cos[:, :4]), dict(cos=cos.t(), sin=cos.t()),
                   dict(q_gain=good["q_gain"].float()), dict(k_gain=good["k_gain"][:60]), dict(q_gain=s.gains[0]), dict(eps=-1.0), dict(eps=NAN),
                   dict(q=good["q"].float()), dict(q=good["q"][:4]), dict(v=good["v"][:, :1]), dict(k=good["k"].double()),
                   dict(out=torch.zeros(5, 4, 64, dtype=E4M3, device="cuda")), dict(out=torch.zeros(5, 3, 64, dtype=F16, device="cuda")),
                   dict(q=None, out=good["q"]), dict(q=good["q"][:, :0])):
        a = dict(good)
        a.update(change)
        pos = [a.pop(n) for n in ("q", "k", "v", "cos", "sin")]
        with pytest.raises(adp.AdpError):
            ops.paged_kv_append(s.c.k, s.c.v, s.c.table, s.c.len_t, s.cu, *pos, **a)


@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_appended_step_by_step_then_attended(ops, dtype):
    """A run of them together: a prompt appended, then single tokens, each attended with a window."""
    hq, hkv, hd, n, window, sinks = 8, 2, 64, 50, 9, 3
    s = Setup([n], [0], hq, hkv, hd, 16, dtype, F16, 64, True, pad=0)
    s.call(ops)
    kr, vr = ops.paged_kv_read(s.c.k, s.c.v, s.c.table, s.c.len_t, s.cu, n, dtype=F32, **s.c.scales)
    s.c.q_dtype = F16
    s.c.kv = [[kr.double().cpu()], [vr.double().cpu()]]
    s.c.k.zero_(), s.c.v.zero_()
    up = [t.cuda() for t in (s.q, s.k, s.v)]
    rest = [s.cos.cuda(), s.sin.cuda()]
    i32 = dict(dtype=torch.int32, device="cuda")
    at = 0
    for m in (30, 1, 1, 17, 1):
        lens = torch.tensor([at + m], **i32)
        q = ops.paged_kv_append(s.c.k, s.c.v, s.c.table, lens, torch.tensor([0, m], **i32), *[t[at:at + m] for t in up], *rest,
                                q_gain=s.gains[0].cuda(), k_gain=s.gains[1].cuda(), eps=EPS, **s.c.scales)
        at += m
        out = ops.paged_attention(q[-1:], s.c.k, s.c.v, s.c.table, lens, window=window, sinks=sinks, **s.c.scales)
        unseen = {(0, p) for p in range(at) if sinks <= p < at - window}
        check_attention(out, q[-1:], s.c, lens=[at], skip=unseen)
