"""adp_paged_forward: packed prompts, single tokens and both together over paged caches, against the oracle."""
import numpy as np
import pytest
import torch

import synth
from gpu_common import ARGMAX_MARGIN, LOGIT_MAX_ABS, LOGIT_REL_L2, oracle_forced

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    assert torch.cuda.is_available(), "a CUDA GPU is required"
    from autoregressive_decode_persistent_gb300 import adp, build
    build.build()
    return adp


def _shapes():
    tiny = synth.get_config("tiny")
    big = synth.shrink(synth.get_config("dense-8b-bf16"))
    e4m3 = synth.shrink(synth.get_config("dense-2.3b-e4m3"), head_dim=128)
    return {"tiny-f16": tiny, "8b-bf16": big, "2.3b-e4m3-weights-hd128": e4m3}


def _assert_close(cfg, got, ref):
    """Logits against the oracle's plain mode: the stated tolerances for fp16 operands.  The path rounds six operands a
    layer (both normalised inputs, q, the probabilities, the attention's output, h) and the last normalised input to
    16 bits, each by at most u = finfo.eps / 2 of its value, independently of one another; a product with a random
    matrix carries a rounding's share of the norm on as it carries the values.  So the logits' relative L2 error is at
    most sqrt(6 L + 1) u: with 2 layers 1.8e-3 for fp16, within the stated 5e-3, and 1.4e-2 for bf16, where the three
    stated bounds are scaled alike."""
    u = 2.0 ** -8 if cfg["kv_dtype"] == "bf16" else 2.0 ** -11
    f = max(1.0, np.sqrt(6 * cfg["n_layers"] + 1) * u / LOGIT_REL_L2)
    for g, r in zip(got.astype(np.float64), ref.astype(np.float64)):
        assert np.max(np.abs(g - r)) <= LOGIT_MAX_ABS * f, np.max(np.abs(g - r))
        assert np.linalg.norm(g - r) <= LOGIT_REL_L2 * f * np.linalg.norm(r), np.linalg.norm(g - r) / np.linalg.norm(r)
        top = np.sort(r)[-2:]
        if top[1] - top[0] > ARGMAX_MARGIN * f:
            assert np.argmax(g) == np.argmax(r)


def _tables(lens, page):
    """A page table for the requests' longest lengths, with pages in mixed order and some spare ones."""
    need = [-(-n // page) for n in lens]
    order = np.random.default_rng(5).permutation(sum(need) + 4).tolist()
    table = -np.ones((len(lens), max(need)), dtype=np.int32)
    for b, n in enumerate(need):
        table[b, :n] = [order.pop() for _ in range(n)]
    return table, sum(need) + 4


@pytest.mark.parametrize("name", list(_shapes()))
def test_prompts_then_steps_then_both_match_the_oracle(lib, name):
    """Five requests (more than the batched step takes): their prompts in one pass, two steps of single tokens, a pass in
    which one request continues with several tokens, one with a single one and one pauses; every logit row within the
    tolerances of the oracle's plain mode on that request alone."""
    from autoregressive_decode_persistent_gb300.model import DecodeModel, PagedCache
    cfg = _shapes()[name]
    W = synth.model_weights(cfg)
    rng = np.random.default_rng(3)
    lens = [3, 17, 1, 40, 33]
    more = [[4, 1, 1], [1, 1, 5], [1, 1, 9], [1, 1, 0], [1, 1, 1]]
    more[0][0] = 1
    total = [n + sum(m) for n, m in zip(lens, more)]
    seqs = [rng.integers(0, cfg["vocab"], n).tolist() for n in total]
    refs = [oracle_forced(cfg, W, s)[0] for s in seqs]
    model = DecodeModel(cfg, W)
    table, n_pages = _tables(total, 16)
    cache = PagedCache(model, n_pages, 16)
    at = [0] * 5
    passes = [lens] + [[m[i] for m in more] for i in range(3)]
    for new in passes:
        tokens = [s[a:a + n] for s, a, n in zip(seqs, at, new)]
        at = [a + n for a, n in zip(at, new)]
        logits = cache.forward(table, tokens, at).cpu().numpy()
        for b in range(5):
            if new[b]:
                _assert_close(cfg, logits[b:b + 1], refs[b][at[b] - 1:at[b]])
            else:
                assert (logits[b] == 0).all()
    model.close()


def test_a_quantised_cache_holds_the_first_layers_rows(lib):
    """Layer 0's keys and values do not depend on the cache: those of an e4m3 cache are the 16-bit cache's, off by half
    a step of a code (2^-4 of the value, at least half the row's least step 2^-9 of its scale) and fp16's rounding."""
    from autoregressive_decode_persistent_gb300.model import DecodeModel, PagedCache
    from autoregressive_decode_persistent_gb300 import ops
    cfg = synth.get_config("tiny")
    W = synth.model_weights(cfg)
    model = DecodeModel(cfg, W)
    lens = [30, 7]
    tokens = [np.random.default_rng(b).integers(0, cfg["vocab"], n).tolist() for b, n in enumerate(lens)]
    table, n_pages = _tables(lens, 8)
    t = torch.from_numpy(table).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 30, 37], dtype=torch.int32, device="cuda")
    rows = []
    for dtype in (None, torch.float8_e4m3fn):
        cache = PagedCache(model, n_pages, 8, dtype)
        logits = cache.forward(table, tokens, lens)
        assert torch.isfinite(logits).all()
        scales = {} if dtype is None else dict(k_scale=cache.k_scale[0], v_scale=cache.v_scale[0])
        rows.append(ops.paged_kv_read(cache.k[0], cache.v[0], t, n, cu, 37, dtype=torch.float32, **scales))
    for exact, got in zip(*rows):
        top = exact.abs().amax(-1, keepdim=True)
        tol = exact.abs() * (2.0 ** -4 + 2.0 ** -10) + top / 448 * 2.0 ** -10 * 1.01 + top * 2.0 ** -11
        assert ((got - exact).abs() <= tol).all()
        assert (exact != 0).any()
    model.close()


def test_what_it_refuses(lib):
    from autoregressive_decode_persistent_gb300.model import DecodeModel, PagedCache
    cfg = synth.get_config("tiny")
    model = DecodeModel(cfg, synth.model_weights(cfg))
    cache = PagedCache(model, 40, 16)

    def code(table, tokens, lens, c=cache):
        with pytest.raises(lib.AdpError) as e:
            c.forward(np.array(table, dtype=np.int32), tokens, lens)
        return e.value.code

    assert code([[0]], [[cfg["vocab"]]], [1]) == lib.ADP_ERR_INVALID_ARG
    assert code([[0]], [[-1]], [1]) == lib.ADP_ERR_INVALID_ARG
    assert code([[0]], [[1, 2]], [1]) == lib.ADP_ERR_INVALID_ARG       # fewer positions than rows
    assert code([[0]], [[]], [1]) == lib.ADP_ERR_INVALID_ARG           # nothing to do
    assert code([[0]], [[1]], [17]) == lib.ADP_ERR_CONTEXT_OVERFLOW    # behind the table
    assert code([[0] * 30], [[1]], [cfg["max_ctx"] + 1]) == lib.ADP_ERR_CONTEXT_OVERFLOW
    assert code([[40]], [[1]], [1]) == lib.ADP_ERR_INVALID_ARG         # no such page
    cache.forward(np.array([[39]], dtype=np.int32), [[1]], [1])        # and the model still works
    moe = synth.shrink(synth.get_config("moe-32x1408-top4-e4m3"))
    m2 = DecodeModel(moe, synth.model_weights(moe))
    assert code([[0]], [[1]], [1], PagedCache(m2, 4, 16)) == lib.ADP_ERR_UNSUPPORTED_CONFIG
    m2.close()
    model.close()


def test_misaligned_logits_are_refused(lib):
    """(The refusal of the C call itself; its stores are 16 bytes wide.)"""
    from autoregressive_decode_persistent_gb300.model import DecodeModel, PagedCache
    cfg = synth.get_config("tiny")
    model = DecodeModel(cfg, synth.model_weights(cfg))
    cache = PagedCache(model, 4, 16)
    room = torch.zeros(cfg["vocab"] + 4, device="cuda")
    assert room.data_ptr() % 16 == 0
    hkv, hd = cfg["n_kv_heads"], cfg["head_dim"]
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    layers = (lib.PagedKV * cfg["n_layers"])()
    for i in range(cfg["n_layers"]):
        layers[i] = lib.PagedKV(cache.k[i].data_ptr(), cache.v[i].data_ptr(), None, None, table.data_ptr(), None,
                                hkv * 16 * hd, 0, 4, 16, hkv, hd, lib.ADP_F16, 1, 1)
    torch.cuda.synchronize()
    for at in (1, 2, 3):
        with pytest.raises(lib.AdpError) as e:
            lib.adp_paged_forward(model.handle, layers, [1], [0, 1], [1], room[at:])
        assert e.value.code == lib.ADP_ERR_INVALID_ARG
    lib.adp_paged_forward(model.handle, layers, [1], [0, 1], [1], room[4:])
    assert (room[:4] == 0).all() and room[4:].any()
    assert torch.equal(room[4:], cache.forward([[0]], [[1]], [1])[0])
    model.close()


def test_an_allocation_that_failed_is_reported_once(lib):
    """The runtime's error of a failed allocation (2 TB of residual rows) is not taken for one of the next launches."""
    from autoregressive_decode_persistent_gb300.model import DecodeModel, PagedCache
    cfg = synth.get_config("tiny")
    model = DecodeModel(cfg, synth.model_weights(cfg))
    cache = PagedCache(model, 4, 16)
    small = dict(table=[[0], [1]], tokens=[[5, 6, 7], [1]], lens=[3, 1])
    first = cache.forward(**small).clone()
    with pytest.raises(lib.AdpError) as e:
        lib.adp_debug_tc_gemm_time(model.handle, 0, 2 ** 31 - 1, 1)
    assert e.value.code == lib.ADP_ERR_CUDA and "out of memory" in str(e.value)
    assert torch.equal(cache.forward(**small), first)
    model.close()


def test_scratch_that_could_not_grow_leaves_the_model_working(lib):
    """A pass whose gathered contexts would take 550 GB is refused by the allocator; the passes behind it run as before."""
    from autoregressive_decode_persistent_gb300.model import DecodeModel, PagedCache
    cfg = synth.shrink(synth.get_config("dense-2.3b-fp16"), head_dim=128, n_kv_heads=8, n_heads=8, max_ctx=32768)
    model = DecodeModel(cfg, synth.model_weights(cfg))
    cache = PagedCache(model, 4, 1024)
    small = dict(table=[[0], [1]], tokens=[[5, 6, 7], []], lens=[3, 0])
    first = cache.forward(**small).clone()
    n = 8192
    for _ in range(2):
        with pytest.raises(lib.AdpError) as e:
            cache.forward(np.zeros((n, 32), dtype=np.int32), [[1, 2]] + [[3]] * (n - 1), [32768] * n)
        assert e.value.code == lib.ADP_ERR_CUDA and "out of memory" in str(e.value)
        for _ in range(2):
            assert torch.equal(cache.forward(**small), first)
    model.close()


def test_a_wrong_later_layer_is_refused_before_anything_is_written(lib):
    from autoregressive_decode_persistent_gb300.model import DecodeModel, PagedCache
    cfg = synth.get_config("tiny")
    model = DecodeModel(cfg, synth.model_weights(cfg))
    cache = PagedCache(model, 4, 16)
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    logits = torch.empty((2, cfg["vocab"]), device="cuda")
    hkv, hd = cfg["n_kv_heads"], cfg["head_dim"]

    def layers(**last):
        out = (lib.PagedKV * cfg["n_layers"])()
        for i in range(cfg["n_layers"]):
            f = dict(k=cache.k[i].data_ptr(), v=cache.v[i].data_ptr(), table=table.data_ptr(), lens=None,
                     page_stride=hkv * 16 * hd, scale_stride=0, n_pages=4, page_size=16, n_kv_heads=hkv, head_dim=hd,
                     dtype=lib.DTYPES[cfg["kv_dtype"]], n_seqs=2, table_width=1)
            f.update(last if i + 1 == cfg["n_layers"] else {})
            for k, x in f.items():
                setattr(out[i], k, x)
        return out

    torch.cuda.synchronize()
    for tokens, cu in (([1, 2, 3], [0, 2, 3]), ([1, 2], [0, 1, 2])):  # prompts, single tokens
        lens = [cu[1], cu[2] - cu[1]]
        for wrong, code in ((dict(k=None), -1), (dict(v=cache.v[-1].data_ptr() + 8), -1), (dict(table=None), -1),
                            (dict(page_stride=hkv * 16 * hd - 8), -1), (dict(n_pages=0), -1), (dict(page_size=24), -2),
                            (dict(dtype=lib.ADP_E4M3), -1), (dict(n_seqs=1), -1)):
            with pytest.raises(lib.AdpError) as e:
                lib.adp_paged_forward(model.handle, layers(**wrong), tokens, cu, lens, logits)
            assert e.value.code == code, wrong
            torch.cuda.synchronize()
            assert not cache.k.any() and not cache.v.any()
        lib.adp_paged_forward(model.handle, layers(), tokens, cu, lens, logits)
        assert cache.k.any() and torch.isfinite(logits).all()
        cache.k.zero_(), cache.v.zero_()
        torch.cuda.synchronize()
    model.close()


def test_an_nvfp4_model_matches_the_oracle(lib):
    from autoregressive_decode_persistent_gb300.model import DecodeModel, PagedCache
    cfg = synth.shrink(synth.get_config("dense-2.3b-nvfp4"))
    W = synth.model_weights(cfg)
    rng = np.random.default_rng(8)
    seqs = [rng.integers(0, cfg["vocab"], n).tolist() for n in (21, 6)]
    refs = [oracle_forced(cfg, W, s)[0] for s in seqs]
    model = DecodeModel(cfg, W)
    table, n_pages = _tables([21, 6], 16)
    cache = PagedCache(model, n_pages, 16)
    for at in ([20, 5], [21, 6]):  # prompts, then one token each
        tokens = [s[at[b] - 1:at[b]] if at == [21, 6] else s[:at[b]] for b, s in enumerate(seqs)]
        logits = cache.forward(table, tokens, at).cpu().numpy()
        for b in range(2):
            _assert_close(cfg, logits[b:b + 1], refs[b][at[b] - 1:at[b]])
    model.close()


@pytest.mark.parametrize("name", ["tiny-f16", "8b-bf16"])
def test_one_token_steps_over_a_quantised_cache(lib, name):
    """Steps of single tokens over e4m3 pages (codes attended as they are) and the same steps beside a request without a new
    row (every context read back to 16 bits, then attended as prompts) are two ways to one result: each is within the
    stated tolerances of the other.  They differ by the 16-bit roundings that _assert_close counts, and by codes of the new
    rows that these turn to a neighbour: a rounding u of the value crosses a border of codes (steps of 2^-3 of the value)
    for a share of 2^4 u of the elements at most and then changes one by 2^-3; of one row among the contexts' 30 and more."""
    from autoregressive_decode_persistent_gb300.model import DecodeModel, PagedCache
    cfg = _shapes()[name]
    model = DecodeModel(cfg, synth.model_weights(cfg))
    rng = np.random.default_rng(9)
    lens = [40, 31, 65]
    seqs = [rng.integers(0, cfg["vocab"], n + 3).tolist() for n in lens]
    table, n_pages = _tables([n + 3 for n in lens], 16)
    idle = np.concatenate([table, np.full((1, table.shape[1]), -1, dtype=np.int32)])
    caches = [PagedCache(model, n_pages, 16, torch.float8_e4m3fn) for _ in range(2)]
    for c in caches:
        c.forward(table, [s[:n] for s, n in zip(seqs, lens)], lens)
    for step in range(3):
        tokens = [[s[n + step]] for s, n in zip(seqs, lens)]
        at = [n + step + 1 for n in lens]
        alone = caches[0].forward(table, tokens, at).cpu().numpy()
        beside = caches[1].forward(idle, tokens + [[]], at + [0]).cpu().numpy()
        assert (beside[3] == 0).all()
        _assert_close(cfg, alone, beside[:3])
        assert np.abs(alone).max() > 0.1
    model.close()


def test_a_request_without_a_new_row_is_not_read(lib):
    """Its context may be anywhere (here: no page at all, so that reading it would be reported), and the others' logits are
    what they are without it."""
    from autoregressive_decode_persistent_gb300.model import DecodeModel, PagedCache
    cfg = synth.get_config("tiny")
    model = DecodeModel(cfg, synth.model_weights(cfg))
    cache = PagedCache(model, 8, 16)
    table = [[0, 1], [-1, -1], [2, 3]]
    for tokens, lens in (([[1, 2, 3], [], [4]], [3, 30, 1]), ([[5], [], [6, 7]], [4, 32, 3])):
        beside = cache.forward(table, tokens, lens).clone()
        others = [[tokens[0], tokens[2]], [lens[0], lens[2]]]
        assert torch.equal(beside[[0, 2]], cache.forward([table[0], table[2]], *others))
        assert (beside[1] == 0).all() and beside[0].any()
    model.close()
