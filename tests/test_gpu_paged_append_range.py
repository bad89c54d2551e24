"""Norms of heads whose squares leave fp32's range, against 64 bits, through ops.paged_kv_append."""
import pytest
import torch

import test_gpu_paged_append as base
from test_gpu_paged_append import BF16, E4M3, F16, F32, Setup, ops  # noqa: F401

pytestmark = pytest.mark.gpu

# what a row's heads are scaled by: squares that vanish, that are subnormal, on both sides of the bound under which heads are scaled,
# ordinary ones, and those that overflow one by one or only as a sum
SIZES = [1e-39, 1e-36, 1e-30, 1e-23, 1e-21, 1e-19, 1e-14, 1e-13, 1e-10, 1.0, 1e10, 3e17, 4e18, 1e25, 7e37]


@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-30])
@pytest.mark.parametrize("rows", [BF16, F32])
@pytest.mark.parametrize("dtype,hd", [(BF16, 128), (F16, 64), (E4M3, 128), (E4M3, 64)])
def test_norms_of_tiny_and_huge_heads(ops, monkeypatch, dtype, hd, rows, eps):  # noqa: F811
    eps = float(torch.tensor(eps, dtype=F32))
    sizes = torch.tensor(SIZES + [1e-44] * (rows == F32), dtype=torch.float64)
    n = 2 * len(sizes)
    s = Setup([n], [3], 5, 3, hd, 16, dtype, rows, hd // 2, True, seed=5, pad=0)
    g = torch.Generator().manual_seed(6)
    for name in ("q", "k"):  # (heads of every size side by side)
        x = getattr(s, name)
        at = (torch.arange(n)[:, None] + torch.arange(x.shape[1])[None]) % len(sizes)
        y = torch.randn(x.shape, generator=g, dtype=torch.float64).clamp(-4, 4) * sizes[at][..., None]
        setattr(s, name, y.to(rows))
        assert torch.isfinite(getattr(s, name)).all()
    monkeypatch.setattr(base, "EPS", eps)
    monkeypatch.setattr(base.turned64, "__defaults__", (eps,))
    was = s.pools()
    s.check(s.call(ops), rows, was)


def test_heads_of_zeros_and_of_non_finite_elements(ops, monkeypatch):  # noqa: F811
    """Zeros stay zeros beside an eps however small, and have no norm without one; an infinity's norm leaves zeros beside it."""
    s = Setup([3], [0], 2, 1, 64, 16, BF16, F32, 64, True, pad=0)
    s.cos, s.sin = torch.ones_like(s.cos), torch.zeros_like(s.sin)
    s.q[0] = 0
    s.q[1, 0, 5], s.q[2, 1, 9] = float("inf"), float("nan")
    for eps in (1e-44, 1e-5, 0.0):
        monkeypatch.setattr(base, "EPS", eps)
        out = s.call(ops).cpu()
        assert torch.isnan(out[0]).all() if eps == 0 else (out[0] == 0).all()
        assert torch.isnan(out[1, 0, 5]) and out[1, 0].isnan().sum() == 2 and (out[1, 0].nan_to_num(0) == 0).all()  # (the pair 5, 37)
        assert torch.isnan(out[2, 1]).all() and torch.isfinite(out[1, 1]).all() and torch.isfinite(out[2, 0]).all()
