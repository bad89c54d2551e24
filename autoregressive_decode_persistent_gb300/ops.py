"""The paged KV cache operators and packed prompt attention on PyTorch tensors (include/adp.h has their semantics).

Argument checks and marshalling only: every computation runs in libadp.so's kernels, on the current
stream of the tensors' device, without synchronising.  Nothing is differentiable.  Wrong arguments raise
adp.AdpError before anything is launched; wrong lengths or page numbers, which only the GPU sees, set the
optional `status` tensor (int32, one element).
"""
from __future__ import annotations

import torch

from . import adp

_CACHE = {torch.float16: adp.ADP_F16, torch.bfloat16: adp.ADP_BF16, torch.float8_e4m3fn: adp.ADP_E4M3}
_ROWS = {torch.float16: adp.ADP_F16, torch.bfloat16: adp.ADP_BF16, torch.float32: adp.ADP_F32}
_HALF = {torch.float16: adp.ADP_F16, torch.bfloat16: adp.ADP_BF16}


def _refuse(where: str, what: str):
    raise adp.AdpError(adp.ADP_ERR_INVALID_ARG, f"{where}: {what}")


def _indices(where: str, name: str, t: torch.Tensor, dims: int, device):
    if t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous() or t.device != device:
        _refuse(where, f"{name} must be a contiguous int32 tensor of {dims} dimension(s) on {device}")


def _rows(where: str, name: str, t: torch.Tensor, heads: int | None, hd: int, device):
    """A [n, heads, head_dim] tensor whose rows may lie apart."""
    if (t.dim() != 3 or t.shape[2] != hd or (heads is not None and t.shape[1] != heads) or t.device != device
            or (t.numel() and (t.stride(2) != 1 or (t.stride(1) != hd and t.shape[1] > 1)))):
        _refuse(where, f"{name} must be [rows, heads, head_dim] on {device} with contiguous heads")


def _row_stride(t: torch.Tensor) -> int:
    """Elements from one row to the next (of a single row the stride says nothing)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _status(where: str, t: torch.Tensor | None, device):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.numel() != 1 or t.device != device:
        _refuse(where, f"status must be one int32 on {device}")
    return t.data_ptr()


def _stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _call(device, fn, *args):
    """fn(*args, stream) with the tensors' device current."""
    if device.index == torch.cuda.current_device():
        fn(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            fn(*args, _stream(device))


def _paged(where: str, k_pages, v_pages, table, lens, k_scale, v_scale) -> adp.PagedKV:
    shape, stride, device = k_pages.shape, k_pages.stride(), k_pages.device
    if device.type != "cuda":
        _refuse(where, "the tensors must be on a CUDA device")
    dtype = _CACHE.get(k_pages.dtype)
    if dtype is None or len(shape) != 4 or v_pages.dtype != k_pages.dtype or v_pages.shape != shape \
            or v_pages.stride() != stride or v_pages.device != device:
        _refuse(where, "k_pages and v_pages must be alike: [pages, kv_heads, page_size, head_dim], f16, bf16 or e4m3")
    n_pages, heads, ps, hd = shape
    if (stride[3] != 1 or (stride[2] != hd and ps > 1) or (stride[1] != ps * hd and heads > 1)) and k_pages.numel():
        _refuse(where, "a page must be contiguous")
    _indices(where, "table", table, 2, device)
    _indices(where, "lens", lens, 1, device)
    n_seqs, width = table.shape
    if lens.shape[0] != n_seqs:
        _refuse(where, "table and lens must name the same sequences")
    ks = vs = None
    ss = 0
    if dtype == adp.ADP_E4M3:
        if k_scale is None or v_scale is None or k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 \
                or k_scale.shape != shape[:3] or v_scale.shape != shape[:3] or k_scale.device != device \
                or v_scale.device != device or k_scale.stride() != v_scale.stride() \
                or (k_scale.stride(2) != 1 and ps > 1) or (k_scale.stride(1) != ps and heads > 1):
            _refuse(where, "e4m3 pages need k_scale and v_scale alike: fp32 [pages, kv_heads, page_size]")
        ks, vs, ss = k_scale.data_ptr(), v_scale.data_ptr(), k_scale.stride(0)
    # (the stride of a single page says nothing)
    return adp.PagedKV(k_pages.data_ptr(), v_pages.data_ptr(), ks, vs, table.data_ptr(), lens.data_ptr(),
                       stride[0] if n_pages > 1 else heads * ps * hd, ss if n_pages > 1 else heads * ps,
                       n_pages, ps, heads, hd, dtype, n_seqs, width)


def paged_kv_write(k_pages, v_pages, table, lens, cu_rows, k, v, *, k_scale=None, v_scale=None, status=None):
    """Write packed rows k, v [rows, kv_heads, head_dim] (f16, bf16 or f32) into their sequences' last positions.

    k_pages, v_pages: [pages, kv_heads, page_size, head_dim] f16, bf16 or float8_e4m3fn (then with fp32
    k_scale, v_scale [pages, kv_heads, page_size]), changed in place.  table: int32 [seqs, width] page numbers;
    lens: int32 [seqs], the rows being written included; cu_rows: int32 [seqs + 1]."""
    where = "paged_kv_write"
    kv = _paged(where, k_pages, v_pages, table, lens, k_scale, v_scale)
    _transfer(where, adp.adp_paged_kv_write, kv, k_pages.device, cu_rows, k, v, status)


def paged_kv_read(k_pages, v_pages, table, lens, cu_rows, n_rows: int, *, dtype=None, k_scale=None, v_scale=None,
                  out=None, status=None):
    """Read every sequence's last cu_rows[s + 1] - cu_rows[s] positions back into packed rows.

    Returns (k, v) [n_rows, kv_heads, head_dim] of `dtype` (default: the pages' type, fp16 for e4m3 pages), or
    writes into out = (k, v); rows from cu_rows[-1] on are left as they were."""
    where = "paged_kv_read"
    kv = _paged(where, k_pages, v_pages, table, lens, k_scale, v_scale)
    if out is None:
        if dtype is None:
            dtype = torch.float16 if kv.dtype == adp.ADP_E4M3 else k_pages.dtype
        shape = (n_rows, kv.n_kv_heads, kv.head_dim)
        out = (torch.empty(shape, dtype=dtype, device=k_pages.device), torch.empty(shape, dtype=dtype, device=k_pages.device))
    k, v = out
    if k.shape[0] != n_rows or (dtype is not None and k.dtype != dtype):
        _refuse(where, "out must hold n_rows rows of dtype")
    _transfer(where, adp.adp_paged_kv_read, kv, k_pages.device, cu_rows, k, v, status)
    return k, v


def _transfer(where, call, kv, device, cu_rows, k, v, status):
    _indices(where, "cu_rows", cu_rows, 1, device)
    if cu_rows.shape[0] != kv.n_seqs + 1:
        _refuse(where, "cu_rows must have one entry more than there are sequences")
    _rows(where, "k", k, kv.n_kv_heads, kv.head_dim, device)
    _rows(where, "v", v, kv.n_kv_heads, kv.head_dim, device)
    dt = _ROWS.get(k.dtype)
    if dt is None or v.dtype != k.dtype or v.shape != k.shape:
        _refuse(where, "k and v rows must be alike, of f16, bf16 or f32")
    _call(device, call, kv, k.data_ptr(), v.data_ptr(), dt, _row_stride(k), _row_stride(v), cu_rows.data_ptr(), k.shape[0],
          _status(where, status, device))


def paged_attention(q, k_pages, v_pages, table, lens, *, scale: float | None = None, k_scale=None, v_scale=None,
                    out=None, workspace=None, status=None):
    """Attention of one new token per sequence, q [seqs, heads, head_dim] f16 or bf16, over its cached positions.

    scale: default 1 / sqrt(head_dim).  workspace: optional uint8 tensor of adp.adp_paged_attention_workspace
    bytes (not shared by calls that may run at the same time); by default one is allocated on the current stream."""
    where = "paged_attention"
    kv = _paged(where, k_pages, v_pages, table, lens, k_scale, v_scale)
    device, hd = k_pages.device, kv.head_dim
    _rows(where, "q", q, None, hd, device)
    dt = _HALF.get(q.dtype)
    if dt is None or q.shape[0] != kv.n_seqs:
        _refuse(where, "q must have one f16 or bf16 row per sequence")
    n, heads, _ = q.shape
    if out is None:
        out = torch.empty((n, heads, hd), dtype=q.dtype, device=device)
    else:
        _rows(where, "out", out, heads, hd, device)
        if out.dtype != q.dtype or out.shape[0] != n:
            _refuse(where, "out must be like q")
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()
                                  or workspace.device != device):
        _refuse(where, "workspace must be a contiguous uint8 tensor on the tensors' device")
    _call(device, _attention, kv, q, dt, heads, hd ** -0.5 if scale is None else scale, out, workspace,
          _status(where, status, device))
    return out


def _attention(kv, q, dt, heads, scale, out, workspace, status, stream):
    if workspace is None:
        workspace = torch.empty(adp.adp_paged_attention_workspace(kv, heads), dtype=torch.uint8, device=q.device)
    adp.adp_paged_attention(kv, q.data_ptr(), dt, heads, _row_stride(q), scale, out.data_ptr(), _row_stride(out),
                            workspace.data_ptr(), workspace.numel(), status, stream)


def packed_attention(q, k, v, cu_q, cu_k, *, scale: float | None = None, out=None, status=None):
    """Causal attention of packed prompts: q [rows, heads, head_dim], k, v [key rows, kv_heads, head_dim], f16 or bf16.

    cu_q, cu_k: int32 [seqs + 1] row offsets; query i of a sequence with lq queries and lk keys sees keys up to
    i + lk - lq.  scale: default 1 / sqrt(head_dim).  Rows of q from cu_q[-1] on are padding: their rows of `out`
    are left as they were (unset where out is allocated here)."""
    where = "packed_attention"
    device = q.device
    if device.type != "cuda" or q.dim() != 3 or k.dim() != 3:
        _refuse(where, "q, k and v must be [rows, heads, head_dim] on a CUDA device")
    n_q, heads, hd = q.shape
    n_k, kv_heads, _ = k.shape
    _rows(where, "q", q, None, hd, device)
    _rows(where, "k", k, kv_heads, hd, device)
    _rows(where, "v", v, kv_heads, hd, device)
    dt = _HALF.get(q.dtype)
    if dt is None or k.dtype != q.dtype or v.dtype != q.dtype or v.shape[0] != n_k:
        _refuse(where, "q, k and v must be alike, of f16 or bf16, with as many rows of v as of k")
    _indices(where, "cu_q", cu_q, 1, device)
    _indices(where, "cu_k", cu_k, 1, device)
    if cu_q.shape[0] < 1 or cu_k.shape != cu_q.shape:
        _refuse(where, "cu_q and cu_k must both have one entry more than there are sequences")
    if out is None:
        out = torch.empty((n_q, heads, hd), dtype=q.dtype, device=device)
    else:
        _rows(where, "out", out, heads, hd, device)
        if out.dtype != q.dtype or out.shape[0] != n_q:
            _refuse(where, "out must be like q")
    _call(device, adp.adp_packed_attention, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, heads, kv_heads, hd, _row_stride(q),
          _row_stride(k), _row_stride(v), cu_q.data_ptr(), cu_k.data_ptr(), cu_q.shape[0] - 1, n_q, n_k,
          hd ** -0.5 if scale is None else scale, out.data_ptr(), _row_stride(out), _status(where, status, device))
    return out
