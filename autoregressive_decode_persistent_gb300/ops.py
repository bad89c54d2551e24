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


# The checks below read each tensor's properties once: on the host of a GB300 a property costs about 0.1 us, and a
# call's marshalling is what its smallest uses wait for.

def _indices(where: str, name: str, t: torch.Tensor, n: int, device: int) -> int:
    """Address of a contiguous int32 [n] tensor on the device."""
    if t.dtype is not torch.int32 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != device:
        _refuse(where, f"{name} must be a contiguous int32 tensor [{n}] on device {device}")
    return t.data_ptr()


def _rows(where: str, name: str, t: torch.Tensor, shape, dtype, device: int) -> int:
    """Elements from one row to the next of a [rows, heads, head_dim] tensor whose rows may lie apart."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        _refuse(where, f"{name} must be {tuple(shape)} of {dtype} on device {device}")
    n, heads, hd = shape
    if t.is_contiguous() or n == 0:
        return heads * hd
    rows, between, inner = t.stride()
    if inner != 1 or (between != hd and heads > 1):
        _refuse(where, f"{name} must have contiguous heads")
    return rows if n > 1 else heads * hd  # (the stride of a single row says nothing)


def _status(where: str, t: torch.Tensor | None, device: int):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.numel() != 1 or t.get_device() != device:
        _refuse(where, f"status must be one int32 on device {device}")
    return t.data_ptr()


def _call(device: int, name: str, *args):
    """The C ABI's function `name` on the current stream, with the tensors' device current."""
    if device == torch._C._cuda_getDevice():
        adp._check(getattr(adp.load_library(), name)(*args, torch._C._cuda_getCurrentRawStream(device)), name)
    else:
        with torch.cuda.device(device):
            adp._check(getattr(adp.load_library(), name)(*args, torch._C._cuda_getCurrentRawStream(device)), name)


def _paged(where: str, k_pages, v_pages, table, lens, k_scale, v_scale, device: int) -> adp.PagedKV:
    if not k_pages.is_cuda:
        _refuse(where, "the tensors must be on a CUDA device")
    shape, torch_dtype = k_pages.shape, k_pages.dtype
    dtype = _CACHE.get(torch_dtype)
    if dtype is None or len(shape) != 4 or v_pages.dtype is not torch_dtype or v_pages.shape != shape \
            or v_pages.get_device() != device:
        _refuse(where, "k_pages and v_pages must be alike: [pages, kv_heads, page_size, head_dim], f16, bf16 or e4m3")
    n_pages, heads, ps, hd = shape
    page = heads * ps * hd
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        stride = k_pages.stride()
        if v_pages.stride() != stride:
            _refuse(where, "k_pages and v_pages must have the same strides")
        if page and (stride[3] != 1 or (stride[2] != hd and ps > 1) or (stride[1] != ps * hd and heads > 1)):
            _refuse(where, "a page must be contiguous")
        if n_pages > 1:  # (the stride of a single page says nothing)
            page = stride[0]
    if table.dtype is not torch.int32 or len(table.shape) != 2 or not table.is_contiguous() or table.get_device() != device:
        _refuse(where, f"table must be a contiguous int32 tensor [seqs, width] on device {device}")
    n_seqs, width = table.shape
    at = _indices(where, "lens", lens, n_seqs, device)
    ks = vs = None
    scales = heads * ps
    if dtype == adp.ADP_E4M3:
        if k_scale is None or v_scale is None or k_scale.dtype is not torch.float32 \
                or v_scale.dtype is not torch.float32 or k_scale.shape != shape[:3] or v_scale.shape != shape[:3] \
                or k_scale.get_device() != device or v_scale.get_device() != device:
            _refuse(where, "e4m3 pages need k_scale and v_scale: fp32 [pages, kv_heads, page_size]")
        if not (k_scale.is_contiguous() and v_scale.is_contiguous()):
            stride = k_scale.stride()
            if v_scale.stride() != stride or (stride[2] != 1 and ps > 1) or (stride[1] != ps and heads > 1):
                _refuse(where, "k_scale and v_scale must have the same strides, and contiguous pages")
            if n_pages > 1:
                scales = stride[0]
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    return adp.PagedKV(k_pages.data_ptr(), v_pages.data_ptr(), ks, vs, table.data_ptr(), at, page, scales, n_pages, ps, heads,
                       hd, dtype, n_seqs, width)


def paged_kv_write(k_pages, v_pages, table, lens, cu_rows, k, v, *, k_scale=None, v_scale=None, status=None):
    """Write packed rows k, v [rows, kv_heads, head_dim] (f16, bf16 or f32) into their sequences' last positions.

    k_pages, v_pages: [pages, kv_heads, page_size, head_dim] f16, bf16 or float8_e4m3fn (then with fp32
    k_scale, v_scale [pages, kv_heads, page_size]), changed in place.  table: int32 [seqs, width] page numbers;
    lens: int32 [seqs], the rows being written included; cu_rows: int32 [seqs + 1]."""
    _transfer("paged_kv_write", k_pages, v_pages, table, lens, cu_rows, k, v, k_scale, v_scale, status)


def paged_kv_read(k_pages, v_pages, table, lens, cu_rows, n_rows: int, *, dtype=None, k_scale=None, v_scale=None,
                  out=None, status=None):
    """Read every sequence's last cu_rows[s + 1] - cu_rows[s] positions back into packed rows.

    Returns (k, v) [n_rows, kv_heads, head_dim] of `dtype` (default: the pages' type, fp16 for e4m3 pages), or
    writes into out = (k, v); rows from cu_rows[-1] on are left as they were."""
    if out is None:
        if dtype is None:
            dtype = torch.float16 if k_pages.dtype is torch.float8_e4m3fn else k_pages.dtype
        if len(k_pages.shape) != 4 or n_rows < 0 or dtype not in _ROWS:
            _refuse("paged_kv_read", "pages [pages, kv_heads, page_size, head_dim] are read as n_rows >= 0 rows of f16, bf16 or f32")
        _, heads, _, hd = k_pages.shape
        like = dict(dtype=dtype, device=k_pages.device)
        k, v = out = torch.empty((n_rows, heads, hd), **like), torch.empty((n_rows, heads, hd), **like)
    else:
        if len(out) != 2:
            _refuse("paged_kv_read", "out must be (k, v)")
        k, v = out
        if len(k.shape) != 3 or k.shape[0] != n_rows or (dtype is not None and k.dtype is not dtype):
            _refuse("paged_kv_read", "out must hold n_rows rows of dtype")
    _transfer("paged_kv_read", k_pages, v_pages, table, lens, cu_rows, k, v, k_scale, v_scale, status)
    return out


def _transfer(where, k_pages, v_pages, table, lens, cu_rows, k, v, k_scale, v_scale, status):
    device = k_pages.get_device()
    kv = _paged(where, k_pages, v_pages, table, lens, k_scale, v_scale, device)
    cu = _indices(where, "cu_rows", cu_rows, kv.n_seqs + 1, device)
    dtype, shape = k.dtype, k.shape
    dt = _ROWS.get(dtype)
    if dt is None or len(shape) != 3:
        _refuse(where, "k and v rows must be [rows, kv_heads, head_dim] of f16, bf16 or f32")
    n = shape[0]
    shape = (n, kv.n_kv_heads, kv.head_dim)
    ks, vs = _rows(where, "k", k, shape, dtype, device), _rows(where, "v", v, shape, dtype, device)
    _call(device, "adp_" + where, kv, k.data_ptr(), v.data_ptr(), dt, ks, vs, cu, n, _status(where, status, device))


def paged_attention(q, k_pages, v_pages, table, lens, *, scale: float | None = None, k_scale=None, v_scale=None,
                    out=None, workspace=None, status=None):
    """Attention of one new token per sequence, q [seqs, heads, head_dim] f16 or bf16, over its cached positions.

    scale: default 1 / sqrt(head_dim).  workspace: optional uint8 tensor of adp.adp_paged_attention_workspace
    bytes (not shared by calls that may run at the same time); by default one is allocated on the current stream.
    The work is split by the table's width: a table no wider than the longest context is fastest."""
    where = "paged_attention"
    device = k_pages.get_device()
    kv = _paged(where, k_pages, v_pages, table, lens, k_scale, v_scale, device)
    dtype, shape = q.dtype, q.shape
    dt = _HALF.get(dtype)
    if dt is None or len(shape) != 3 or shape[0] != kv.n_seqs or shape[2] != kv.head_dim or shape[2] < 1:
        _refuse(where, "q must be [seqs, heads, head_dim] of f16 or bf16")
    qs = _rows(where, "q", q, shape, dtype, device)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        os = shape[1] * shape[2]
    else:
        os = _rows(where, "out", out, shape, dtype, device)
    if workspace is not None:
        need = workspace.numel()
        if workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != device:
            _refuse(where, "workspace must be a contiguous uint8 tensor on the tensors' device")
    else:
        if device == torch._C._cuda_getDevice():
            need = adp.adp_paged_attention_workspace(kv, shape[1])
        else:
            with torch.cuda.device(device):
                need = adp.adp_paged_attention_workspace(kv, shape[1])
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _call(device, "adp_paged_attention", kv, q.data_ptr(), dt, shape[1], qs, shape[2] ** -0.5 if scale is None else scale,
          out.data_ptr(), os, workspace.data_ptr() if need else None, need, _status(where, status, device))
    return out


def packed_attention(q, k, v, cu_q, cu_k, *, scale: float | None = None, out=None, status=None):
    """Causal attention of packed prompts: q [rows, heads, head_dim], k, v [key rows, kv_heads, head_dim], f16 or bf16.

    cu_q, cu_k: int32 [seqs + 1] row offsets; query i of a sequence with lq queries and lk keys sees keys up to
    i + lk - lq.  scale: default 1 / sqrt(head_dim).  Rows of q from cu_q[-1] on are padding: their rows of `out`
    are left as they were (unset where out is allocated here).  A wait inside the kernel that ran out (on a GPU that stood
    still for a second) leaves rows unset, too: `status` tells."""
    where = "packed_attention"
    device = q.get_device()
    if not q.is_cuda or len(q.shape) != 3 or len(k.shape) != 3:
        _refuse(where, "q, k and v must be [rows, heads, head_dim] on a CUDA device")
    shape, kv_shape, dtype = q.shape, k.shape, q.dtype
    n_q, heads, hd = shape
    n_k, kv_heads, kd = kv_shape
    dt = _HALF.get(dtype)
    if dt is None or kd != hd or hd < 1:
        _refuse(where, "q, k and v must be of f16 or bf16, with one head_dim")
    qs = _rows(where, "q", q, shape, dtype, device)
    ks, vs = _rows(where, "k", k, kv_shape, dtype, device), _rows(where, "v", v, kv_shape, dtype, device)
    n = cu_q.numel()
    if n < 1:
        _refuse(where, "cu_q must have one entry more than there are sequences")
    cq, ck = _indices(where, "cu_q", cu_q, n, device), _indices(where, "cu_k", cu_k, n, device)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        os = heads * hd
    else:
        os = _rows(where, "out", out, shape, dtype, device)
    _call(device, "adp_packed_attention", q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, heads, kv_heads, hd, qs, ks, vs,
          cq, ck, n - 1, n_q, n_k, hd ** -0.5 if scale is None else scale, out.data_ptr(), os, _status(where, status, device))
    return out
