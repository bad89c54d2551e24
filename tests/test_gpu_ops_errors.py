"""Errors of PyTorch inside the tensor calls keep their type."""
import pytest
import torch

from test_gpu_paged import F16, Cache, ops  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture
def no_room(ops):  # noqa: F811
    """PyTorch's allocator may take nothing more of the GPU, and has nothing left of what it took."""
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction(max(torch.cuda.memory_reserved(), 1 << 20) / total)
    held, size = [], 64 << 20
    while size >= 512:
        try:
            held.append(torch.empty(size, dtype=torch.uint8, device="cuda"))
        except torch.OutOfMemoryError:
            size //= 2
    yield
    torch.cuda.set_per_process_memory_fraction(1.0)


def test_no_room_for_a_result_or_a_workspace(ops, request):  # noqa: F811
    c = Cache([9000, 40], 2, 64, 16, F16, 1)
    q = torch.zeros(2, 8, 64, dtype=F16, device="cuda")
    kv = torch.zeros(2, 2, 64, dtype=F16, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    angles = torch.zeros(9000, 32, device="cuda")
    wide = torch.full((2, 20000), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    out = torch.zeros_like(q)
    calls = [lambda o: ops.paged_kv_append(c.k, c.v, c.table, c.len_t, cu, q, kv, kv, angles, angles, out=o),
             lambda o: ops.paged_attention(q, c.k, c.v, wide, c.len_t, out=o),
             lambda o: ops.paged_attention(q, c.k, c.v, wide, c.len_t, window=20000, out=o),
             lambda o: ops.paged_chunk_attention(q, c.k, c.v, wide, c.len_t, cu, out=o)]
    want = [call(out).clone() for call in calls]
    torch.cuda.synchronize()
    request.getfixturevalue("no_room")
    for call in calls:
        with pytest.raises(torch.OutOfMemoryError):
            call(None)
    for call in calls[1:]:
        with pytest.raises(torch.OutOfMemoryError):
            call(out)
    calls[0](out)  # (needs no workspace)
    torch.cuda.set_per_process_memory_fraction(1.0)
    for call, w in zip(calls, want):
        assert torch.equal(call(None), w)
