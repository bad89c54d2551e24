"""Packed prompt attention without a GPU: what it refuses."""
import pytest

FAKE = 0x10000  # a 16-byte aligned address that no refused call reads


@pytest.fixture(scope="module")
def adp():
    from autoregressive_decode_persistent_gb300 import adp, build
    build.build()
    return adp


ARGS = dict(q=FAKE, k=FAKE, v=FAKE, dtype=0, n_heads=20, n_kv_heads=4, head_dim=128, q_stride=2560, k_stride=512,
            v_stride=512, cu_q=FAKE, cu_k=FAKE, n_seqs=3, n_q=100, n_k=200, scale=0.1, out=FAKE, out_stride=2560)


@pytest.mark.parametrize("change,code", [
    (dict(n_heads=0), -1), (dict(n_kv_heads=0), -1), (dict(n_heads=18), -1), (dict(n_seqs=-1), -1), (dict(n_q=-1), -1),
    (dict(n_k=-1), -1), (dict(scale=float("nan")), -1), (dict(scale=float("-inf")), -1), (dict(dtype=2), -2), (dict(dtype=3), -2),
    (dict(head_dim=96), -2), (dict(head_dim=256, q_stride=5120, out_stride=5120, k_stride=1024, v_stride=1024), -2),
    (dict(n_heads=129, n_kv_heads=1, q_stride=129 * 128, out_stride=129 * 128), -2), (dict(cu_q=None), -1), (dict(cu_k=None), -1),
    (dict(cu_q=FAKE + 2), -1), (dict(cu_k=FAKE + 1), -1), (dict(q=None), -1), (dict(out=None), -1), (dict(k=None), -1),
    (dict(v=None), -1), (dict(q=FAKE + 8), -1), (dict(k=FAKE + 2), -1), (dict(v=FAKE + 4), -1), (dict(out=FAKE + 8), -1),
    (dict(q_stride=2552), -1), (dict(q_stride=2564), -1), (dict(out_stride=2559), -1), (dict(k_stride=504), -1),
    (dict(v_stride=516), -1), (dict(dev_status=FAKE + 2), -1)])
def test_wrong_arguments_are_refused(adp, change, code):
    a = dict(ARGS)
    a.update(change)
    with pytest.raises(adp.AdpError) as e:
        adp.adp_packed_attention(**a)
    assert e.value.code == code


def test_no_sequences_and_no_queries_are_no_work(adp):
    adp.adp_packed_attention(**dict(ARGS, n_seqs=0, q=None, out=None))
    adp.adp_packed_attention(**dict(ARGS, n_q=0, q=None, out=None, k=None, v=None))


def test_tensors_off_the_gpu_are_refused():
    import torch
    from autoregressive_decode_persistent_gb300 import adp, ops
    x, cu = torch.zeros(4, 2, 64, dtype=torch.float16), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(adp.AdpError):
        ops.packed_attention(x, x, x, cu, cu)


def test_the_wait_limit_grows_with_the_work(tmp_path):
    """packed_wait_ns (csrc/paged.h): a wait may last for a whole piece of work, 13 ns a key, or for the search through
    the sequences, under 100 ns each; a quarter of the limit holds either, beyond a second for everything else."""
    import ctypes
    import os
    import subprocess
    src, lib = tmp_path / "wait.cpp", tmp_path / "wait.so"
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "autoregressive_decode_persistent_gb300", "csrc")
    src.write_text('#include "%s/paged.h"\nextern "C" uint64_t t_wait(int32_t k, int32_t s) { return adp::packed_wait_ns(k, s); }\n' % csrc)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    wait = ctypes.CDLL(str(lib)).t_wait
    wait.restype = ctypes.c_uint64
    top = 2 ** 31 - 1
    for keys in (0, 1, 8192, 10 ** 8, top):
        for seqs in (0, 1, 8192, 10 ** 7, top):
            assert wait(keys, seqs) >= 10 ** 9 + 4 * max(13 * keys, 100 * seqs)
            assert wait(keys, seqs) <= wait(top, top) < 2 ** 43  # (and ends)
    # the kernel takes its limits from there alone
    text = open(os.path.join(csrc, "packed_attention.cu")).read()
    assert "packed_wait_ns(n_k, n_seqs)" in text and "kWaitNs" not in text and "1000000000" not in text
