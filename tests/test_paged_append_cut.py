"""How a row's heads are cut over warps (host code, shared with the launch of paged_kv_append)."""
import ctypes
import os
import random
import subprocess

import pytest

from test_paged import ROOT


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    d = tmp_path_factory.mktemp("append_cut")
    src, lib = d / "cut.cpp", d / "cut.so"
    src.write_text('#include "%s"\nextern "C" int32_t cut(int32_t h, int32_t s, int32_t n, int32_t w) { return adp::row_part_heads(h, s, n, w); }\n'
                   % os.path.join(ROOT, "autoregressive_decode_persistent_gb300", "csrc", "paged.h"))
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib)).cut


def test_rows_are_cut_no_finer_than_warps_run_at_once(cut):
    rng = random.Random(2)
    for _ in range(5000):
        step, held = rng.choice([4, 8]), rng.choice([1, 16, 108 * 16, 152 * 16, 152 * 20])
        heads, n = rng.randint(2, rng.choice([6, 48, 6144])), rng.choice([1, rng.randint(1, 40), rng.randint(1, 5000), 2 ** 31 - 1])
        own = cut(heads, step, n, held)
        parts = -(-heads // own)
        assert own % step == 0 and own >= step
        assert parts == 1 or n * parts <= held
        finer = own - step  # and not coarser than that allows
        assert finer == 0 or n * -(-heads // finer) > held or n > held
    assert cut(48, 4, 152 * 2, 152 * 16) == 8 and cut(48, 4, 152 * 12, 152 * 16) == 48 and cut(48, 4, 1, 152 * 16) == 4
