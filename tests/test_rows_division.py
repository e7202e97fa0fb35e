"""The row attention kernel's row / (query heads per KV head), checked on the
host over divisors and rows up to 2^32, and the sizes that depend on it taken
by the calls (no device work)."""
import ctypes
import os
import subprocess

import pytest

from test_decode_layout import NVCC, ROOT, HERE
from test_rows_args import cross, desc, lib, shared  # noqa: F401 (lib is a fixture)


@pytest.mark.timeout(600)
def test_division_is_exact(tmp_path):
    exe = str(tmp_path / "row_division_check")
    subprocess.run([NVCC, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a",
                    "-I", os.path.join(ROOT, "bit_kv_cache_centroid_b200", "csrc"),
                    os.path.join(HERE, "host", "row_division_check.cu"), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-3000:]


def test_large_groups_are_taken_up_to_the_row_limit(lib):  # noqa: F811
    # (ws of no bytes: the call ends at the workspace's check)
    p, c = desc(B=1), desc(B=6101)
    assert shared(lib, p, c, H_q=2000, n=0) == 6
    assert lib.kv2_attention_shared_workspace_size(ctypes.byref(p), ctypes.byref(c), 2000, 256, 256) > 0
    assert cross(lib, desc(B=1), Nq=4097, H_q=1 << 17, n=0) == 6                 # 2^16 heads a KV head
    # one row below, at and above 2^30
    assert cross(lib, desc(B=1, H_kv=1), Nq=1 << 10, H_q=1 << 20, n=0) == 6
    assert cross(lib, desc(B=1, H_kv=1), Nq=1 << 10, H_q=(1 << 20) + 1, n=0) == 2
    assert shared(lib, p, desc(B=1 << 10, H_kv=1), H_q=(1 << 20) + 1, n=0) in (1, 2)
    assert shared(lib, desc(B=1, H_kv=1), desc(B=1 << 10, H_kv=1), H_q=(1 << 20) + 1, n=0) == 2
