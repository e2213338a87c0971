"""bench.py's passes are found in a profile by kernel name: every name it looks for is one of a
kernel that the library has, and of one kernel only (but for the products' tile forms)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402
from hadamard_rotated_precision_halo_amd import build  # noqa: E402


@pytest.fixture(scope="module")
def kernels():
    """Demangled names of the library's kernel handles, as a profile prints them."""
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("no nm")
    if not os.path.exists(build.LIB):
        build.build()
    out = subprocess.run([nm, "-C", build.LIB], capture_output=True, text=True, check=True).stdout
    names = [l.split(" ", 2)[2] for l in out.splitlines() if l.count(" ") >= 2]
    names = [n for n in names if "kernel" in n and "__device_stub__" not in n]
    assert names
    return names


@pytest.mark.parametrize("key", [k for k in bench.PASSES if k != "copy_neg"])
def test_pass_names_a_kernel_of_the_library(kernels, key):
    hits = {n.split("(halo::")[0].split("(float*")[0] for n in kernels if bench.pass_match(key, n, None)}
    assert hits, bench.PASSES[key]
    if not key.startswith("gemm"):
        assert len(hits) == 1, hits
