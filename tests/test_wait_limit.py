"""A bounded wait takes a WaitLimit and nothing else: a number of keys or rows of the same name as the
limit cannot be taken for one. Compiles one line each way; no GPU needed."""
import os
import subprocess

import pytest

from sparse_kv_cache_snapkv_gb300 import _build

LINE = """#include "common.cuh"
__global__ void k(uint64_t* bar, int last, bool* out) { *out = rkv::%s(bar, 0u, %s); }
"""


@pytest.mark.parametrize("wait", ["mbar_wait", "mbar_wait_warp"])
@pytest.mark.parametrize("limit,builds", [("rkv::kWaitLimit", True), ("last", False)])
def test_wait_takes_a_limit_only(tmp_path, wait, limit, builds):
    src = os.path.join(tmp_path, "w.cu")
    with open(src, "w") as f:
        f.write(LINE % (wait, limit))
    r = subprocess.run([_build._nvcc(), *_build.ARCH, "-std=c++17", f"-I{_build.CSRC}",
                        f"-I{os.path.join(_build.ROOT, 'include')}", "-c", src, "-o", src + ".o"],
                       capture_output=True, text=True)
    assert (r.returncode == 0) == builds, r.stderr
    if not builds:
        assert "WaitLimit" in r.stderr
