"""Appends whose host allocations fail at every point in turn (tests/host/append_host.cpp), on the CPU: KV_ERR_OOM
leaves the pool as it was."""
import os
import shutil
import subprocess

import pytest

from test_lib_host_pool import CSRC, CUDA, ROOT


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime.h")):
        pytest.skip("g++ or the CUDA runtime headers are not available")
    exe = str(tmp_path_factory.mktemp("append") / "append_host")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-x", "c++", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                        "-I" + os.path.join(CUDA, "include"), os.path.join(ROOT, "tests", "host", "append_host.cpp"),
                        os.path.join(CSRC, "kvq_pool.cu"), "-o", exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                       text=True)
    assert r.returncode == 0, r.stdout
    return exe


@pytest.mark.parametrize("how", ["once", "on"])
@pytest.mark.parametrize("what", ["runs", "small", "mixed"])
def test_failing_allocations(host, what, how):
    r = subprocess.run([host, what, how], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
