"""The pool's host side against a CUDA runtime that fails where it is told to (tests/host/pool_host.cpp),
on the CPU: plans that get no memory, the order of calls on several streams."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixed_precision_kv_gb300", "csrc")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime.h")):
        pytest.skip("g++ or the CUDA runtime headers are not available")
    exe = str(tmp_path_factory.mktemp("host") / "pool_host")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-x", "c++", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                        "-I" + os.path.join(CUDA, "include"), os.path.join(ROOT, "tests", "host", "pool_host.cpp"),
                        os.path.join(CSRC, "kvq_pool.cu"), "-o", exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                       text=True)
    assert r.returncode == 0, r.stdout
    return exe


@pytest.mark.parametrize("what", ["plan", "groups", "streams"])
def test_host_side(host, what):
    r = subprocess.run([host, what], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
