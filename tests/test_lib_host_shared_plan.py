"""The plan of decode steps over shared prefixes beside the decode's (tests/host/shared_plan_host.cpp), on the CPU."""
import os
import shutil
import subprocess

import pytest

from test_lib_host_pool import CSRC, CUDA, ROOT


def test_plans_apart(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime.h")):
        pytest.skip("g++ or the CUDA runtime headers are not available")
    exe = str(tmp_path / "shared_plan_host")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-x", "c++", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                        "-I" + os.path.join(CUDA, "include"), os.path.join(ROOT, "tests", "host", "shared_plan_host.cpp"),
                        os.path.join(CSRC, "kvq_pool.cu"), "-o", exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                       text=True)
    assert r.returncode == 0, r.stdout
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
