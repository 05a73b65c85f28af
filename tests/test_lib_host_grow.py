"""How the library's workspaces grow (csrc/kvq_grow.h), on the CPU: the sizes asked for, in order,
where there is memory for `limit` bytes."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = r"""
#include <cstdio>
#include <cstdlib>
#include "kvq_grow.h"
int main(int c, char** v) {
  const size_t limit = strtoull(v[4], nullptr, 10);
  const size_t got = kvq::grow(strtoull(v[1], nullptr, 10), strtoull(v[2], nullptr, 10), strtoull(v[3], nullptr, 10),
                               [&](size_t n) { printf("%zu ", n); return n <= limit; });
  printf("%zu\n", got);
}
"""
MAX = 2 ** 64 - 1
G = 1 << 30


@pytest.fixture(scope="module")
def grow(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not available")
    d = tmp_path_factory.mktemp("grow")
    (d / "grow.cpp").write_text(SRC)
    subprocess.run(["g++", "-std=c++17", "-I" + os.path.join(ROOT, "mixed_precision_kv_gb300", "csrc"), str(d / "grow.cpp"),
                    "-o", str(d / "grow")], check=True)
    return lambda *a: list(map(int, subprocess.run([str(d / "grow"), *map(str, a)], capture_output=True, text=True,
                                                   check=True).stdout.split()))


def test_doubled_while_it_grows(grow):
    assert grow(0, 1000, MAX, MAX) == [1024, 1024]
    assert grow(1024, 1025, MAX, MAX) == [2048, 2048]
    assert grow(1024, 5000, MAX, MAX) == [5120, 5120]


def test_not_doubled_past_its_bound(grow):
    assert grow(3 * G, 3 * G + 1, 4 * G, MAX) == [4 * G, 4 * G]
    assert grow(3 * G, 5 * G, 4 * G, MAX) == [5 * G, 5 * G]           # needed
    assert grow(5 * G, 6 * G, 4 * G, MAX) == [6 * G, 6 * G]


def test_what_is_needed_where_there_is_no_memory_for_more(grow):
    assert grow(3 * G, 3 * G + 1, MAX, 5 * G) == [6 * G, 3 * G + 256, 3 * G + 256]
    assert grow(3 * G, 3 * G + 1, MAX, 2 * G) == [6 * G, 3 * G + 256, 0]
    assert grow(0, 3 * G, MAX, 2 * G) == [3 * G, 0]                   # not asked for twice
