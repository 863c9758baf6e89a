"""When paged_tables_fork and paged_pages_compact are one cluster, and that they are
launched by grids where the GPU runs no cluster of that size: on a CUDA runtime that is
made up (host_clusters.cpp)."""
import os
import shutil
import subprocess

import pytest

import paged_kv_decode_rope_gb300 as pkv
from paged_kv_decode_rope_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc())))
    exe = str(tmp_path_factory.mktemp("host") / "host_clusters")
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-O1", "-rdynamic", f"-I{build.CSRC}", f"-I{cuda}/include",
                    os.path.join(HERE, "host_clusters.cpp"), "-o", exe, "-ldl"], check=True)
    pkv.lib()  # (built)
    return subprocess.run([exe, pkv.LIBRARY], check=True, capture_output=True, text=True).stdout.splitlines()


def launches(lines, what):
    got = []
    for line in lines:
        if line.startswith(what):
            rc, made = line.split(": ", 1)[1].split(";")[0].split(",")
            assert rc == "0", line
            got.append(made.split())
    return got


@pytest.mark.parametrize("what,rest", [("fork", 0), ("compaction", 1)])  # rest: launches after the cluster's
def test_one_cluster_or_grids(lines, what, rest):
    got = launches(lines, what)
    for i, made in enumerate(got):
        if i in (0, 3, 6, 8, 9, 10):
            assert made[:2] == ["cluster", "16"] and len(made) == 2 + rest, lines
        else:
            assert "cluster" not in made and len(made) == 3 + rest, lines
    assert len(got) == 11


@pytest.mark.parametrize("what", ["fork", "compaction"])
def test_a_device_is_asked_once(lines, what):
    asked = [int(line.split("asked ")[1].split()[0]) for line in lines if line.startswith(what)]
    assert asked == [1, 1, 1, 1, 2, 2, 2, 3, 4, 5, 6]  # (again where there was no answer, and past 64 devices)
