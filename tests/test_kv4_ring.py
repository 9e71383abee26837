"""The ring of stages of the attention over the 4-bit cache, on the host: a
model of producer, copies and consumer warps runs over the kernel's own order
of tiles and choice of barriers (csrc/kv4_ring.cuh)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def faults(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("ring") / "model")
    r = subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-x", "c++", "-I",
                        os.path.join(ROOT, "learned_kv_chunk_b200", "csrc"),
                        os.path.join(ROOT, "tests", "kv4_ring_model.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120, check=True).stdout
    lines = [line.split() for line in out.splitlines()]
    return {(int(nt), int(p), rule): (int(runs), int(bad)) for nt, p, rule, runs, bad in lines}


@pytest.mark.parametrize("nt,p", [(1, 1), (1, 2), (2, 1), (2, 2)])
def test_a_wait_passes_with_its_block_only(faults, nt, p):
    runs, bad = faults[nt, p, "two"]
    assert runs >= 1000 and bad == 0


@pytest.mark.parametrize("nt,p", [(1, 1), (2, 1), (2, 2)])
def test_the_model_finds_what_one_barrier_a_stage_does(faults, nt, p):
    """Warps of these shapes skip whole blocks: with one barrier they pass on a block that they never waited for."""
    assert faults[nt, p, "one"][1] > 0
