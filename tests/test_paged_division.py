"""The paged kernels' division by the page size, and the decode call's walk over
whole units, on the host; planted mistakes in a copy must be found."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_io_aware_65_b200", "csrc")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

pytestmark = pytest.mark.skipif(not os.path.exists(NVCC), reason="needs nvcc")


def run(out_dir, include_dir, name="div_check"):
    exe = os.path.join(out_dir, name)
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O2", "-I",
                    os.path.join(ROOT, "include"), "-I", include_dir,
                    os.path.join(ROOT, "tests", "host", name + ".cu"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=120)


def test_division_by_the_page_size(tmp_path):
    r = run(str(tmp_path), CSRC)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


def test_a_planted_mistake_is_found(tmp_path):
    inc = tmp_path / "inc"
    inc.mkdir()
    for f in os.listdir(CSRC):
        if f.endswith((".h", ".cuh")):
            shutil.copy(os.path.join(CSRC, f), inc)
    src = (inc / "paged.cuh").read_text()
    old = "(((1ull << (31 + s)) + d - 1) / d)"
    assert src.count(old) == 1
    (inc / "paged.cuh").write_text(src.replace(old, "((1ull << (31 + s)) / d)"))
    assert run(str(tmp_path), str(inc)).returncode == 1


def test_whole_units(tmp_path):
    r = run(str(tmp_path), CSRC, "whole_check")
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout


def test_a_planted_mistake_in_the_walk_is_found(tmp_path):
    inc = tmp_path / "inc"
    inc.mkdir()
    for f in os.listdir(CSRC):
        if f.endswith((".h", ".cuh")):
            shutil.copy(os.path.join(CSRC, f), inc)
    src = (inc / "paged.cuh").read_text()
    old = "return w.blk > 0 ? w.at + (w.nblk - w.blk) : w.at;"
    assert src.count(old) == 1
    (inc / "paged.cuh").write_text(src.replace(old, "return w.at + (w.nblk - w.blk);"))
    assert run(str(tmp_path), str(inc), "whole_check").returncode == 1
