"""Where the append kernel finds a position's row, on the host: tests/host/place_check.cu
runs the functions of paged.cuh that it uses over positions inside and outside the table.  Mistakes planted in a copy must be found."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_io_aware_65_b200", "csrc")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

pytestmark = pytest.mark.skipif(not os.path.exists(NVCC), reason="needs nvcc")


def _run(out_dir, include_dir=CSRC):
    exe = os.path.join(out_dir, "place_check")
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O2", "-I",
                    os.path.join(ROOT, "include"), "-I", include_dir,
                    os.path.join(ROOT, "tests", "host", "place_check.cu"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


def test_every_position_ends_in_its_row_or_nowhere(tmp_path):
    r = _run(str(tmp_path))
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


@pytest.mark.parametrize("old,new", [
    ("if (pos < 0 || i >= c.max_pages) return -1;", "if (i >= c.max_pages) return -1;"),
    ("if (pos < 0 || i >= c.max_pages) return -1;", "if (pos < 0 || i > c.max_pages) return -1;"),
    ("return Divider{(uint32_t)(((1ull << (31 + s)) + d - 1) / d), 31 + s};",
     "return Divider{(uint32_t)((1ull << (31 + s)) / d), 31 + s};"),
], ids=["negative", "one_past", "rounded_down"])
def test_planted_mistakes_are_found(tmp_path, old, new):
    inc = tmp_path / "inc"
    inc.mkdir()
    for f in os.listdir(CSRC):
        if f.endswith((".h", ".cuh")):
            shutil.copy(os.path.join(CSRC, f), inc)
    src = (inc / "paged.cuh").read_text()
    assert src.count(old) == 1
    (inc / "paged.cuh").write_text(src.replace(old, new))
    assert _run(str(tmp_path), str(inc)).returncode != 0
