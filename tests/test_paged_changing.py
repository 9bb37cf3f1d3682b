"""The decode kernel's walk on the host, over lengths that another stream changes while
it runs: tests/host/changing_check.cu.  Its results are undefined then, but it ends and
stays within its sequences.  Mistakes planted in a copy must be found."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_io_aware_65_b200", "csrc")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

pytestmark = pytest.mark.skipif(not os.path.exists(NVCC), reason="needs nvcc")


def _run(out_dir, include_dir=CSRC):
    exe = os.path.join(out_dir, "changing_check")
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O2", "-I",
                    os.path.join(ROOT, "include"), "-I", include_dir,
                    os.path.join(ROOT, "tests", "host", "changing_check.cu"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


def test_the_walk_ends_within_its_sequences(tmp_path):
    r = _run(str(tmp_path))
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


@pytest.mark.parametrize("old,new", [
    ("if (w.hu >= k.HU) w.at = w.end;", ""),
    ("if (w.b + 1 >= k.B) return;", ""),
    ("return w.at < w.end && w.nblk > 0;", "return w.at < w.end;"),
    ("  if (c >= grid) c = grid - 1;", ""),
], ids=["unit", "sequence", "no_blocks", "past_the_last_cta"])
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
