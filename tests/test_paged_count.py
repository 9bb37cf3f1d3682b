"""The counters of a divided unit's parts, on the host: tests/host/count_check.cu
runs the function of paged.cuh with threads as the CTAs, over words of any contents.
Mistakes planted in a copy must be found."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_io_aware_65_b200", "csrc")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

pytestmark = pytest.mark.skipif(not os.path.exists(NVCC), reason="needs nvcc")


def _run(out_dir, include_dir=CSRC):
    exe = os.path.join(out_dir, "count_check")
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O2", "-I",
                    os.path.join(ROOT, "include"), "-I", include_dir,
                    os.path.join(ROOT, "tests", "host", "count_check.cu"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


def test_parts_are_counted_over_any_contents(tmp_path):
    r = _run(str(tmp_path))
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


@pytest.mark.parametrize("old,new", [
    ("  if (((seen ^ tag) & ~COUNT) == 0) return (int)(seen & COUNT);", "  return (int)(seen & COUNT);"),
    ("if (was == seen) return 0;", "if (was == seen) return 1;"),
    ("const unsigned long long was = w.cas(seen, tag | 1u);", "const unsigned long long was = w.cas(seen, tag);"),
    ("return (int)(w.add(1) & COUNT);\n", "return (int)(was & COUNT);\n"),
], ids=["any_word_counts", "first_number", "first_not_counted", "later_not_counted"])
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


def test_no_counter_outlives_a_call():
    # the decode kernels' only words of their own on the device would be shared by
    # calls that have workspaces of their own
    src = open(os.path.join(CSRC, "fa_paged_decode.cu")).read()
    assert not [line for line in src.splitlines() if line.startswith("__device__") and "(" not in line]
