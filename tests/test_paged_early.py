"""The eviction's rule for idle SMs, on the host: tests/host/early_check.cu.  (With few
idle SMs each had the rows of up to 147 heads to wait for, one after the other: 352 us
for a call of 63.)  Mistakes planted in a copy must be found."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_io_aware_65_b200", "csrc")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

pytestmark = pytest.mark.skipif(not os.path.exists(NVCC), reason="needs nvcc")


def _run(out_dir, include_dir=CSRC):
    exe = os.path.join(out_dir, "early_check")
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O2", "-I",
                    os.path.join(ROOT, "include"), "-I", include_dir,
                    os.path.join(ROOT, "tests", "host", "early_check.cu"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


def test_idle_sms_have_few_heads_each(tmp_path):
    r = _run(str(tmp_path))
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


@pytest.mark.parametrize("old,new", [
    ("  if (heads > 2 * idle) return 0;\n", "  if (idle <= 0) return 0;\n"),
    ("return (int)(fit < recent ? fit : recent);", "return (int)fit;"),
    ("idle * (256LL << 10)", "idle * (256LL << 14)"),
], ids=["any_idle", "more_than_recent", "too_many"])
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
