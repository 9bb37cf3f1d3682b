"""Slots with one owner each (slots.h): tests/host/slots_check.cu runs them with
threads on the host.  Mistakes planted in a copy must be found."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_io_aware_65_b200", "csrc")
CXX = os.environ.get("CXX", "g++")

pytestmark = pytest.mark.skipif(shutil.which(CXX) is None, reason="needs a C++ compiler")


def _run(out_dir, include_dir=CSRC):
    exe = os.path.join(out_dir, "slots_check")
    subprocess.run([CXX, "-x", "c++", "-std=c++17", "-O2", "-pthread", "-I", include_dir,
                    os.path.join(ROOT, "tests", "host", "slots_check.cu"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


def test_a_slot_has_one_owner(tmp_path):
    r = _run(str(tmp_path))
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr


@pytest.mark.parametrize("old,new", [
    ("const uint32_t w = (first + i) % (N / 64);", "const uint32_t w = first;"),
    ("u | 1ull << bit", "u"),
    ("fetch_and(~(1ull << (slot % 64))", "fetch_and(~0ull"),
    ("fetch_and(~(1ull << (slot % 64))", "fetch_and(0ull"),
], ids=["one_word", "not_marked", "never_given_back", "too_many_given_back"])
def test_planted_mistakes_are_found(tmp_path, old, new):
    inc = tmp_path / "inc"
    inc.mkdir()
    src = open(os.path.join(CSRC, "slots.h")).read()
    assert src.count(old) == 1
    (inc / "slots.h").write_text(src.replace(old, new))
    assert _run(str(tmp_path), str(inc)).returncode != 0


def test_a_captured_launch_takes_a_slot_of_its_own():
    # (a turn over a pool would lend a graph's slot again while the graph lives)
    src = open(os.path.join(CSRC, "fa_fwd.cu")).read()
    body = src[src.index("static fa_status next_slot("):]
    body = body[:body.index("\n}\n")]
    assert body.index("graph_slots.take()") < body.index("cudaGraphRetainUserObject(")
    assert "% TURN_SLOTS" in body and "TURN_SLOTS + (uint32_t)mine" in body
