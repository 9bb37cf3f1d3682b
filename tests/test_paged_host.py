"""The paged cache calls without a GPU: the functions that place rows and
divide work, walked on the host over good and bad tables (planted mistakes in a
copy must be found), and what the C ABI and the binding refuse before a
launch."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import exact_io_aware_65_b200 as fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_io_aware_65_b200", "csrc")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
needs_nvcc = pytest.mark.skipif(not os.path.exists(NVCC), reason="needs nvcc")


def _run(out_dir, include_dir=CSRC):
    exe = os.path.join(out_dir, "paged_check")
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O2", "-I",
                    os.path.join(ROOT, "include"), "-I", include_dir,
                    os.path.join(ROOT, "tests", "host", "paged_check.cu"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


@needs_nvcc
def test_every_block_is_walked_once_and_every_row_is_in_the_pool(tmp_path):
    r = _run(str(tmp_path))
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


@needs_nvcc
@pytest.mark.parametrize("old,new", [
    ("if (page < 0 || page >= c.num_pages) return -1;", "if (page >= c.num_pages) return -1;"),
    ("if (pos < 0 || i >= c.max_pages) return -1;", "if (pos < 0 || i > c.max_pages) return 0;"),
    ("return 2 * c + (cta_begin >= unit_begin ? 0 : 1);", "return 2 * c;"),
    ("  } while (w.nblk == 0 && w.b + 1 < k.B);", "  } while (false);"),
], ids=["negative_page", "table_width", "part_slot", "empty_sequences"])
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


# ---- the C ABI's refusals.  The pointers are never dereferenced.
FAKE = 1 << 20


def cache(**kw):
    c = dict(K=FAKE, V=FAKE, dtype=0, num_pages=10, page_size=16, Hkv=2, d=64, page_stride=2048, head_stride=1024,
             row_stride=64, k_scale=None, v_scale=None, page_table=FAKE, B=3, max_pages=4, table_stride=4)
    c.update(kw)
    return fa._PagedCache(*[c[f] for f, _ in fa._PagedCache._fields_])


def rows(**kw):
    r = dict(data=FAKE, row_stride=128, head_stride=64)
    r.update(kw)
    return fa._Rows(*[r[f] for f, _ in fa._Rows._fields_])


def call(name, c, *args):
    return getattr(fa.lib(), name)(ctypes.byref(c) if c is not None else None, *args, None)


BAD_CACHE = [
    (dict(K=None), 1), (dict(V=0), 1), (dict(page_table=None), 1), (dict(dtype=2), 1), (dict(num_pages=0), 1),
    (dict(page_size=0), 1), (dict(page_size=-16), 1), (dict(Hkv=0), 1), (dict(B=0), 1), (dict(max_pages=0), 1),
    (dict(K=FAKE + 8), 1), (dict(V=FAKE + 2), 1), (dict(page_table=FAKE + 2), 1), (dict(page_stride=2044), 1),
    (dict(head_stride=-1024), 1), (dict(row_stride=68), 1), (dict(row_stride=1 << 41), 1), (dict(table_stride=-1), 1),
    (dict(d=0), 1), (dict(d=96), 2), (dict(d=256), 2),
    (dict(dtype=1, row_stride=72), 1),                                # 8-bit rows on 8-byte boundaries
    (dict(max_pages=1 << 27), 2),                                     # positions past 2^30
    (dict(B=1 << 20, Hkv=32), 2), (dict(B=1 << 20, max_pages=1 << 15), 2),
]


@pytest.mark.parametrize("bad,code", BAD_CACHE, ids=[str(b) for b, _ in BAD_CACHE])
def test_every_call_refuses_a_bad_cache(bad, code):
    r = ctypes.byref(rows())
    c = cache(**bad)
    assert call("fa_paged_append", c, r, r, FAKE, FAKE, 5) == code
    assert call("fa_paged_decode", c, r, 4, FAKE, 0.1, None, 0, 0, 0, FAKE, FAKE, FAKE, 1 << 40) == code
    assert call("fa_paged_evict", c, FAKE, FAKE, 4, 4, FAKE, 128, 64, 16, 4, FAKE, 32, 16, 16, FAKE, FAKE) == code
    assert call("fa_paged_append", None, r, r, FAKE, FAKE, 5) == 1


def test_eight_bit_pools_need_scales_where_values_are_made_or_read():
    r = ctypes.byref(rows())
    for scales in (dict(k_scale=FAKE), dict(v_scale=FAKE), dict(k_scale=FAKE, v_scale=FAKE + 2)):
        c = cache(dtype=1, **scales)
        assert call("fa_paged_append", c, r, r, FAKE, FAKE, 5) == 1
        assert call("fa_paged_decode", c, r, 4, FAKE, 0.1, None, 0, 0, 0, FAKE, FAKE, FAKE, 1 << 40) == 1


def test_append_refusals():
    c, r = cache(), ctypes.byref(rows())
    assert call("fa_paged_append", c, r, r, FAKE, FAKE, -1) == 1
    assert call("fa_paged_append", c, r, r, None, FAKE, 5) == 1
    assert call("fa_paged_append", c, r, r, FAKE, FAKE + 1, 5) == 1
    assert call("fa_paged_append", c, r, r, FAKE, FAKE, (1 << 30) + 1) == 2
    for bad in (dict(data=None), dict(data=FAKE + 8), dict(row_stride=124), dict(head_stride=-64)):
        assert call("fa_paged_append", c, ctypes.byref(rows(**bad)), r, FAKE, FAKE, 5) == 1
        assert call("fa_paged_append", c, r, ctypes.byref(rows(**bad)), FAKE, FAKE, 5) == 1
    assert call("fa_paged_append", c, None, None, FAKE, FAKE, 0) == 0     # nothing to write: nothing is looked at


def test_decode_refusals():
    c, r = cache(), ctypes.byref(rows())

    def go(q=r, Hq=4, lens=FAKE, scale=0.1, W=None, wb=0, wh=0, O=FAKE, L=FAKE, ws=FAKE, n=1 << 40):
        return call("fa_paged_decode", c, q, Hq, lens, scale, W, wb, wh, 0, O, L, ws, n)

    for kw in (dict(q=None), dict(Hq=3), dict(Hq=0), dict(lens=None), dict(scale=0.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(scale=-1.0), dict(O=None), dict(O=FAKE + 8), dict(L=None), dict(L=FAKE + 2),
               dict(W=FAKE + 1), dict(W=FAKE, wb=-1), dict(W=FAKE, wh=-4)):
        assert go(**kw) == 1, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 16), dict(n=0), dict(W=FAKE, n=fa.paged_decode_workspace_size(3, 4, 2, 64, 64))):
        assert go(**kw) == 4, kw
    assert go(Hq=1 << 24) == 2


def test_decode_workspace_size():
    size = fa.paged_decode_workspace_size
    assert size(3, 4, 2, 64, 64) > 0
    assert size(3, 4, 2, 64, 1000, True) - size(3, 4, 2, 64, 1000) >= 3 * 4 * 1000 * 4
    assert size(3, 4, 2, 64, 1 << 20) == size(100, 4, 2, 64, 64)          # without weights: the GPU's, not the cache's
    for bad in ((0, 4, 2, 64, 64), (3, 5, 2, 64, 64), (3, 0, 2, 64, 64), (3, 4, 0, 64, 64), (3, 4, 2, 96, 64),
                (3, 4, 2, 64, 0), (3, 4, 2, 64, (1 << 30) + 1)):
        assert size(*bad) == 0


def test_evict_refusals():
    c = cache()   # 4 pages of 16: 64 positions at most

    def go(lens=FAKE, out=FAKE, ts=2, width=2, W=FAKE, wb=128, wh=64, budget=32, recent=4, Wo=FAKE, ob=64, oh=32, n=32,
           kept=FAKE, ln=FAKE):
        return call("fa_paged_evict", c, lens, out, ts, width, W, wb, wh, budget, recent, Wo, ob, oh, n, kept, ln)

    for kw in (dict(lens=None), dict(out=None), dict(W=None), dict(Wo=None), dict(kept=None), dict(ln=None),
               dict(W=FAKE + 2), dict(kept=FAKE + 1), dict(ts=-2), dict(wb=-1), dict(oh=-1), dict(budget=0),
               dict(budget=-5), dict(recent=-1), dict(recent=33), dict(width=0), dict(width=1), dict(n=31),
               dict(budget=100, n=63), dict(budget=100, n=64, width=3)):
        assert go(**kw) == 1, kw
    assert go(n=(1 << 30) + 1) == 2
    assert go(budget=(1 << 30) + 1, n=64, width=4) == 2


# ---- the binding's refusals
def test_binding_refuses_host_tensors_and_wrong_types():
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    pool = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    i = torch.zeros((2,), dtype=torch.int32)
    t = torch.zeros((2, 3), dtype=torch.int32)
    w = torch.zeros((2, 2, 48))
    for f in (lambda: fa.paged_append(q, q, i, i, pool, pool, t), lambda: fa.paged_decode(q, pool, pool, t, i),
              lambda: fa.paged_evict(w, pool, pool, t, i, t, 10, 2, w), lambda: fa._rows(q, "Q"),
              lambda: fa._rows(None, "Q"), lambda: fa._paged_cache(None, pool, t)):
        with pytest.raises(fa.FAError) as e:
            f()
        assert e.value.code == 1


CPU = torch.device("cpu")


def test_binding_checks_of_tables_lengths_and_weights():
    t = torch.zeros((3, 8), dtype=torch.int32)
    assert fa._table(t[:, :5], "t", CPU)[1:] == (5, 8)          # a slice of a wider table
    assert fa._table(t[:1], "t", CPU)[1:] == (8, 8)
    for bad in (t.long(), t[:, ::2], t[0], t[:0], t[:, :0], None):
        with pytest.raises(fa.FAError):
            fa._table(bad, "t", CPU)
    n = torch.zeros(4, dtype=torch.int32)
    assert fa._int32(n, "n", 4, CPU) == n.data_ptr()
    for bad in (n.float(), n[:3], torch.zeros(8, dtype=torch.int32)[::2], n[None], 4):
        with pytest.raises(fa.FAError):
            fa._int32(bad, "n", 4, CPU)
    w = torch.zeros(2, 3, 10)
    assert fa._weights(w[..., :7], "w", 2, 3, 7, CPU)[1:] == (30, 10)
    for bad in (w[..., :6], w.double(), w[..., ::2], w[0], w.transpose(0, 1), None):
        with pytest.raises(fa.FAError):
            fa._weights(bad, "w", 2, 3, 7, CPU)
