"""The packed attention calls without a GPU: their schedules and masks walked on
the host (planted mistakes in a copy must be found), the 64-bit gradients
against differences, and what the C ABI and the binding refuse before a
launch."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import exact_io_aware_65_b200 as fa
import packed_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_io_aware_65_b200", "csrc")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
needs_nvcc = pytest.mark.skipif(not os.path.exists(NVCC), reason="needs nvcc")


def _run(out_dir, include_dir=CSRC):
    exe = os.path.join(out_dir, "pack_check")
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O2", "-I",
                    os.path.join(ROOT, "include"), "-I", include_dir,
                    os.path.join(ROOT, "tests", "host", "pack_check.cu"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


@needs_nvcc
def test_schedules_and_masks_of_packed_sequences(tmp_path):
    r = _run(str(tmp_path))
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


@needs_nvcc
@pytest.mark.parametrize("header,old,new", [
    ("pack.cuh", "return -L & 127;", "return L & 127;"),
    ("pack.cuh", "return (sq >> 7) + b;", "return (sq >> 7);"),
    ("pack.cuh", "s.Lk = min(max(ld_ro(k.cu_k + b + 1), s.sk), k.Tk) - s.sk;", "s.Lk = ld_ro(k.cu_k + b + 1) - s.sk;"),
    ("pack.cuh", "const int gsize = min(u.group, u.heads - g * u.group);", "const int gsize = u.group;"),
    ("fwd_sched.cuh", "it.q0 = it.has1 ? it.q1 - 1 : 0;", "it.q0 = it.q1 - 1;"),
    ("fwd_sched.cuh", "max(0, min(nkb, qt + off + 1)) : nkb;", "max(0, min(nkb, qt + off)) : nkb;"),
    ("fwd_sched.cuh", "it.j1 = it.part < it.parts ? e * (it.part + 1) / it.parts : 0;",
     "it.j1 = it.part < it.parts ? e / it.parts * (it.part + 1) : 0;"),
    ("fwd_sched.cuh", "nq - 1 - (nq - 1 - qt) / 2 * 2 : qt;", "qt / 2 * 2 + 1 : qt;"),
    ("bwd_sched.cuh", "return p.mask_kind == FA_MASK_CAUSAL ? max(0, it.j - it.off) : 0;",
     "return p.mask_kind == FA_MASK_CAUSAL ? max(0, it.j) : 0;"),
    ("bwd_sched.cuh", "it.g1 = (it.part + 1) * p.pk.G / p.parts;", "it.g1 = it.g0 + p.pk.G / p.parts;"),
], ids=["pad", "slot_base", "clamp", "last_group", "odd_pair", "kv_end", "key_parts", "join_tile", "first_query", "parts"])
def test_planted_mistakes_are_found(tmp_path, header, old, new):
    inc = tmp_path / "inc"
    inc.mkdir()
    for f in os.listdir(CSRC):
        if f.endswith((".h", ".cuh")):
            shutil.copy(os.path.join(CSRC, f), inc)
    src = (inc / header).read_text()
    assert src.count(old) == 1
    (inc / header).write_text(src.replace(old, new))
    assert _run(str(tmp_path), str(inc)).returncode != 0


@pytest.mark.parametrize("causal", [False, True])
def test_the_64_bit_gradients_are_the_differences(causal):
    g = torch.Generator().manual_seed(0)
    x = [torch.randn(s, generator=g, dtype=torch.float64) for s in ((30, 6, 8), (41, 2, 8), (41, 2, 8), (30, 6, 8))]
    cq, ck, scale = [0, 7, 7, 30], [0, 12, 20, 41], 0.3
    f = lambda Q, K, V: float((ref.fwd(Q, K, V, cq, ck, causal, scale)[0] * x[3]).sum())
    O, L = ref.fwd(*x[:3], cq, ck, causal, scale)[:2]
    grads = ref.bwd(*x[:3], O, x[3], L, cq, ck, causal, scale)
    h = 1e-5
    for i in range(3):
        r = torch.randn(x[i].shape, generator=g, dtype=torch.float64)
        step = lambda e: f(*[t + e * r if j == i else t for j, t in enumerate(x[:3])])
        assert abs((step(h) - step(-h)) / (2 * h) - float((grads[i][0] * r).sum())) < 1e-7


# ---- the C ABI's refusals.  The pointers are never dereferenced.
FAKE = 1 << 20


def rows(**kw):
    r = dict(data=FAKE, row_stride=256, head_stride=64)
    r.update(kw)
    return fa._Rows(*[r[f] for f, _ in fa._Rows._fields_])


def calls(over, **kw):
    """Status of the forward and of the backward with one argument changed."""
    a = dict(Q=rows(), K=rows(), V=rows(), O=rows(), dO=rows(), LSE=FAKE, cu_q=FAKE, cu_k=FAKE, B=2, Tq=100, Tk=120,
             Hq=4, Hkv=2, d=64, mask=1, scale=0.1, dQ=rows(), dK=rows(), dV=rows(), ws=FAKE, wn=1 << 40)
    a.update(over)
    p = {k: ctypes.byref(v) if isinstance(v, fa._Rows) else v for k, v in a.items()}
    sizes = [p[k] for k in ("B", "Tq", "Tk", "Hq", "Hkv", "d", "mask", "scale")]
    L = fa.lib()
    return (L.fa_fwd_packed(p["Q"], p["K"], p["V"], p["cu_q"], p["cu_k"], *sizes, p["O"], p["LSE"], p["ws"], p["wn"], None),
            L.fa_bwd_packed(p["Q"], p["K"], p["V"], p["O"], p["dO"], p["LSE"], p["cu_q"], p["cu_k"], *sizes, 0, p["dQ"],
                            p["dK"], p["dV"], p["ws"], p["wn"], None))


@pytest.mark.parametrize("over,code", [
    (dict(Q=None), 1), (dict(K=rows(data=0)), 1), (dict(V=rows(data=FAKE + 8)), 1), (dict(O=rows(row_stride=260)), 1),
    (dict(Q=rows(head_stride=0)), 1), (dict(K=rows(row_stride=0)), 1), (dict(V=rows(row_stride=-256)), 1),
    (dict(LSE=None), 1), (dict(LSE=FAKE + 2), 1), (dict(cu_q=None), 1), (dict(cu_k=FAKE + 1), 1), (dict(B=0), 1),
    (dict(Tq=-1), 1), (dict(Tk=-5), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(d=0), 1), (dict(d=96), 2), (dict(mask=2), 2),
    (dict(mask=3), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(Tq=(1 << 28) + 1), 2), (dict(Tk=(1 << 28) + 1), 2), (dict(B=1 << 25), 2), (dict(Hq=1 << 30), 2),
], ids=str)
def test_both_calls_refuse(over, code):
    assert calls(over) == (code, code)


def test_the_backward_refuses_more():
    for over, code in ((dict(dO=None), 1), (dict(dQ=rows(data=0)), 1), (dict(dK=rows(head_stride=4)), 1),
                       (dict(dV=rows(row_stride=0)), 1), (dict(ws=None), 4), (dict(ws=FAKE + 128), 4), (dict(wn=1000), 4)):
        assert calls(over)[1] == code, over


def test_the_binding_packs_the_header_s_structures():
    for packed, struct in ((fa._ROWS, fa._Rows), (fa._CACHE, fa._PagedCache)):
        n = len(struct._fields_)
        assert packed.size == ctypes.sizeof(struct)
        assert packed.pack(*range(1, n + 1)) == bytes(struct(*range(1, n + 1)))


def test_nothing_to_do():
    empty = dict(Tq=0, Q=rows(data=0), O=rows(data=0), dO=rows(data=0), dQ=rows(data=0))
    assert calls(empty | dict(Tk=0, K=rows(data=0), V=rows(data=0), dK=rows(data=0), dV=rows(data=0), ws=None)) == (0, 0)


def test_forward_workspace_sizes():
    size = fa.fwd_packed_workspace_size
    assert size(1, 100, 3, 2, 64) == 0 and size(1, 100, 4, 2, 96) == 0 and size(0, 1, 1, 1, 64) == 0 and size(1, 0, 1, 1, 64) == 0
    assert size(4, 8192, 32, 8, 128) == 0                     # enough query tiles: the keys stay whole
    one = 100 * 4 * (128 + 2) * 4                             # a part: unnormalised O, maximum and sum
    assert size(1, 100, 4, 2, 128) >= 2 * one
    for over in (dict(ws=None), dict(ws=FAKE + 128), dict(wn=1000)):
        assert calls(dict(Tk=5000) | over)[0] == 4


def test_workspace_sizes():
    size = fa.bwd_packed_workspace_size
    assert size(1, 100, 100, 3, 2, 64) == 0 and size(1, 100, 100, 4, 2, 96) == 0 and size(0, 1, 1, 1, 1, 64) == 0
    assert size(1, (1 << 28) + 1, 1, 1, 1, 64) == 0
    one = 2 * 128 * 64 * 4  # two slots of 128 rows for up to 255 rows in one sequence
    assert one < size(1, 200, 200, 1, 1, 64) < one + 2 * 128 * 8 + 2048
    assert size(1, 200, 200, 8, 1, 64) > 8 * one  # and the key head's parts


def test_the_binding_refuses_host_tensors_and_other_shapes():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(fa.FAError):
        fa.fwd_packed(x, x, x, cu, cu)
    with pytest.raises(fa.FAError):
        fa.bwd_packed(x, x, x, x, x, torch.zeros(2, 4), cu, cu)


def test_evict_refuses_what_it_would_overwrite_while_reading():
    F = 1 << 20   # an address: nothing is launched
    c = fa._PagedCache(**dict(K=F, V=F, dtype=0, num_pages=5, page_size=16, Hkv=2, d=64, page_stride=2048, head_stride=1024,
                              row_stride=64, k_scale=None, v_scale=None, page_table=F, B=3, max_pages=4, table_stride=4))
    go = lambda lens, out, W, Wo, ln: fa.lib().fa_paged_evict(ctypes.byref(c), lens, out, 2, 2, W, 128, 64, 32, 4, Wo, 64, 32, 32,
                                                            F + 4096, ln, None)
    a = [F + 4096 * i for i in range(2, 7)]
    assert go(a[0], a[1], a[2], a[3], a[0]) == 1      # lens
    assert go(a[0], a[1], a[2], a[2], a[4]) == 1      # weights
    assert go(a[0], F, a[2], a[3], a[4]) == 1         # the table


def test_paged_calls_refuse_outputs_whose_rows_lie_on_top_of_each_other():
    F = 1 << 20
    base = dict(K=F, V=F, dtype=0, num_pages=5, page_size=16, Hkv=2, d=64, page_stride=2048, head_stride=1024, row_stride=64,
                k_scale=None, v_scale=None, page_table=F, B=3, max_pages=4, table_stride=4)
    r = fa._Rows(data=F, row_stride=128, head_stride=64)
    lib, ref_of = fa.lib(), ctypes.byref
    for bad in (dict(page_stride=0), dict(head_stride=0), dict(row_stride=0)):
        c = fa._PagedCache(**{**base, **bad})
        assert lib.fa_paged_append(ref_of(c), ref_of(r), ref_of(r), F, F + 64, 5, None) == 1
        assert lib.fa_paged_evict(ref_of(c), F + 64, F + 128, 2, 2, F, 128, 64, 32, 4, F + 4096, 64, 32, 32, F, F + 256, None) == 1
    c = fa._PagedCache(**base)
    for wb, wh in ((0, 64), (128, 0)):
        assert lib.fa_paged_decode(ref_of(c), ref_of(r), 4, F, 0.1, F, wb, wh, 0, F, F, F, 1 << 40, None) == 1
        assert lib.fa_paged_evict(ref_of(c), F + 64, F + 128, 2, 2, F, 128, 64, 32, 4, F + 4096, wb, wh, 32, F, F + 256, None) == 1
