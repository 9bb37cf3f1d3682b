"""The packed and paged calls through the native binding and through ctypes: the
same results, outputs into the caller's buffers, the same refusals, and nothing
taken that the Python checks would refuse."""
import math

import pytest
import torch

import exact_io_aware_65_b200 as fa
import paged_ref as ref
from helpers import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a B200")]


@pytest.fixture(params=["native", "ctypes"])
def path(request, monkeypatch):
    fa.lib()
    if request.param == "native":
        assert fa._fast is not None, "_binding.so is missing"
    else:
        monkeypatch.setattr(fa, "_fast", None)
    return request.param


@pytest.fixture
def only_native(monkeypatch):
    """The Python paths fail: what passes was taken natively."""
    fa.lib()

    def never(*a, **k):
        raise AssertionError("went through Python")

    for name in ("_rows", "_paged_cache"):
        monkeypatch.setattr(fa, name, never)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


def packed():
    x = randn(90, 10, 64)  # a fused projection: 6 query, 2 key and 2 value heads
    return x[:, :6], x[:, 6:8], x[:, 8:], i32([0, 40, 90])


def test_every_call_is_taken_natively(only_native):
    Q, K, V, cu = packed()
    O, L = fa.fwd_packed(Q, K, V, cu, cu, mask="causal")
    fa.bwd_packed(Q, K, V, O, randn(90, 6, 64, seed=1), L, cu, cu, mask="causal", deterministic=True)
    c = ref.dev(ref.make_cache([30, 20], 2, 64, 16, seed=3, extra_pages=4, poison=False))
    fa.paged_append(K[:2], V[:2], i32([0, 1, 2]), i32([29, 19]), c["kc"], c["vc"], c["table"])
    w = torch.zeros(2, 2, 32, device="cuda")
    fa.paged_decode(Q[:2], c["kc"], c["vc"], c["table"], c["lens"], weights=w, accumulate=True)
    out = i32([[c["free"][0]], [c["free"][1]]])
    fa.paged_evict(w, c["kc"], c["vc"], c["table"], c["lens"], out, 8, 2, torch.zeros(2, 2, 8, device="cuda"))
    assert fa.device_status() == 0


def test_both_paths_give_the_same(path, monkeypatch):
    Q, K, V, cu = packed()
    dO = randn(90, 6, 64, seed=1)
    O, L = fa.fwd_packed(Q, K, V, cu, cu, mask="causal")
    G = fa.bwd_packed(Q, K, V, O, dO, L, cu, cu, mask="causal", deterministic=True)
    # into buffers of the caller: slices of a fused gradient
    o, l = torch.empty_like(O), torch.empty_like(L)
    assert fa.fwd_packed(Q, K, V, cu, cu, mask=1, scale=0.125, O=o, LSE=l)[0] is o
    fused = torch.zeros(90, 10, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(fa.bwd_packed_workspace_size(2, 90, 90, 6, 2, 64), dtype=torch.uint8, device="cuda")
    fa.bwd_packed(Q, K, V, O, dO, L, cu, cu, mask="causal", scale=64 ** -0.5, dQ=fused[:, :6], dK=fused[:, 6:8],
                  dV=fused[:, 8:], workspace=ws, deterministic=True)
    assert torch.equal(o, O) and torch.equal(l, L) and torch.equal(fused, torch.cat(G, 1))
    monkeypatch.setattr(fa, "_fast", None)
    O2, L2 = fa.fwd_packed(Q, K, V, cu, cu, mask="causal")
    assert torch.equal(O, O2) and torch.equal(L, L2)
    for a, b in zip(G, fa.bwd_packed(Q, K, V, O, dO, L, cu, cu, mask="causal", deterministic=True)):
        assert torch.equal(a, b)


def test_refusals_are_the_same(path):
    Q, K, V, cu = packed()
    O, L = fa.fwd_packed(Q, K, V, cu, cu)
    c = ref.dev(ref.make_cache([30, 20], 2, 64, 16, seed=3, poison=False))
    kc, vc, t, n = c["kc"], c["vc"], c["table"], c["lens"]
    w = torch.zeros(2, 2, 32, device="cuda")
    q = Q[:2]
    bad = [
        lambda: fa.fwd_packed(Q.float(), K, V, cu, cu), lambda: fa.fwd_packed(Q.cpu(), K, V, cu, cu),
        lambda: fa.fwd_packed(Q[:, :5], K, V, cu, cu), lambda: fa.fwd_packed(Q, K, V[:80], cu, cu),
        lambda: fa.fwd_packed(Q, K[..., :32], V, cu, cu), lambda: fa.fwd_packed(Q, K, V, cu.long(), cu),
        lambda: fa.fwd_packed(Q, K, V, cu, cu[:2]), lambda: fa.fwd_packed(Q, K, V, cu[:1], cu[:1]),
        lambda: fa.fwd_packed(Q, K, V, cu, cu, scale=0.0), lambda: fa.fwd_packed(Q, K, V, cu, cu, scale=math.nan),
        lambda: fa.fwd_packed(Q, K, V, cu, cu, mask="block"), lambda: fa.fwd_packed(Q, K, V, cu, cu, mask=7),
        lambda: fa.fwd_packed(Q, K, V, cu, cu, O=O[:80]), lambda: fa.fwd_packed(Q, K, V, cu, cu, LSE=L.t()),
        lambda: fa.fwd_packed(Q[:, :1].expand(90, 6, 64), K, V, cu, cu), lambda: fa.fwd_packed(None, K, V, cu, cu),
        lambda: fa.fwd_packed(Q.transpose(1, 2), K, V, cu, cu), lambda: fa.fwd_packed(Q[1:, :, 4:], K, V, cu, cu),
        lambda: fa.bwd_packed(Q, K, V, O, O[:, :2], L, cu, cu), lambda: fa.bwd_packed(Q, K, V, O, O, L.t(), cu, cu),
        lambda: fa.bwd_packed(Q, K, V, O, O, L, cu, cu, workspace=w), lambda: fa.bwd_packed(Q, K, V, O, O, L, cu, cu, dK=O),
        lambda: fa.bwd_packed(Q, K, V, O, O.sum().expand_as(O), L, cu, cu),
        lambda: fa.paged_append(K[:2], V[:1], i32([0, 1, 2]), n, kc, vc, t), lambda: fa.paged_append(K[:2], V[:2], n, n, kc, vc, t),
        lambda: fa.paged_append(K[:2], V[:2], i32([0, 1, 2]), n, kc, vc.float(), t),
        lambda: fa.paged_append(K[:2], V[:2], i32([0, 1, 2]), n, kc, vc, t, k_scale=w[0, 0, :2]),
        lambda: fa.paged_decode(Q[:3], kc, vc, t, n), lambda: fa.paged_decode(Q[:2, :5], kc, vc, t, n),
        lambda: fa.paged_decode(q, kc, vc, t.long(), n), lambda: fa.paged_decode(q, kc, vc, t, n, weights=w[..., :31]),
        lambda: fa.paged_decode(q, kc, vc, t, n, weights=w.half()), lambda: fa.paged_decode(q, kc, vc, t, n, scale=-1.0),
        lambda: fa.paged_decode(q, kc, vc, t, n, O=O), lambda: fa.paged_decode(q, kc, vc, t, n, workspace=n),
        lambda: fa.paged_decode(q, kc.to(torch.float8_e4m3fn), vc.to(torch.float8_e4m3fn), t, n),
        lambda: fa.paged_evict(w, kc, vc, t, n, t, 0, 0, w), lambda: fa.paged_evict(w, kc, vc, t, n, t, 8, 9, w),
        lambda: fa.paged_evict(w, kc, vc, t, n, t[:1], 8, 2, w), lambda: fa.paged_evict(w, kc, vc, t, n, t, 8, 2, w[..., :7]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(fa.FAError):
            f()
            raise AssertionError(f"call {i} was taken")
    assert fa.device_status() == 0
