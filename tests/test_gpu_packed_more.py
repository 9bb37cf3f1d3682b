"""More of packed attention on the GPU: layouts, streams and graphs, values that
must not spread, starts that lie outside, many sequences, agreement with the
padded calls at length, and the way from a prompt through the cache to the next
token."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_65_b200 as fa
import packed_ref as ref
from helpers import has_gpu
from test_gpu_packed import BF16, cu, i32, randn, within

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a B200")]


def batch(n, nk, Hq, Hkv, d, seed=0):
    t = [randn(sum(n), Hq, d, seed=seed), randn(sum(nk), Hkv, d, seed=seed + 1), randn(sum(nk), Hkv, d, seed=seed + 2),
         randn(sum(n), Hq, d, seed=seed + 3)]
    return [x.cuda() for x in t] + [i32(cu(n)), i32(cu(nk))]


def run(Q, K, V, dO, cq, ck, mask="causal", **kw):
    O, L = fa.fwd_packed(Q, K, V, cq, ck, mask=mask)
    return (O, L, *fa.bwd_packed(Q, K, V, O, dO, L, cq, ck, mask=mask, deterministic=True, **kw))


def equal(a, b):
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), i


@pytest.mark.parametrize("d", [64, 128])
def test_strided_rows_give_the_bits_of_contiguous_ones(d):
    n, Hq, Hkv = [70, 0, 200, 1], 6, 2
    Q, K, V, dO, c, _ = batch(n, n, Hq, Hkv, d)
    T = sum(n)
    want = run(Q, K, V, dO, c, c)
    # slices of a fused projection and its gradient; heads before rows; a wider row
    fused, grad = torch.cat([Q, K, V], 1), torch.zeros(T, Hq + 2 * Hkv, d, dtype=BF16, device="cuda")
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    got = run(q, k, v, dO, c, c, dQ=grad[:, :Hq], dK=grad[:, Hq:Hq + Hkv], dV=grad[:, Hq + Hkv:])
    equal(got, want)
    heads_first = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((T, Hkv, d + 24), math.nan, dtype=BF16, device="cuda")
    wide[..., 8:8 + d] = V
    equal(run(heads_first(Q), heads_first(K), wide[..., 8:8 + d], heads_first(dO), c, c), want)
    O2 = torch.zeros(Hq, T, d, dtype=BF16, device="cuda").transpose(0, 1)
    fa.fwd_packed(Q, K, V, c, c, mask="causal", O=O2)
    assert torch.equal(O2, want[0])


@pytest.mark.parametrize("more", [0, 5000], ids=["whole", "divided"])
def test_streams_and_graphs(more):
    n = [130, 40]
    Q, K, V, dO, cq, ck = batch(n, [x + more for x in n], 8, 2, 64, seed=5)
    want = run(Q, K, V, dO, cq, ck)
    torch.cuda.synchronize()
    # two streams at once, each with buffers of its own
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = []
    for r in range(4):
        for s in streams:
            O, L = fa.fwd_packed(Q, K, V, cq, ck, mask="causal", stream=s)
            both.append((s, O, L))
    with torch.cuda.stream(streams[0]):
        grads = run(Q, K, V, dO, cq, ck)
    torch.cuda.synchronize()
    for _, O, L in both:
        equal((O, L), want[:2])
    equal(grads, want)
    # a graph, replayed on new inputs while other launches run
    st = [t.clone() for t in (Q, K, V, dO)]
    bufs = [torch.empty_like(t) for t in want]
    wf = torch.empty(max(1, fa.fwd_packed_workspace_size(2, 170, 8, 2, 64)), dtype=torch.uint8, device="cuda")
    wb = torch.empty(fa.bwd_packed_workspace_size(2, 170, K.shape[0], 8, 2, 64), dtype=torch.uint8, device="cuda")

    def step():
        fa.fwd_packed(*st[:3], cq, ck, mask="causal", O=bufs[0], LSE=bufs[1], workspace=wf)
        fa.bwd_packed(*st[:3], bufs[0], st[3], bufs[1], cq, ck, mask="causal", dQ=bufs[2], dK=bufs[3], dV=bufs[4],
                      workspace=wb, deterministic=True)

    with torch.cuda.stream(streams[0]):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for r in range(3):
        for i, t in enumerate(st):
            t.copy_(randn(*t.shape, seed=20 + 4 * r + i))
        for t in (wf, wb, *bufs):
            t.fill_(1)
        g.replay()
        for _ in range(5):
            fa.fwd_packed(Q, K, V, cq, ck, mask="causal", stream=streams[1])
        torch.cuda.synchronize()
        equal(bufs, run(*st, cq, ck))
    assert fa.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("more", [0, 4000], ids=["whole", "divided"])
def test_values_that_are_not_seen_do_not_spread(d, more):
    n, Hq, Hkv = [150, 90], 4, 2
    nk = [x + more for x in n]
    Q, K, V, dO, cq, ck = batch(n, nk, Hq, Hkv, d, seed=9)
    O, L = fa.fwd_packed(Q, K, V, cq, ck, mask="causal")
    for t, bad in ((K, math.nan), (V, math.inf), (Q, math.nan)):
        x = t.clone()
        x[-60 if t is not Q else -30, 0] = bad  # the second sequence, head 0
        args = [x if t is y else y for y in (Q, K, V)]
        O2, L2 = fa.fwd_packed(*args, cq, ck, mask="causal")
        same = torch.ones(sum(n), Hq, dtype=torch.bool)
        if t is Q:
            same[-30, 0] = False
            assert torch.isnan(O2[-30, 0]).all() and torch.isnan(L2[0, -30])
        else:
            same[150:, :2] = False  # the rows of its two query heads ...
            if t is K:
                # ... are NaN from the row that sees it, and as they were before
                assert torch.isnan(O2[-60:, :2]).all() and torch.isnan(L2[:2, -60:]).all()
                assert torch.equal(L2[:2, 150:-60], L[:2, 150:-60])
            else:
                assert not torch.isfinite(O2[-60:, :2]).any() and torch.equal(L2, L)
        assert torch.equal(O2[same], O[same])
        G = fa.bwd_packed(*args, O, dO, L, cq, ck, mask="causal")
        for g, rows in zip(G, (150, nk[0], nk[0])):
            assert torch.isfinite(g[:rows]).all()       # the first sequence
            assert torch.isfinite(g[:, -1]).all()       # and another head
    # an infinite score below all others, and above: -inf leaves the row's other keys
    k = K.clone()
    k[7, 0] = -torch.sign(Q[20, 0].float()).to(BF16) * 3e38
    O2, L2 = fa.fwd_packed(Q, k, V, cq, ck, mask="causal")
    keep = [j for j in range(21 + more) if j != 7]
    s = (Q[20, 0].double() @ K[keep, 0].double().T) * d ** -0.5
    assert abs(float(L2[0, 20]) - float(torch.logsumexp(s, 0))) < 1e-3
    assert torch.isfinite(O2[20, 0]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_that_is_seen_reaches_the_gradients(d):
    n = [150, 90]
    Q, K, V, dO, c, _ = batch(n, n, 4, 2, d, seed=12)
    K[200, 1, 5] = math.nan  # row 50 of the second sequence, key head 1: seen by its queries from 50 on
    O, L = fa.fwd_packed(Q, K, V, c, c, mask="causal")
    assert torch.isnan(L[2:, 200:]).all() and torch.isfinite(L[:, :200]).all() and torch.isfinite(L[:2]).all()
    dQ, dK, dV = fa.bwd_packed(Q, K, V, O, dO, L, c, c, mask="causal")
    assert torch.isnan(dQ[200:, 2:]).all() and torch.isnan(dV[150:, 1]).all() and torch.isnan(dK[150:, 1]).all()
    for g in (dQ[:150], dQ[:, :2], dK[:150], dK[:, 0], dV[:150], dV[:, 0]):
        assert torch.isfinite(g).all()


def test_starts_outside_the_tensors_are_held_to_them():
    Q, K, V, dO, _, _ = batch([300], [300], 4, 2, 64, seed=3)
    ok = run(Q, K, V, dO, i32([0, 100, 300]), i32([0, 100, 300]))
    wild = run(Q, K, V, dO, i32([-2 ** 31, 100, 2 ** 31 - 1]), i32([-5, 100, 301]))
    equal(ok, wild)
    for bad in ([200, 100, 300], [0, 300, 0], [2 ** 31 - 1, 0, -1], [300, 300, 300]):
        out = run(Q, K, V, dO, i32(bad), i32(bad[::-1]))
        assert len(out) == 5
    assert fa.device_status() == 0


def test_many_sequences():
    g = torch.Generator().manual_seed(0)
    n = torch.randint(0, 40, (1500,), generator=g).tolist()
    n[700], n[31], n[32] = 600, 0, 257
    more = torch.randint(0, 30, (1500,), generator=g).tolist()
    nk = [a + b for a, b in zip(n, more)]
    Q, K, V, dO, cq, ck = batch(n, nk, 4, 2, 64, seed=2)
    O, L, dQ, dK, dV = run(Q, K, V, dO, cq, ck)
    assert fa.device_status() == 0
    a, b = cu(n), cu(nk)
    for s in (0, 1, 30, 31, 32, 33, 699, 700, 701, 1000, 1498, 1499):
        q, k = slice(a[s], a[s + 1]), slice(b[s], b[s + 1])
        x = [t.cpu() for t in (Q[q], K[k], V[k], O[q], dO[q], L[:, q])]
        wO, wL, tO, tL = ref.fwd(*x[:3], [0, n[s]], [0, nk[s]], True, 0.125)
        within(O[q], wO, tO, f"sequence {s} O")
        within(L[:, q], wL, tL, f"sequence {s} LSE")
        for got, (w, t), name in zip((dQ[q], dK[k], dV[k]), ref.bwd(*x, [0, n[s]], [0, nk[s]], True, 0.125), ("dQ", "dK", "dV")):
            within(got, w, t, f"sequence {s} {name}")
    assert torch.isfinite(O).all() and all(torch.isfinite(t).all() for t in (dQ, dK, dV))


@pytest.mark.parametrize("d", [64, 128])
def test_long_sequences_agree_with_the_padded_calls(d):
    B, H, N = 2, 4, 5000
    q, k, v, do = (randn(B, H, N, d, seed=i).cuda() for i in range(4))
    pack = lambda t: t.transpose(1, 2).reshape(B * N, H, d).contiguous()
    unpack = lambda t: t.view(B, N, H, d).transpose(1, 2).double()
    c = i32([0, N, 2 * N])
    O, L = fa.fwd(q, k, v, mask="causal")
    o, l = fa.fwd_packed(pack(q), pack(k), pack(v), c, c, mask="causal")
    # each is within (2^-8 + small) sum P |v| + 2^-8 |O| of the exact value
    A = fa.fwd(q, k, v.abs(), mask="causal")[0].double() * 1.01
    assert ((unpack(o) - O.double()).abs() <= 2 * (1.02 * (2.0 ** -8 + 2.0 ** -12) * A + 2.0 ** -8 * O.double().abs())).all()
    assert (l.view(H, B, N).transpose(0, 1) - L).abs().max() < 2e-4  # (5000 + 64) 2^-23 and less, each
    for got, want in zip(fa.bwd_packed(pack(q), pack(k), pack(v), pack(O), pack(do), L.transpose(0, 1).reshape(H, B * N).contiguous(),
                                       c, c, mask="causal"), fa.bwd(q, k, v, O, do, L, mask="causal")):
        got, want = unpack(got), want.double()
        # roundings to bf16 of independent terms: 2 2^-8 of the whole, in the mean square, with room
        assert float((got - want).norm() / want.norm()) < 2.0 ** -7


@pytest.mark.parametrize("d", [64, 128])
def test_from_a_prompt_through_the_cache_to_the_next_token(d):
    # the prompts' attention, their keys and values into the cache, the next
    # token against it; the same token as the last row of a packed prompt
    n, Hq, Hkv, page = [100, 1, 257], 8, 2, 16
    B, W = len(n), 18
    one = [x + 1 for x in n]
    Q, K, V, _, _, c1 = batch(one, one, Hq, Hkv, d, seed=40)
    a = cu(one)
    first = torch.tensor([t for b in range(B) for t in range(a[b], a[b + 1] - 1)], device="cuda")
    last = torch.tensor([a[b + 1] - 1 for b in range(B)], device="cuda")
    full, Lfull = fa.fwd_packed(Q, K, V, c1, c1, mask="causal")
    O, L = fa.fwd_packed(Q[first], K[first], V[first], i32(cu(n)), i32(cu(n)), mask="causal")
    kc, vc = (torch.full((B * W, Hkv, page, d), math.nan, dtype=BF16, device="cuda") for _ in range(2))
    table = torch.randperm(B * W, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, W).cuda()
    fa.paged_append(K[first], V[first], i32(cu(n)), i32([0] * B), kc, vc, table)
    fa.paged_append(K[last], V[last], i32(list(range(B + 1))), i32(n), kc, vc, table)
    Od, Ld = fa.paged_decode(Q[last], kc, vc, table, i32(one))
    # and as a chunk of one query a sequence against all its keys
    Oc, Lc = fa.fwd_packed(Q[last], K, V, i32(list(range(B + 1))), c1, mask="causal")
    assert fa.device_status() == 0
    wO, wL, tO, tL = ref.fwd(Q.cpu(), K.cpu(), V.cpu(), a, a, True, float(np.float32(d ** -0.5)))
    f, e = first.cpu(), last.cpu()
    for got, gl, rows, what in ((full, Lfull, slice(None), "all"), (O, L, f, "prompt"), (Od, Ld.t(), e, "token"), (Oc, Lc, e, "chunk")):
        within(got, wO[rows], tO[rows], what + " O")
        within(gl, wL[:, rows], tL[:, rows], what + " LSE")
