"""More of the paged calls on the GPU: every 16-bit value at many scales into an
8-bit cache, pages that lie further apart than 32 bits of 16-byte pieces reach,
and selections that the histograms' borders cut."""
import numpy as np
import pytest
import torch

import exact_io_aware_65_b200 as fa
import paged_ref as ref
from helpers import has_gpu
from test_gpu_paged import BF16, E4M3, bits, randn, within

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a B200")]


def test_append_rounds_every_value_as_the_division_does():
    # all 2^16 bf16 values (rows of 64), each head with a scale of its own: close
    # to powers of two, random, tiny, huge, negative, zero, infinite, NaN
    H = 96
    g = torch.Generator().manual_seed(1)
    s = torch.exp2(torch.empty(H).uniform_(-20, 20, generator=g))
    s[:12] = torch.tensor([1.0, 0.5, 1 - 2.0 ** -24, 1 + 2.0 ** -23, 3.0, 448.0, 2.0 ** -62, 2.0 ** 62, 1e-38, 3e38, 2.0 ** -149, 0.1])
    s[12:16] = torch.tensor([-0.7, 0.0, float("inf"), float("nan")])
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16).view(1024, 1, 64).expand(1024, H, 64).contiguous()
    kc = torch.zeros(64, H, 16, 64, device="cuda").to(E4M3)
    vc = kc.clone()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    xd, sd = x.cuda(), s.cuda()
    fa.paged_append(xd, xd, i32([0, 1024]), i32([0]), kc, vc, i32([list(range(64))]), k_scale=sd, v_scale=sd)
    assert fa.device_status() == 0
    q = x.float() / s[:, None]
    want = torch.where(torch.isnan(q), q, q.clamp(-448, 448)).to(E4M3).float()
    for pool in (kc, vc):
        got = pool.cpu().float().permute(0, 2, 1, 3).reshape(1024, H, 64)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fin = ~torch.isnan(want)
        assert torch.equal(got[fin], want[fin])


def test_decode_over_pages_more_than_2_to_the_36_bytes_apart():
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free device memory")
    page, d = 16, 64
    n_pages = (1 << 36) // (page * d * 2) + 100
    pool = torch.empty((n_pages, 1, page, d), dtype=BF16, device="cuda")  # K and V at once: only read
    lens, pages = [40, 70], [[n_pages - 1, 0, n_pages - 50, -1, -1], [5, n_pages - 2, n_pages // 2, n_pages - 90, 7]]
    small = randn(8, 1, page, d, seed=1)
    flat = [p for row in pages for p in row if p >= 0]
    for i, p in enumerate(flat):
        pool[p] = small[i].cuda()
    table = torch.tensor(pages, dtype=torch.int32)
    compact = torch.tensor([[flat.index(p) if p >= 0 else -1 for p in row] for row in pages], dtype=torch.int32)
    Q = randn(2, 2, d, seed=2)
    O, L = fa.paged_decode(Q.cuda(), pool, pool, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=0.125)
    assert fa.device_status() == 0
    for b, r in enumerate(ref.decode(Q, small, small, compact, lens, 0.125)):
        within(O[b], r["O"], r["O_tol"], f"sequence {b} O")
        within(L[b], r["LSE"], r["LSE_tol"], f"sequence {b} LSE")


@pytest.mark.parametrize("kind", ["equal", "two values", "last bits", "signs", "zeros", "one binade"])
def test_evict_where_keys_share_their_upper_bits(kind):
    n, budget, recent, page = 5000, 1234, 100, 16
    c = ref.make_cache([n, n - 7], 2, 64, page, seed=3, extra_pages=170, poison=False)
    g = torch.Generator().manual_seed(4)
    shape = (2, 2, c["table"].shape[1] * page)
    u = torch.rand(shape, generator=g)
    w = {"equal": torch.full(shape, 0.3), "two values": (u < 0.4).float(),
         "last bits": (torch.randint(0, 1200, shape, generator=g, dtype=torch.int32) + 0x3f800000).view(torch.float32),
         "signs": u - 0.5, "zeros": torch.where(u < 0.9, torch.where(u < 0.5, -0.0, 0.0), u), "one binade": 1 + u}[kind]
    out = torch.tensor([c["free"][:78], c["free"][78:156]], dtype=torch.int32)
    dv = ref.dev(c)
    wo = torch.empty((2, 2, budget), device="cuda")
    kept, left = fa.paged_evict(w.cuda(), dv["kc"], dv["vc"], dv["table"], dv["lens"], out.cuda(), budget, recent, wo)
    assert fa.device_status() == 0 and left.tolist() == [budget, budget]
    for b in range(2):
        for h in range(2):
            assert kept[b, h].tolist() == ref.evict(w[b, h].tolist(), n - 7 * b, budget, recent)


@pytest.mark.parametrize("recent", [0, 50, 600])
@pytest.mark.parametrize("d,e4m3", [(64, True), (64, False), (128, False)])
def test_evict_moves_last_rows_while_others_are_selected(d, e4m3, recent):
    # budgets that a second kernel moves, with SMs to spare: lengths of zero, one,
    # below, at and just above the budget, and past the rows that move early
    lens, budget, Hkv, page = [0, 1, 37, 1100, 1101, 1700, 4000], 1100, 3, 24
    left = [min(n, budget) for n in lens]
    c = ref.make_cache(lens, Hkv, d, page, e4m3, seed=31, extra_pages=sum(-(-n // page) for n in left) + 2)
    g = torch.Generator().manual_seed(32)
    w = torch.rand((len(lens), Hkv, c["table"].shape[1] * page), generator=g)
    table_out = torch.full((len(lens), -(-budget // page)), -1, dtype=torch.int32)
    free = list(c["free"])
    for b, n in enumerate(left):
        for i in range(-(-n // page)):
            table_out[b, i] = free.pop()
    dv = ref.dev(c)
    wo = torch.full((len(lens), Hkv, budget + 5), 3.0, device="cuda")
    kept, n_out = fa.paged_evict(w.cuda(), dv["kc"], dv["vc"], dv["table"], dv["lens"], table_out.cuda(), budget, recent, wo)
    assert fa.device_status() == 0 and n_out.tolist() == left
    want = [c["kc"].clone(), c["vc"].clone()]
    for b in range(len(lens)):
        for h in range(Hkv):
            k = ref.evict(w[b, h].tolist(), lens[b], budget, recent)
            assert kept[b, h].tolist() == k + [-1] * (budget - len(k)), (b, h)
            got = wo[b, h].cpu()
            assert torch.equal(got[:len(k)], w[b, h, k]) and not got[len(k):].any()
            at, frm = torch.arange(len(k)), torch.tensor(k, dtype=torch.long)
            for pool in want:
                pool[table_out[b, at // page].long(), h, at % page] = pool[c["table"][b, frm // page].long(), h, frm % page]
    for got, x in ((dv["kc"], want[0]), (dv["vc"], want[1])):
        assert torch.equal(bits(got.cpu().contiguous()), bits(x.contiguous()))


def test_decode_calls_at_once_and_many_after_another():
    # divided units on two streams and in a graph, each with buffers of its own;
    # then more calls than there are rows of counters
    c = ref.dev(ref.make_cache([5000, 700, 3100], 2, 128, 16, seed=7, poison=False))
    e = ref.dev(ref.make_cache([9000], 2, 64, 64, True, seed=8, poison=False))
    Q, R = randn(3, 8, 128, seed=9).cuda(), randn(1, 20, 64, seed=10).cuda()
    f = lambda **k: fa.paged_decode(Q, c["kc"], c["vc"], c["table"], c["lens"], **k)
    h = lambda **k: fa.paged_decode(R, e["kc"], e["vc"], e["table"], e["lens"], k_scale=e["ks"], v_scale=e["vs"], **k)
    want = [t.clone() for t in (*f(), *h())]
    bufs = [torch.empty_like(t) for t in want]
    ws = [torch.empty(fa.paged_decode_workspace_size(*a), dtype=torch.uint8, device="cuda")
          for a in ((3, 8, 2, 128, c["table"].shape[1] * 16), (1, 20, 2, 64, e["table"].shape[1] * 64))]

    def step():
        f(O=bufs[0], LSE=bufs[1], workspace=ws[0])
        h(O=bufs[2], LSE=bufs[3], workspace=ws[1])

    streams = [torch.cuda.Stream() for _ in range(3)]
    with torch.cuda.stream(streams[2]):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    got = []
    for _ in range(20):
        for t in (*bufs, *ws):
            t.fill_(1)
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[2]):
            graph.replay()
        for s in streams[:2]:
            got += [(f(stream=s), 0), (h(stream=s), 2)]
        torch.cuda.synchronize()
        for t, w in zip(bufs, want):
            assert torch.equal(t, w)
    for (O, L), i in got:
        assert torch.equal(O, want[i]) and torch.equal(L, want[i + 1])
    for _ in range(2200):
        O, L = h()
    assert torch.equal(O, want[2]) and torch.equal(L, want[3]) and fa.device_status() == 0
