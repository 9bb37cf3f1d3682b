"""The paged cache on the GPU: append, decode and evict against the 64-bit
forms and bounds of paged_ref.py, at the sizes and masks where they can go
wrong, and the three together as a serving loop uses them."""
import numpy as np
import pytest
import torch

import exact_io_aware_65_b200 as fa
import paged_ref as ref
from helpers import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a B200")]

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def randn(*shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16)


def within(got, want, tol, what):
    got, want = got.detach().cpu().to(torch.float64), want
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin) and torch.equal(got[~fin], want[~fin]), f"{what}: non-finite entries differ"
    off = (got - want).abs()[fin] - tol[fin]
    assert off.numel() == 0 or float(off.max()) <= 0, f"{what}: {float(off.max()):.3e} past its bound"


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


# ------------------------------------------------------------------ append ---
APPEND = [
    # new rows and rows held, per sequence; Hkv, d, page
    ([1], [0], 1, 64, 16),
    ([1] * 33, list(range(33)), 8, 128, 16),
    ([5, 0, 130, 1, 17], [3, 9, 0, 63, 16], 3, 64, 24),
    ([0, 0, 4, 0], [1, 2, 3, 4], 2, 128, 1),
    ([700, 1], [0, 1000], 5, 128, 128),
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["heads", "rows"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{len(c[0])}x{c[2]}x{c[3]}-page{c[4]}")
def test_append_writes_its_rows_and_nothing_else(case, layout, e4m3):
    n, held, Hkv, d, page = case
    c = ref.make_cache([a + b for a, b in zip(n, held)], Hkv, d, page, e4m3, seed=1, layout=layout)
    T = sum(n)
    # new rows as slices of a fused projection, with two rows behind the last sequence
    fused = (3.0 * torch.randn(T + 2, 2 * Hkv + 1, d, generator=torch.Generator().manual_seed(2))).to(BF16)
    fused[0, 0, :4] = torch.tensor([1e4, -1e4, 0.0, -0.0])
    K, V = fused[:, :Hkv], fused[:, Hkv:2 * Hkv]
    cu = torch.tensor([0] + np.cumsum(n).tolist(), dtype=torch.int32)
    want = [c["kc"].clone(), c["vc"].clone()]
    for pool, x, s in zip(want, (K, V), (c["ks"], c["vs"])):
        x = x if s is None else (x.float() / s[:, None]).clamp(-448, 448).to(E4M3)
        for b in range(len(n)):
            for i in range(n[b]):
                p = held[b] + i
                pool[int(c["table"][b, p // page]), :, p % page] = x[int(cu[b]) + i]
    g = ref.dev(c)
    f = fused.cuda()
    fa.paged_append(f[:, :Hkv], f[:, Hkv:2 * Hkv], cu.cuda(), torch.tensor(held, dtype=torch.int32).cuda(), g["kc"], g["vc"],
                    g["table"], k_scale=g["ks"], v_scale=g["vs"])
    assert fa.device_status() == 0
    for got, w, name in ((g["kc"], want[0], "K"), (g["vc"], want[1], "V")):
        # (the NaN that stand behind the sequences must keep their bits too)
        assert torch.equal(bits(got.cpu().contiguous()), bits(w.contiguous())), name


def test_append_of_nothing_and_bad_pages():
    c = ref.dev(ref.make_cache([20, 20], 2, 64, 8, seed=3, poison=False))
    before = c["kc"].clone()
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    empty = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    fa.paged_append(empty, empty, cu, c["lens"], c["kc"], c["vc"], c["table"])
    x = randn(4, 2, 64, seed=4).cuda()
    held = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for bad in (-1, c["kc"].shape[0], 2 ** 31 - 1, -2 ** 31):
        t = c["table"].clone()
        t[0, 0] = bad
        k = before.clone()
        fa.paged_append(x, x, cu, held, k, c["vc"], t)
        assert fa.device_status() == 6
        page, slot = int(t[1, 2]), 0
        assert torch.equal(k[page, :, slot], x[2])          # the other sequence's rows arrive
        k[page, :, :2] = before[page, :, :2]
        assert torch.equal(k, before)                        # and the bad page's go nowhere
    # positions past the table's width, and a negative count of rows held
    for n in (24, 2 ** 31 - 2, -1):
        k = before.clone()
        fa.paged_append(x, x, cu, torch.tensor([n, n], dtype=torch.int32, device="cuda"), k, c["vc"], c["table"])
        assert fa.device_status() == 6 and torch.equal(k, before)
    assert fa.device_status() == 0


# ------------------------------------------------------------------ decode ---
DECODE = [
    # lens, Hq, Hkv, d, page
    ([1], 1, 1, 64, 16),
    ([1, 0, 2, 15, 16, 17, 127, 128, 129, 0], 8, 2, 128, 16),
    ([777], 32, 8, 128, 16),
    ([0, 0, 0], 4, 4, 64, 8),
    ([300, 5, 1000, 64], 12, 12, 64, 24),
    ([33, 400], 9, 3, 128, 1),
    ([513, 1, 90], 16, 1, 64, 128),
    ([200, 31], 34, 2, 128, 7),          # 17 heads a group: two units of the kernel
    ([100, 260], 40, 1, 64, 64),         # 40 heads a group: three
    ([20011], 8, 1, 128, 32),            # one sequence over every SM
    ([5000, 1, 0, 3300, 4999, 2], 10, 2, 64, 16),
]
IDS = [f"{len(c[0])}seq-max{max(c[0])}-{c[1]}over{c[2]}x{c[3]}-page{c[4]}" for c in DECODE]


def run_decode(c, Q, scale, **kw):
    return fa.paged_decode(Q, c["kc"], c["vc"], c["table"], c["lens"], scale=scale, k_scale=c["ks"], v_scale=c["vs"], **kw)


def check_decode(want, O, L, W=None, base=None):
    for b, r in enumerate(want):
        within(O[b], r["O"], r["O_tol"], f"sequence {b} O")
        within(L[b], r["LSE"], r["LSE_tol"], f"sequence {b} LSE")
        if W is not None:
            n = r["W"].shape[1]
            add = 0.0 if base is None else base[b, :, :n].double()
            # (adding to what is there rounds once more)
            within(W[b, :, :n], r["W"] + add, r["W_tol"] + 2.0 ** -24 * (r["W"] + add), f"sequence {b} weights")


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", DECODE, ids=IDS)
def test_decode_matches_the_64_bit_form(case, e4m3):
    lens, Hq, Hkv, d, page = case
    c = ref.make_cache(lens, Hkv, d, page, e4m3, seed=len(lens) + d, layout="rows" if page % 2 else "heads")
    scale = float(np.float32(d ** -0.5))
    B = len(lens)
    fused = randn(B, Hq + 2, d, seed=5)  # the queries as a slice of a fused projection
    want = ref.decode(fused[:, :Hq], c["kc"], c["vc"], c["table"], lens, scale, c["ks"], c["vs"])
    g, Q = ref.dev(c), fused.cuda()[:, :Hq]
    cap = c["table"].shape[1] * page
    O, L = run_decode(g, Q, scale)
    base = torch.rand(B, Hkv, cap + 3, generator=torch.Generator().manual_seed(6))
    W, A = base.cuda(), base.cuda()
    O2, L2 = run_decode(g, Q, scale, weights=W)
    O3, L3 = run_decode(g, Q, scale, weights=A, accumulate=True)
    assert fa.device_status() == 0
    for x, y in ((O, O2), (O, O3), (L, L2), (L, L3)):
        assert torch.equal(bits(x), bits(y)), "the same call gives other bits"
    check_decode(want, O, L, W.cpu())
    check_decode(want, O, L, A.cpu(), base)
    for b, n in enumerate(lens):  # behind the sequence: as it was
        assert torch.equal(W[b, :, n:].cpu(), base[b, :, n:]) and torch.equal(A[b, :, n:].cpu(), base[b, :, n:])


def test_decode_with_large_scores_and_queries_of_any_magnitude():
    # scores that grow along the cache (the running maximum moves at every
    # block), queries far outside fp16's range against the 8-bit cache
    for e4m3 in (False, True):
        c = ref.make_cache([1500, 700], 2, 64, 16, e4m3, seed=8, poison=False)
        for b, n in enumerate((1500, 700)):
            for p in range(0, n, 5):
                row = c["kc"][int(c["table"][b, p // 16]), :, p % 16]
                row.copy_((row.float() * (1 + 6 * p / n)).clamp(-448, 448).to(row.dtype))
        for mag in (1.0, 2.0 ** 40, 2.0 ** -60):
            Q = (randn(2, 6, 64, seed=9).float() * mag).to(BF16)
            scale = float(np.float32(4.0 / mag))
            want = ref.decode(Q, c["kc"], c["vc"], c["table"], [1500, 700], scale, c["ks"], c["vs"])
            g = ref.dev(c)
            O, L = run_decode(g, Q.cuda(), scale)
            assert fa.device_status() == 0
            check_decode(want, O, L)


def test_decode_keeps_nan_where_it_is_seen():
    c = ref.make_cache([40, 50], 2, 64, 16, seed=10)
    c["vc"][int(c["table"][0, 1]), 1, 3, 7] = torch.nan    # sequence 0, head 1, position 19
    g = ref.dev(c)
    O, L = run_decode(g, randn(2, 4, 64, seed=11).cuda(), 0.125)
    bad = torch.isnan(O).cpu()
    assert bad[0, 2:, 7].all() and bad.sum() == 2 and torch.isfinite(L).all()
    c = ref.make_cache([40, 50], 2, 64, 16, True, seed=10)
    c["kc"][int(c["table"][1, 0]), 0, 3, 7] = torch.nan    # a NaN of the 8-bit type
    g = ref.dev(c)
    O, L = run_decode(g, randn(2, 4, 64, seed=11).cuda(), 0.125)
    assert torch.isnan(L).cpu().tolist() == [[False] * 4, [True, True, False, False]]
    assert torch.isnan(O[1, :2]).all() and torch.isfinite(O[0]).all() and torch.isfinite(O[1, 2:]).all()


def test_decode_of_a_large_batch_of_short_sequences():
    # more sequences than one launch takes (4096), some empty
    B, page, d = 4500, 16, 64
    lens = [(7 * b) % 23 for b in range(B)]
    c = ref.make_cache(lens, 1, d, page, seed=12)
    Q = randn(B, 2, d, seed=13)
    g = ref.dev(c)
    W = torch.zeros(B, 1, c["table"].shape[1] * page, device="cuda")
    O, L = run_decode(g, Q.cuda(), 0.125, weights=W)
    assert fa.device_status() == 0
    pick = [0, 1, 2, 23, 100, 4095, 4096, 4097, 4499]
    want = ref.decode(Q[pick], c["kc"], c["vc"], c["table"][pick], [lens[b] for b in pick], 0.125)
    check_decode(want, O[pick], L[pick], W[pick].cpu())
    n = torch.tensor(lens)
    assert torch.equal(torch.isinf(L[:, 0]).cpu(), n == 0) and torch.isfinite(O).all()
    # every sequence's weights sum to the number of its query heads, to 23 times 2^-20
    sums = W.sum((1, 2)).cpu()
    assert float((sums - 2.0 * (n > 0)).abs().max()) < 1e-4


def test_decode_with_bad_pages_and_lengths_ends_with_a_status():
    c = ref.dev(ref.make_cache([100, 100], 2, 64, 16, seed=14, poison=False))
    Q = randn(2, 4, 64, seed=15).cuda()
    O, L = run_decode(c, Q, 0.125)
    for bad in (-1, c["kc"].shape[0], 2 ** 31 - 1):
        t = c["table"].clone()
        t[1, 3] = bad
        O2, L2 = fa.paged_decode(Q, c["kc"], c["vc"], t, c["lens"], scale=0.125)
        assert fa.device_status() == 6
        assert torch.equal(O2[0], O[0]) and torch.isfinite(O2).all()
    # lengths are held to the table's width, and to zero
    over = torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32, device="cuda")
    t = c["table"].clone()
    t[t < 0] = 0
    O3, L3 = fa.paged_decode(Q, c["kc"], c["vc"], t, over, scale=0.125)
    full = torch.tensor([t.shape[1] * 16, 0], dtype=torch.int32, device="cuda")
    O4, L4 = fa.paged_decode(Q, c["kc"], c["vc"], t, full, scale=0.125)
    assert fa.device_status() == 0 and torch.equal(O3, O4) and torch.equal(L3, L4)
    assert not O3[1].any() and torch.isneginf(L3[1]).all()


def test_decode_into_buffers_on_another_stream():
    c = ref.dev(ref.make_cache([900, 30, 2000], 2, 128, 16, seed=16))
    Q = randn(3, 8, 128, seed=17).cuda()
    O, L = run_decode(c, Q, 0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    O2, L2 = run_decode(c, Q, 0.1, stream=side)
    O3, L3 = torch.empty_like(O), torch.empty_like(L)
    ws = torch.empty(fa.paged_decode_workspace_size(3, 8, 2, 128, c["table"].shape[1] * 16), dtype=torch.uint8, device="cuda")
    run_decode(c, Q, 0.1, stream=side, O=O3, LSE=L3, workspace=ws)
    side.synchronize()
    assert torch.equal(O, O2) and torch.equal(L, L2) and torch.equal(O, O3) and torch.equal(L, L3)


# ------------------------------------------------------------------- evict ---
EVICT = [
    # lens, budget, recent, Hkv, d, page
    ([1], 1, 0, 1, 64, 16),
    ([100, 0, 7, 8, 9, 1], 8, 3, 2, 64, 16),
    ([1000, 700], 250, 64, 4, 64, 16),
    ([500, 40], 64, 64, 3, 128, 24),     # only the recent rows stay
    ([500, 63], 64, 0, 2, 128, 7),       # only the weights decide
    ([3000, 2999, 100], 2999, 1, 1, 64, 64),
    ([90], 4000, 100, 2, 128, 32),       # a budget that nothing reaches
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"{len(c[0])}seq-max{max(c[0])}-keep{c[1]}-recent{c[2]}")
def test_evict_keeps_the_right_rows(case, e4m3):
    lens, budget, recent, Hkv, d, page = case
    B = len(lens)
    left = [min(n, budget) for n in lens]
    c = ref.make_cache(lens, Hkv, d, page, e4m3, seed=20, extra_pages=sum(-(-n // page) for n in left) + 2,
                       layout="rows" if page % 2 else "heads")
    cap = c["table"].shape[1] * page
    g = torch.Generator().manual_seed(21)
    w = torch.randn(B, Hkv, cap + 5, generator=g).mul(2).exp()
    w = torch.where(torch.rand(w.shape, generator=g) < 0.3, w.round(), w)   # ties, many of them zero
    w[0, 0, ::7] = -0.0
    w[-1, -1, ::5] = torch.nan
    w[0, -1, ::11] = -w[0, -1, ::11]
    w[-1, 0, 1::13] = torch.inf
    table_out = torch.full((B, max(1, -(-min(budget, cap) // page))), -1, dtype=torch.int32)
    free = list(c["free"])
    for b in range(B):
        for i in range(-(-left[b] // page)):
            table_out[b, i] = free.pop()
    dv = ref.dev(c)
    wo = torch.full((B, Hkv, min(budget, cap) + 9), 3.0, device="cuda")
    kept, n_out = fa.paged_evict(w.cuda(), dv["kc"], dv["vc"], dv["table"], dv["lens"], table_out.cuda(), budget, recent, wo)
    assert fa.device_status() == 0
    assert n_out.tolist() == left
    want = [c["kc"].clone(), c["vc"].clone()]
    for b in range(B):
        for h in range(Hkv):
            k = ref.evict(w[b, h].tolist(), lens[b], budget, recent)
            assert kept[b, h].tolist() == k + [-1] * (budget - len(k)), (b, h)
            got = wo[b, h].cpu()
            assert torch.equal(bits(got[:len(k)]), bits(w[b, h, k])) and not got[len(k):].any()
            for i, p in enumerate(k):
                for pool in want:
                    pool[int(table_out[b, i // page]), h, i % page] = pool[int(c["table"][b, p // page]), h, p % page]
    for got, x in ((dv["kc"], want[0]), (dv["vc"], want[1])):
        assert torch.equal(bits(got.cpu().contiguous()), bits(x.contiguous()))


def test_evict_selects_from_more_keys_than_fit_on_chip():
    n, budget, recent, page = 60000, 777, 30, 16
    c = ref.make_cache([n], 1, 64, page, seed=22, extra_pages=60, poison=False)
    g = torch.Generator().manual_seed(23)
    w = torch.randint(0, 300, (1, 1, c["table"].shape[1] * page), generator=g).float()  # 200 of each: ties at the border
    table_out = torch.tensor([c["free"][:-(-budget // page)]], dtype=torch.int32)
    dv = ref.dev(c)
    wo = torch.empty((1, 1, budget), device="cuda")
    kept, _ = fa.paged_evict(w.cuda(), dv["kc"], dv["vc"], dv["table"], dv["lens"], table_out.cuda(), budget, recent, wo)
    assert fa.device_status() == 0
    assert kept[0, 0].tolist() == ref.evict(w[0, 0].tolist(), n, budget, recent)


def test_evict_with_bad_pages_ends_with_a_status():
    c = ref.dev(ref.make_cache([50, 50], 2, 64, 16, seed=24, poison=False))
    w = torch.rand(2, 2, 64, device="cuda")
    wo = torch.empty(2, 2, 8, device="cuda")
    free = c["free"]
    before = c["kc"].clone()
    out = torch.tensor([[-1], [free[0]]], dtype=torch.int32, device="cuda")
    fa.paged_evict(w, c["kc"], c["vc"], c["table"], c["lens"], out, 8, 2, wo)
    assert fa.device_status() == 6
    changed = (c["kc"] != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [free[0]]
    src = c["table"].clone()
    src[0] = 2 ** 31 - 1
    out[0, 0] = free[1]
    fa.paged_evict(w, c["kc"], c["vc"], src, c["lens"], out, 8, 2, wo)
    assert fa.device_status() == 6 and torch.equal(c["kc"][free[1]], before[free[1]])


# ------------------------------------------------------- as they are used ---
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_serving_loop(e4m3):
    """Prompts into the cache, decoding steps that accumulate weights, an
    eviction, and steps on the smaller cache, against the 64-bit forms on the
    rows that the cache then holds."""
    Hq, Hkv, d, page, budget, recent = 8, 2, 64, 16, 48, 8
    lens = [100, 1, 61]
    B, W = 3, 8
    pages = 3 * W + 3 * 6
    dt = E4M3 if e4m3 else BF16
    kc, vc = (torch.full((pages, Hkv, page, d), torch.nan).to(dt).cuda() for _ in range(2))
    ks = vs = None
    if e4m3:
        ks, vs = torch.tensor([0.01, 0.02]).cuda(), torch.tensor([0.015, 0.01]).cuda()
    table = torch.randperm(3 * W, generator=torch.Generator().manual_seed(30)).to(torch.int32).view(3, W).cuda()
    scale = 0.125
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    acc = torch.zeros(B, Hkv, W * page, device="cuda")
    base = torch.zeros(B, Hkv, W * page)

    def step(new, tab, counts, seed):
        T = sum(new)
        K, V, Q = (randn(T, h, d, seed=seed + i).cuda() for i, h in enumerate((Hkv, Hkv, Hq)))
        cu = torch.tensor([0] + np.cumsum(new).tolist(), dtype=torch.int32).cuda()
        fa.paged_append(K, V, cu, counts, kc, vc, tab, k_scale=ks, v_scale=vs)
        return Q, counts + torch.tensor(new, dtype=torch.int32).cuda()

    def decode(Q, tab, counts, acc, base):
        O, L = fa.paged_decode(Q, kc, vc, tab, counts, scale=scale, k_scale=ks, v_scale=vs, weights=acc, accumulate=True)
        assert fa.device_status() == 0
        cpu = lambda t: None if t is None else t.cpu()
        want = ref.decode(Q.cpu(), kc.cpu(), vc.cpu(), tab.cpu(), counts.tolist(), scale, cpu(ks), cpu(vs))
        check_decode(want, O, L, acc.cpu(), base)
        return acc.cpu().clone()

    _, n = step(lens, table, n, 40)
    for s in range(4):
        Q, n = step([1] * B, table, n, 50 + 3 * s)
        base = decode(Q, table, n, acc, base)
    out = (3 * W + torch.arange(18, dtype=torch.int32)).view(3, 6).cuda()
    acc2 = torch.empty(B, Hkv, 6 * page, device="cuda")
    kept, n2 = fa.paged_evict(acc, kc, vc, table, n, out, budget, recent, acc2)
    assert fa.device_status() == 0 and n2.tolist() == [min(x + 4, budget) for x in lens]
    for b in range(B):
        for h in range(Hkv):
            k = ref.evict(base[b, h].tolist(), lens[b] + 4, budget, recent)
            assert kept[b, h, :len(k)].tolist() == k
    base = acc2.cpu().clone()
    for s in range(3):
        Q, n2 = step([1] * B, out, n2, 70 + 3 * s)
        base = decode(Q, out, n2, acc2, base)


def test_serving_step_in_a_graph():
    """Append, decode and evict captured once and replayed on new inputs."""
    c = ref.dev(ref.make_cache([200, 37], 2, 64, 16, seed=60, extra_pages=8, poison=False))
    B, Hq, Hkv, d = 2, 8, 2, 64
    cap = c["table"].shape[1] * 16
    held = torch.tensor([199, 36], dtype=torch.int32, device="cuda")
    cu = torch.arange(3, dtype=torch.int32, device="cuda")
    K, V, Q = (randn(B, h, d, seed=61 + i).cuda() for i, h in enumerate((Hkv, Hkv, Hq)))
    out = torch.tensor(c["free"][:4], dtype=torch.int32, device="cuda").view(2, 2)
    W, W2 = torch.zeros(B, Hkv, cap, device="cuda"), torch.zeros(B, Hkv, 32, device="cuda")
    O, L = torch.empty(B, Hq, d, dtype=BF16, device="cuda"), torch.empty(B, Hq, device="cuda")
    kept, n2 = torch.empty(B, Hkv, 20, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(fa.paged_decode_workspace_size(B, Hq, Hkv, d, cap, True), dtype=torch.uint8, device="cuda")

    def step():
        fa.paged_append(K, V, cu, held, c["kc"], c["vc"], c["table"])
        fa.paged_decode(Q, c["kc"], c["vc"], c["table"], c["lens"], weights=W, O=O, LSE=L, workspace=ws)
        fa.paged_evict(W, c["kc"], c["vc"], c["table"], c["lens"], out, 20, 5, W2, kept=kept, lens_out=n2)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (O, L, W, W2, kept, n2, c["kc"], c["vc"])
    for r in range(3):
        for i, t in enumerate((K, V, Q)):
            t.copy_(randn(*t.shape, seed=70 + 3 * r + i))
        graph.replay()
        got = [t.clone() for t in outs]
        ws.fill_(255)
        step()
        torch.cuda.synchronize()
        assert fa.device_status() == 0
        for a, b in zip(got, outs):
            assert torch.equal(a, b)
