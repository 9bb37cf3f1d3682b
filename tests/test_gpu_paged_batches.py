"""Paged decode of serving batches: more than 32 sequences of mixed lengths with units
divided between CTAs (the walk then starts from a prefix that the block sums), against the
64-bit form."""
import random

import numpy as np
import pytest
import torch

import exact_io_aware_65_b200 as fa
import paged_ref as ref
from helpers import has_gpu
from test_gpu_paged import bits, check_decode, randn, run_decode

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a B200")]


def mixed(B, most, seed):
    """Many short sequences, a few long ones, some empty, in no order."""
    r = random.Random(seed)
    n = [0, 1, most, 128, 129] + [r.choice([0, 1, r.randint(1, 60), r.randint(1, 60), r.randint(100, 400)]) for _ in range(B - 7)]
    n += [most - 77, 0]
    r.shuffle(n)
    return n


CASES = [
    # sequences, longest, Hq, Hkv, d, page
    (33, 5000, 4, 1, 64, 16),
    (64, 3000, 32, 8, 128, 64),
    (40, 2500, 24, 2, 128, 24),   # 12 heads a group: two tiles of eight
    (300, 4000, 6, 2, 64, 16),
    (300, 1500, 17, 1, 64, 128),  # two units a key head
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}seq-max{c[1]}-{c[2]}over{c[3]}x{c[4]}-page{c[5]}")
def test_decode_of_a_serving_batch(case, e4m3):
    B, most, Hq, Hkv, d, page = case
    lens = mixed(B, most, seed=B + d)
    c = ref.make_cache(lens, Hkv, d, page, e4m3, seed=B)
    cap = c["table"].shape[1] * page
    assert len(lens) == B > 32 and cap > 512
    scale = float(np.float32(d ** -0.5))
    Q = randn(B, Hq, d, seed=B + 1)
    want = ref.decode(Q, c["kc"], c["vc"], c["table"], lens, scale, c["ks"], c["vs"])
    g, Qd = ref.dev(c), Q.cuda()
    base = torch.rand(B, Hkv, cap, generator=torch.Generator().manual_seed(6))
    W, A = base.cuda(), base.cuda()
    O, L = run_decode(g, Qd, scale)
    O2, L2 = run_decode(g, Qd, scale, weights=W)
    O3, L3 = run_decode(g, Qd, scale, weights=A, accumulate=True)
    assert fa.device_status() == 0
    for x, y in ((O, O2), (O, O3), (L, L2), (L, L3)):
        assert torch.equal(bits(x), bits(y)), "the same call gives other bits"
    check_decode(want, O, L, W.cpu())
    check_decode(want, O, L, A.cpu(), base)
    behind = torch.arange(cap)[None] >= torch.tensor(lens)[:, None]
    for x in (W, A):
        assert torch.equal(x.cpu().transpose(1, 2)[behind], base.transpose(1, 2)[behind])


@pytest.mark.parametrize("B,Hkv,recent", [(21, 7, 40), (37, 4, 0), (20, 8, 300), (50, 6, 64)],
                         ids=["147 heads", "148 heads", "160 heads", "300 heads"])
def test_eviction_with_a_head_for_every_sm(B, Hkv, recent):
    # rows enough for a second kernel to move them
    budget, page, d = 300, 24, 128
    r = random.Random(B)
    lens = [0, 1, budget, budget + 1, 299] + [r.randint(1, 900) for _ in range(B - 5)]
    left = [min(n, budget) for n in lens]
    c = ref.make_cache(lens, Hkv, d, page, seed=B, extra_pages=sum(-(-n // page) for n in left) + 2, poison=False)
    w = torch.rand((B, Hkv, c["table"].shape[1] * page), generator=torch.Generator().manual_seed(7))
    w = (w * 50).floor() / 50  # many equal ones
    table_out = torch.full((B, -(-budget // page)), -1, dtype=torch.int32)
    free = list(c["free"])
    for b, n in enumerate(left):
        for i in range(-(-n // page)):
            table_out[b, i] = free.pop()
    dv = ref.dev(c)
    wo = torch.full((B, Hkv, budget + 5), 3.0, device="cuda")
    kept, n_out = fa.paged_evict(w.cuda(), dv["kc"], dv["vc"], dv["table"], dv["lens"], table_out.cuda(), budget, recent, wo)
    assert fa.device_status() == 0 and n_out.tolist() == left
    kept, wo = kept.cpu(), wo.cpu()
    want = [c["kc"].clone(), c["vc"].clone()]
    for b in range(B):
        for h in range(Hkv):
            k = ref.evict(w[b, h].tolist(), lens[b], budget, recent)
            assert kept[b, h].tolist() == k + [-1] * (budget - len(k)), (b, h)
            assert torch.equal(wo[b, h, :len(k)], w[b, h, k]) and not wo[b, h, len(k):].any()
            at, frm = torch.arange(len(k)), torch.tensor(k, dtype=torch.long)
            for pool in want:
                pool[table_out[b, at // page].long(), h, at % page] = pool[c["table"][b, frm // page].long(), h, frm % page]
    for got, x in ((dv["kc"], want[0]), (dv["vc"], want[1])):
        assert torch.equal(bits(got.cpu()), bits(x))
