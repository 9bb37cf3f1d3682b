"""Paged decode where every score of a head is -inf: the head sees its keys and gives
them nothing, so that O = 0, LSE = -inf and its share of the weights is zero, set or
added (eviction goes by the sums: a NaN there would stay)."""
import pytest
import torch

import exact_io_aware_65_b200 as fa
import paged_ref as ref
from helpers import has_gpu
from test_gpu_paged import bits, randn, run_decode

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a B200")]


@pytest.mark.parametrize("lens", [[40, 90], [3000, 2]], ids=["short", "long"])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_a_head_whose_scores_are_all_minus_infinity_draws_nothing(lens, e4m3):
    page, d, Hq, Hkv = 16, 64, 6, 2
    c = ref.make_cache(lens, Hkv, d, page, e4m3, seed=1)
    Q = randn(2, Hq, d, seed=2)
    # the queries of sequence 0 and key head 1: positive, over 8 bits near the type's largest
    Q[0, 3:] = Q[0, 3:].abs() + 1
    if e4m3:
        Q[0, 3:] = 3e38
        c["ks"][1] = 1.0
    base = torch.rand(2, Hkv, c["table"].shape[1] * page, generator=torch.Generator().manual_seed(3)).cuda()

    def run():
        W, A, g, Qd = base.clone(), base.clone(), ref.dev(c), Q.cuda()
        O, L = run_decode(g, Qd, 1.0, weights=W)
        O2, L2 = run_decode(g, Qd, 1.0, weights=A, accumulate=True)
        assert fa.device_status() == 0 and torch.equal(bits(O), bits(O2)) and torch.equal(bits(L), bits(L2))
        return O, L, W, A

    before = run()
    # its keys: every product -inf, in bf16 by the keys, over 8 bits by the scaled sum
    for p in range(lens[0]):
        c["kc"][int(c["table"][0, p // page]), 1, p % page] = -448.0 if e4m3 else -torch.inf
    O, L, W, A = run()
    n = lens[0]
    assert not O[0, 3:].any() and torch.isneginf(L[0, 3:]).all()
    assert not W[0, 1, :n].any() and torch.equal(A[0, 1, :n], base[0, 1, :n])
    # everything else as before
    for x, y in zip((O, L, W, A), before):
        x, y = x.clone(), y.clone()
        for t in (x, y):
            t[(0, slice(3, None)) if t.shape[1] == Hq else (0, 1, slice(0, n))] = 0
        assert torch.equal(bits(x), bits(y))
