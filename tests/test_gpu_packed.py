"""Packed attention with grouped heads on the GPU, forward and backward, against
the 64-bit forms and bounds of packed_ref.py, at the lengths, masks and layouts
where it can go wrong."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_65_b200 as fa
import packed_ref as ref
from helpers import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a B200")]

BF16 = torch.bfloat16


def cu(n, first=0):
    return [first] + (first + np.cumsum(n)).tolist()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(*shape, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(BF16)


def within(got, want, tol, what):
    got = got.detach().cpu().to(torch.float64)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin) and torch.equal(got[~fin], want[~fin]), f"{what}: non-finite entries differ"
    off = (got - want).abs()[fin] - tol[fin]
    assert off.numel() == 0 or float(off.max()) <= 0, f"{what}: {float(off.max()):.3e} past its bound"


def poisoned(n_q, n_k, Hq, Hkv, d, seed, front=0, back=0):
    """Q, K, V, dO with NaN and infinities in rows that belong to no sequence."""
    Tq, Tk = sum(n_q) + front + back, sum(n_k) + front + back
    x = dict(Q=randn(Tq, Hq, d, seed=seed), K=randn(Tk, Hkv, d, seed=seed + 1), V=randn(Tk, Hkv, d, seed=seed + 2),
             dO=randn(Tq, Hq, d, seed=seed + 3))
    for t in x.values():
        t[:front] = math.nan
        t[t.shape[0] - back:] = math.inf
    return x, cu(n_q, front), cu(n_k, front)


CASES = [
    # query lengths, keys before each sequence's queries (or None: as many keys as given), Hq, Hkv
    ([1], [0], 1, 1),
    ([1, 0, 2, 127, 128, 129, 0, 3], [0, 5, 0, 0, 0, 0, 0, 300], 4, 2),
    ([400], [0], 3, 1),
    ([5, 300, 64], [0, 100, 31], 8, 1),
    ([257, 1, 130], [500, 129, 0], 12, 12),
    ([33] * 40, [7] * 40, 2, 2),              # more sequences than a warp looks at
    ([260, 100], [-60, -100], 6, 2),          # fewer keys than queries: rows that see nothing, no keys at all
    ([0, 0], [17, 0], 4, 4),                  # nobody asks
    ([700], [700], 16, 1),
    ([640, 384, 512], [0, 0, 0], 10, 2),      # whole tiles
    ([1], [4999], 8, 2),                      # few query tiles, many keys: divided between work items
    ([200, 3, 0], [4000, 2500, 3000], 3, 1),  # (pairs of query tiles at d = 128)
    ([2300], [0], 4, 1),
    ([130, 1, 129, 2], [2100, 0, 6000, 1], 6, 2),  # (some sequences divided, some not)
]
IDS = [f"{len(c[0])}seq-max{max(c[0])}+{max(c[1])}-{c[2]}over{c[3]}" for c in CASES]


@pytest.mark.parametrize("mask", ["causal", "none"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_and_backward_match_the_64_bit_form(case, d, mask):
    n, more, Hq, Hkv = case
    nk = [a + b for a, b in zip(n, more)]
    x, cq, ck = poisoned(n, nk, Hq, Hkv, d, seed=len(n) + d, front=3, back=2)
    scale = float(np.float32(d ** -0.5))
    causal = mask == "causal"
    g = {k: v.cuda() for k, v in x.items()}
    Tq, Tk = g["Q"].shape[0], g["K"].shape[0]
    O = torch.full((Tq, Hq, d), 7.0, dtype=BF16, device="cuda")
    L = torch.full((Hq, Tq), 7.0, device="cuda")
    assert fa.fwd_packed(g["Q"], g["K"], g["V"], i32(cq), i32(ck), mask=mask, scale=scale, O=O, LSE=L)[0] is O
    assert fa.device_status() == 0
    wO, wL, tO, tL = ref.fwd(x["Q"], x["K"], x["V"], cq, ck, causal, scale)
    q, k = slice(cq[0], cq[-1]), slice(ck[0], ck[-1])
    within(O[q], wO[q], tO[q], "O")
    within(L[:, q], wL[:, q], tL[:, q], "LSE")
    for t in (O, L.t()):  # rows of no sequence: as they were
        assert (t[:cq[0]] == 7).all() and (t[cq[-1]:] == 7).all()
    grads = [torch.full(t.shape, 7.0, dtype=BF16, device="cuda") for t in (g["Q"], g["K"], g["V"])]
    for det in (False, True):
        fa.bwd_packed(g["Q"], g["K"], g["V"], O, g["dO"], L, i32(cq), i32(ck), mask=mask, scale=scale, dQ=grads[0],
                      dK=grads[1], dV=grads[2], deterministic=det)
        assert fa.device_status() == 0
        want = ref.bwd(x["Q"], x["K"], x["V"], O.cpu(), x["dO"], L.cpu(), cq, ck, causal, scale)
        for t, (w, tol), rows, name in zip(grads, want, (q, k, k), ("dQ", "dK", "dV")):
            within(t[rows], w[rows], tol[rows], name)
            assert (t[:rows.start] == 7).all() and (t[rows.stop:] == 7).all(), name
            t[rows] = 7.0
