"""The packed backward where a key head's query heads are divided into more than one
part and fewer than there are heads, some parts a head more than others, against the
64-bit form."""
import numpy as np
import pytest
import torch

import exact_io_aware_65_b200 as fa
import packed_ref as ref
from helpers import has_gpu
from test_gpu_packed import BF16, cu, i32, poisoned, within

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a B200")]


def parts(B, Tq, Tk, Hq, Hkv, d):
    """Read from the workspace: each part of a call that has several holds fp32 dK and dV."""
    more = fa.bwd_packed_workspace_size(B, Tq, Tk, Hq, Hkv, d) - fa.bwd_packed_workspace_size(B, Tq, Tk, Hq, Hq, d)
    return round(more / (2 * Tk * Hkv * d * 4)) or 1


CASES = [
    # query lengths, keys before each sequence's queries, Hq, Hkv, d
    ([200, 143, 300, 257, 100], [0] * 5, 21, 3, 64),
    ([400, 500, 350, 450, 300], [0] * 5, 12, 4, 64),
    ([200, 150, 250, 1, 399], [0, 64, 0, 7, 1], 17, 1, 64),
    ([400, 300, 500, 130, 670], [0] * 5, 10, 2, 128),
    ([200, 201], [0, 0], 40, 8, 128),
    ([700], [0], 34, 2, 128),
]


@pytest.mark.parametrize("mask", ["causal", "none"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}seq-{c[2]}over{c[3]}x{c[4]}")
def test_uneven_parts_of_a_group(case, mask):
    n, more, Hq, Hkv, d = case
    nk = [a + b for a, b in zip(n, more)]
    x, cq, ck = poisoned(n, nk, Hq, Hkv, d, seed=len(n) + d + Hq, front=2, back=3)
    Tq, Tk, G = x["Q"].shape[0], x["K"].shape[0], Hq // Hkv
    p = parts(len(n), Tq, Tk, Hq, Hkv, d)
    assert 1 < p < G and G % p != 0, p
    scale, causal = float(np.float32(d ** -0.5)), mask == "causal"
    g = {k: v.cuda() for k, v in x.items()}
    O, L = fa.fwd_packed(g["Q"], g["K"], g["V"], i32(cq), i32(ck), mask=mask, scale=scale)
    grads = [torch.full(t.shape, 7.0, dtype=BF16, device="cuda") for t in (g["Q"], g["K"], g["V"])]
    q, k = slice(cq[0], cq[-1]), slice(ck[0], ck[-1])
    want = ref.bwd(x["Q"], x["K"], x["V"], O.cpu(), x["dO"], L.cpu(), cq, ck, causal, scale)
    first = None
    for det in (False, True):
        ws = torch.full((fa.bwd_packed_workspace_size(len(n), Tq, Tk, Hq, Hkv, d),), 255, dtype=torch.uint8, device="cuda")
        fa.bwd_packed(g["Q"], g["K"], g["V"], O, g["dO"], L, i32(cq), i32(ck), mask=mask, scale=scale, dQ=grads[0],
                      dK=grads[1], dV=grads[2], deterministic=det, workspace=ws)
        assert fa.device_status() == 0
        for t, (w, tol), rows, name in zip(grads, want, (q, k, k), ("dQ", "dK", "dV")):
            within(t[rows], w[rows], tol[rows], name)
            assert (t[:rows.start] == 7).all() and (t[rows.stop:] == 7).all(), name
        if first is None:
            first = [t.clone() for t in grads[1:]]
        assert all(torch.equal(a, b) for a, b in zip(first, grads[1:]))  # dK, dV: the same bits
        for t, rows in zip(grads, (q, k, k)):
            t[rows] = 7.0
