"""Many work items without a visible tile, one after the other: short sequences
in wide padding, masks that keep next to nothing, and packed sequences that
bring only queries or only keys.  The kernels' roles must stay in step over
them, and what has nothing to see comes out as zeros."""
import pytest
import torch

import exact_io_aware_65_b200 as fa
from helpers import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a B200")]


@pytest.fixture(autouse=True)
def short_waits():
    fa.set_wait_timeout_ns(500_000_000)
    yield
    fa.set_wait_timeout_ns(0)


def randn(*shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("mask", ["causal", "none"])
@pytest.mark.parametrize("d", [64, 128])
def test_short_sequences_in_wide_padding(d, mask):
    B, H, N = 12, 8, 4096
    lens = torch.tensor([0, 0, 1, 0, 130, 0, 0, 4096, 0, 0, 2, 0], dtype=torch.int32, device="cuda")
    Q, K, V, dO = (randn(B, H, N, d) for _ in range(4))
    for rep in range(3):
        O, L = fa.fwd(Q, K, V, mask, seqlens_q=lens, seqlens_k=lens)
        grads = fa.bwd(Q, K, V, O, dO, L, mask, seqlens_q=lens, seqlens_k=lens)
        assert fa.device_status() == 0
    for b, n in enumerate(lens.tolist()):
        for t in (O, *grads):
            assert not t[b, :, n:].any() and torch.isfinite(t[b]).all()
        assert torch.isneginf(L[b, :, n:]).all() and torch.isfinite(L[b, :, :n]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_block_mask_that_keeps_one_tile(d):
    B, H, N = 2, 16, 4096
    m = torch.zeros(N // 128, N // 128, dtype=torch.uint8, device="cuda")
    m[20, 11] = 1
    Q, K, V, dO = (randn(B, H, N, d) for _ in range(4))
    O, L = fa.fwd(Q, K, V, "block", m)
    dQ, dK, dV = fa.bwd(Q, K, V, O, dO, L, "block", m)
    assert fa.device_status() == 0
    for t, at in ((O, 20), (dQ, 20), (dK, 11), (dV, 11)):
        assert t[:, :, 128 * at:128 * at + 128].any()
        t[:, :, 128 * at:128 * at + 128] = 0
        assert not t.any()


@pytest.mark.parametrize("d", [64, 128])
def test_packed_sequences_of_queries_or_keys_alone(d):
    B, Hq, Hkv = 200, 8, 4
    n = [300 if b % 2 else 0 for b in range(B)]
    k = [0 if b % 2 else 300 for b in range(B)]
    cu = lambda x: torch.tensor([0] + torch.tensor(x).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    Q, dO, K, V = randn(sum(n), Hq, d), randn(sum(n), Hq, d), randn(sum(k), Hkv, d), randn(sum(k), Hkv, d)
    for mask in ("causal", "none"):
        O, L = fa.fwd_packed(Q, K, V, cu(n), cu(k), mask=mask)
        grads = fa.bwd_packed(Q, K, V, O, dO, L, cu(n), cu(k), mask=mask)
        assert fa.device_status() == 0
        assert not O.any() and torch.isneginf(L).all() and not any(g.any() for g in grads)
