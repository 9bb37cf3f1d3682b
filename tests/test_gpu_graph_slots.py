"""Forward launches in many graphs: a captured launch's work counter is its
graph's own, and comes back when the graph goes."""
import gc

import pytest
import torch

import exact_io_aware_65_b200 as fa
from helpers import has_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a B200")]


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


class Call:
    """A forward with buffers of its own, which every call must fill with the same bits."""

    def __init__(self, f, Q, K, V, lse):
        self.f, self.x, self.out = f, (Q, K, V), (torch.empty_like(Q), torch.empty(lse, device="cuda"))
        self()
        self.want = [t.clone() for t in self.out]

    def __call__(self):
        self.f(*self.x, mask="causal", O=self.out[0], LSE=self.out[1])

    def spoil(self):
        for t in self.out:
            t.fill_(7)

    def right(self):
        return all(torch.equal(a, b) for a, b in zip(self.out, self.want))


def fixed(B, H, N, d, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return Call(fa.fwd, *(randn(g, B, H, N, d) for _ in range(3)), (B, H, N))


def packed(lens, Hq, Hkv, d, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    T = sum(lens)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    return Call(lambda Q, K, V, **k: fa.fwd_packed(Q, K, V, cu, cu, **k), *(randn(g, T, h, d) for h in (Hq, Hkv, Hkv)), (Hq, T))


def capture(f, n=1):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            f()
    return graph


@pytest.mark.parametrize("kind", ["fixed", "packed"])
def test_graphs_thousands_of_captures_apart_replayed_at_once(kind):
    if kind == "fixed":
        first, last = fixed(2, 8, 2048, 128, 1), fixed(3, 8, 1500, 64, 2)
    else:
        first, last = packed([2000, 3, 1500], 16, 4, 128, 1), packed([900, 2500, 64], 8, 8, 64, 2)
    small = fixed(1, 1, 64, 64, 3)
    torch.cuda.synchronize()
    a = capture(first)
    between = capture(small, 2047)
    b = capture(last)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        first.spoil()
        last.spoil()
        torch.cuda.synchronize()
        for _ in range(20):
            for s, g in zip(streams, (a, b)):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert first.right() and last.right()
    small.spoil()
    between.replay()
    assert small.right() and fa.device_status() == 0


def test_counters_come_back_with_their_graphs():
    # more captured launches than there are counters, a few graphs alive at a time
    c = fixed(1, 2, 200, 64, 4)
    torch.cuda.synchronize()
    alive = []
    for i in range(72):
        alive = [*alive[-2:], capture(c, 1000)]
        if i % 24 == 0:
            c.spoil()
            alive[-1].replay()
            torch.cuda.synchronize()
            assert c.right()
    del alive
    gc.collect()
    c.spoil()
    c()
    assert c.right() and fa.device_status() == 0
