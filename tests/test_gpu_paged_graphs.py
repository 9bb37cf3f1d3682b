"""Paged decode in many graphs, and over workspaces of any contents: divided units
are joined right whoever else is decoding at the same time."""
import pytest
import torch

import exact_io_aware_65_b200 as fa
import paged_ref as ref
from helpers import has_gpu
from test_gpu_paged import randn

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a B200")]


class Call:
    """A decode call with buffers and a workspace of its own."""

    def __init__(self, lens, Hq, Hkv, d, page, e4m3, seed):
        self.c = ref.dev(ref.make_cache(lens, Hkv, d, page, e4m3, seed=seed, poison=False))
        self.Q = randn(len(lens), Hq, d, seed=seed + 1).cuda()
        n = fa.paged_decode_workspace_size(len(lens), Hq, Hkv, d, self.c["table"].shape[1] * page)
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.want = [t.clone() for t in self.made()]
        self.out = [torch.empty_like(t) for t in self.want]

    def made(self, **k):
        c = self.c
        return fa.paged_decode(self.Q, c["kc"], c["vc"], c["table"], c["lens"], k_scale=c["ks"], v_scale=c["vs"], **k)

    def __call__(self):
        self.made(O=self.out[0], LSE=self.out[1], workspace=self.ws)

    def right(self):
        return all(torch.equal(x, y) for x, y in zip(self.out, self.want))


def test_graphs_a_thousand_captures_apart_replayed_at_once():
    # a server captures one decode a layer and batch size; any two of the graphs may run together
    first, last = Call([9000, 30], 16, 2, 128, 16, False, seed=1), Call([12000], 8, 1, 64, 64, True, seed=3)
    between = Call([700], 4, 1, 64, 16, False, seed=5)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(3)]
    with torch.cuda.graph(graphs[0]):
        first()
    with torch.cuda.graph(graphs[1]):
        for _ in range(1023):
            between()
    with torch.cuda.graph(graphs[2]):
        last()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for c in (first, last):
            for t in c.out:
                t.fill_(7)
        torch.cuda.synchronize()
        for _ in range(20):
            for s, g in zip(streams, (graphs[0], graphs[2])):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert first.right() and last.right()
    graphs[1].replay()
    assert between.right() and fa.device_status() == 0


@pytest.mark.parametrize("args", [([9000, 30, 0, 1500], 16, 2, 128, 16, False), ([777], 32, 8, 128, 16, False),
                                  ([3000] * 40, 10, 2, 64, 64, True)], ids=["mixed", "one", "many"])
def test_the_workspace_may_hold_anything(args):
    a = Call(*args, seed=11)
    g = torch.Generator("cuda").manual_seed(12)
    for _ in range(3):
        fills = [lambda: a.ws.zero_(), lambda: a.ws.fill_(255), lambda: a.ws.fill_(1), lambda: None,
                 lambda: a.ws.copy_(torch.randint(0, 256, a.ws.shape, generator=g, device="cuda", dtype=torch.uint8)),
                 lambda: a.ws.view(torch.float32)[:a.ws.numel() // 4].fill_(float("nan"))]
        for fill in fills:
            fill()
            for t in a.out:
                t.fill_(7)
            a()
            assert a.right()
    # a workspace that a call of another shape has used, and then this one's own again
    b = Call([5000, 4000], 24, 8, 64, 24, False, seed=13)
    both = torch.empty(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device="cuda")
    a.ws = b.ws = both
    for _ in range(4):
        for c in (a, b):
            c()
            assert c.right()
    assert fa.device_status() == 0
