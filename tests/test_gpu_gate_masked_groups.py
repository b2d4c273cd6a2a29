"""Groups that are masked whole: their worth, -inf, is exact, so they neither change the other groups' order nor send
tokens to the slower order in 64 bits."""
import statistics

import pytest
import torch

import mixture_experts_router_amd as moe
from test_gpu_gate import check, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,G,group_k,k", [(256, 8, 4, 8), (64, 8, 3, 4), (64, 2, 1, 4), (96, 6, 4, 6), (250, 50, 9, 8),
                                           (126, 63, 5, 5), (128, 4, 3, 6), (60, 3, 2, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_best", [1, 2])
def test_order_with_groups_masked(E, G, group_k, k, score, group_best):
    """0 .. G groups of a row masked by their logits, and some by their bias: fewer left than are kept, too."""
    T, gs = 4 * (G + 1), E // G
    l = logits_of(E + G, T, E)
    g = torch.Generator().manual_seed(G)
    for t in range(T):
        out = torch.randperm(G, generator=g)[:t % (G + 1)]
        l[t].view(G, gs)[out] = -torch.inf
        l[t].view(G, gs)[torch.randperm(G, generator=g)[:1], 1:] = -torch.inf  # one of one expert
    bias = torch.randn(E, generator=g) * 0.1
    kw = dict(score=score, groups=G, group_k=group_k, group_best=group_best)
    check(l, k, bias=bias, **kw)
    if group_best == 2:
        check(l, k, **kw)
    bias.view(G, gs)[G // 2] = -torch.inf
    bias.view(G, gs)[0, 1:] = torch.finfo(torch.float32).min  # two of them: beyond fp32, not beyond fp64
    check(l, k, bias=bias, **kw)


def test_time_with_a_group_masked():
    """16384 tokens with one of eight groups masked take at most twice the time of the same tokens without (1.0 times
    is usual, 4 where every token is ordered in 64 bits)."""
    T, E = 16384, 256
    l = logits_of(3, T, E).cuda()
    m = l.clone()
    m[:, 32:64] = -torch.inf
    bias = (torch.randn(E, generator=torch.Generator().manual_seed(4)) * 0.1).cuda()
    out = (torch.empty(T, 8, dtype=torch.int32, device="cuda"), torch.empty(T, 8, device="cuda"))
    graphs = []
    for x in (l, m):
        run = lambda: moe.gate_from_logits(x, 8, score="sigmoid", bias=bias, groups=8, group_k=4, group_best=2, out=out)  # noqa: E731,B023
        run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(20):
                run()
    times = ([], [])
    for _ in range(9):
        for g, t in zip(graphs, times):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            t.append(a.elapsed_time(b))
    plain, masked = (statistics.median(t) for t in times)
    print("plain %.1f us, masked %.1f us" % (plain * 50, masked * 50), flush=True)
    assert masked < 2 * plain
