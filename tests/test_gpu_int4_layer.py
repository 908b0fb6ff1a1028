"""The 4-bit integer layer under a captured graph: weights that change, tokens that change."""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _say(*a):
    print("[gpu-int4-layer]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


def _inputs(T, d, E, f, seed):
    g = torch.Generator().manual_seed(seed)

    def make(*shape, s=1.0):
        return (torch.randn(*shape, generator=g) * s).to(DEV)
    return make(T, E), make(T, d).to(BF), make(E, 2 * f, d, s=d ** -0.5).to(BF), make(E, d, f, s=f ** -0.5).to(BF)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T", [3, 60, 300])
def test_weights_requantized_under_a_graph(moe, T, zeros):
    """Replays read the codes quantised anew in place: each one bit for bit what a layer made with those weights gives,
    in the forms for single tokens, few and many rows."""
    from routing_grouped_gemm_amd.layer import MoELayer
    d, E, f, k, group = 256, 8, 128, 2, 64
    _say(T, zeros)
    kw = dict(group=group, zeros=zeros, act=moe.MOE_ACT_GELU)
    logits, x, w13, w2 = _inputs(T, d, E, f, 1)
    lay = MoELayer(T, d, E, f, k, moe.MOE_INT4, **kw)
    lay.set_weights(w13, w2)
    held = [t.data_ptr() for w in (lay.w13_4, lay.w2_4) for t in w if t is not None]
    lay.forward(logits, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay.forward(logits, x)
    seen = []
    for n in range(3):
        l2, x2, w13, w2 = _inputs(T, d, E, f, 10 + n)
        logits.copy_(l2)
        x.copy_(x2)
        lay.requantize_weights(w13, w2)
        assert held == [t.data_ptr() for w in (lay.w13_4, lay.w2_4) for t in w if t is not None]
        fresh = MoELayer(T, d, E, f, k, moe.MOE_INT4, **kw)
        fresh.set_weights(w13, w2)
        want = fresh.forward(logits, x).clone()
        lay.out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lay.out, want), n
        seen.append(want)
    assert not torch.equal(seen[0], seen[1])
