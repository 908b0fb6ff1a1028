"""The MXFP4 layer between calls: codes refreshed in place reach the backward, eager and captured; the weight
gradient by itself reads this batch's rows."""
import sys

import pytest
import torch

import moe_synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _say(*a):
    print("[gpu-mx4-layer]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


def _inputs(T, d, E, f, k, seed):
    inp = moe_synth.make_inputs(T=T, d=d, E=E, f=f, k=k, seed=seed)
    return {n: inp[n].to(DEV) for n in ("logits", "x", "w13", "w2", "dout")}


def _codes(moe, g, d, f):
    """w13 and w2 in 4 bits: codes, scales of each."""
    q = []
    for w, K in ((g["w13"], d), (g["w2"], f)):
        c = torch.empty(*w.shape[:2], K // 2, dtype=torch.uint8, device=DEV)
        s = torch.empty(*w.shape[:2], K // 32, dtype=torch.uint8, device=DEV)
        moe.moe_quantize_mxfp4(w.reshape(-1, K), c.view(-1, K // 2), s.view(-1, K // 32))
        q += [c, s]
    return q


def test_codes_refreshed_in_place_reach_the_backward(moe):
    """A layer given its weights in 4 bits reads the tensors it was given: after they are quantised
    anew in place, as an optimizer step does, out and dx both come from the new ones."""
    _say("refreshed")
    from routing_grouped_gemm_amd.layer import MoELayer
    T, d, E, f, k = 150, 256, 4, 128, 2
    old, new = _inputs(T, d, E, f, k, 1), _inputs(T, d, E, f, k, 2)
    want = MoELayer(T, d, E, f, k, moe.MOE_MXFP4)
    want.set_weights_mxfp4(*_codes(moe, new, d, f))
    ref = {"out": want.forward(old["logits"], old["x"]).clone()}
    ref.update(zip(("dx", "dw13", "dw2"), [t.clone() for t in want.backward(old["dout"])]))

    def check(lay, what):
        torch.cuda.synchronize()
        for n, v in ref.items():
            assert torch.equal(getattr(lay, n), v), (what, n)
            getattr(lay, n).fill_(0)

    lay = MoELayer(T, d, E, f, k, moe.MOE_MXFP4)
    mine = _codes(moe, old, d, f)
    lay.set_weights_mxfp4(*mine)

    def step():
        lay.forward(old["logits"], old["x"])
        lay.backward(old["dout"])
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    fresh = _codes(moe, new, d, f)
    for a, b in zip(mine, fresh):
        a.copy_(b)
    for rep in range(3):
        step()
        check(lay, "eager")
        graph.replay()
        check(lay, "replayed")
    # stage by stage: the gradients of the activations before and after another refresh
    first = _codes(moe, old, d, f)
    for codes in (first, fresh):
        for a, b in zip(mine, codes):
            a.copy_(b)
        lay.forward(old["logits"], old["x"])
        for op in (moe.MOE_GEMM_DGRAD_DOWN, moe.MOE_GEMM_DGRAD_GATE_UP):
            lay.gemm_stage(op)
    torch.cuda.synchronize()
    assert torch.equal(lay.dx_perm, want.dx_perm)


def test_accumulating_after_single_stages_reads_this_batch(moe):
    """The activation gradients stage by stage, then the weight gradient into fp32 accumulators without the
    bf16 stage in between: it is this batch's, the rows of the batch before have been decoded there."""
    _say("accumulate")
    from routing_grouped_gemm_amd.layer import MoELayer
    T, d, E, f, k = 90, 256, 4, 128, 2
    a, b = _inputs(T, d, E, f, k, 5), _inputs(T, d, E, f, k, 6)
    lay, want = (MoELayer(T, d, E, f, k, moe.MOE_MXFP4) for _ in range(2))
    for x in (lay, want):
        x.set_weights(a["w13"], a["w2"])
    lay.forward(a["logits"], a["x"])
    lay.backward(a["dout"])
    acc = [[torch.zeros(E, 2 * f, d, device=DEV), torch.zeros(E, d, f, device=DEV)] for _ in range(2)]
    for x in (lay, want):
        x.forward(b["logits"], b["x"])
    want.backward(b["dout"])
    want.wgrad_accumulate(*acc[1])
    moe.moe_permute(moe.MOE_BF16, b["dout"], k, lay.s_dst, lay.dy_perm, row_scale=lay.s_w)
    for op in (moe.MOE_GEMM_DGRAD_DOWN, moe.MOE_GEMM_DGRAD_GATE_UP):
        lay.gemm_stage(op)
    lay.wgrad_accumulate(*acc[0])
    torch.cuda.synchronize()
    assert torch.equal(lay.dx_perm, want.dx_perm)
    assert torch.equal(acc[0][0], acc[1][0]) and torch.equal(acc[0][1], acc[1][1])
