"""The MXFP4 layer between calls: codes refreshed in place reach the backward, eager and captured; the weight
gradient by itself reads this batch's rows; dw2 from the 4-bit h."""
import sys

import numpy as np
import pytest
import torch

import moe_synth
from tests import _plain
from tests._chain import BF16_TOL, assert_close, np64

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


@pytest.mark.parametrize("T,d,E,f,k,S,C", [(300, 256, 6, 256, 2, 0, 0), (64, 128, 8, 128, 2, 1, 0),
                                           (120, 384, 4, 128, 2, 0, 60)])
def test_dw2_of_the_forward_that_ran(moe, T, d, E, f, k, S, C):
    """decode_h: dw2 is the derivative of <dout, out> in the (decoded) W2, by the formula and by differences
    of a 64-bit forward; the other gradients are those of the layer without it."""
    _say("dw2", T, d, E, f, k, S, C)
    from routing_grouped_gemm_amd.layer import MoELayer
    inp = moe_synth.make_inputs(T=T, d=d, E=E + S, f=f, k=k, seed=T)
    inp["logits"] = inp["logits"][:, :E].contiguous()
    g = {n: inp[n].to(DEV) for n in ("logits", "x", "w13", "w2", "dout")}
    lays = []
    for decode in (False, True):
        lay = MoELayer(T, d, E, f, k, moe.MOE_MXFP4, capacity=C, n_shared=S, decode_h=decode)
        lay.set_weights(g["w13"], g["w2"])
        lay.forward(g["logits"], g["x"])
        lay.backward(g["dout"])
        lays.append(lay)
    torch.cuda.synchronize()
    plain, lay = lays
    for n in ("out", "dx", "dw13"):
        assert torch.equal(getattr(plain, n), getattr(lay, n)), n
    off = lay.s_off.cpu().numpy().astype(np.int64)
    if C and not S:
        off = np.arange(E + 1) * C
    h, w2 = np64(lay.h), np64(lay.w2_d)
    used = np.zeros(h.shape[0], bool)
    for a, b in zip(off[:-1], off[1:]):
        used[a:b] = True
    hq = np.zeros_like(h)
    hq[used] = _plain.mxfp4_qdq(h[used])
    np.testing.assert_array_equal(np64(lay.h_d)[used], hq[used])
    dst, w = lay.s_dst.cpu().numpy(), np64(lay.s_w).reshape(-1)
    K = k + S
    dout = np64(inp["dout"])
    dy = np.zeros((h.shape[0], d))
    live = dst >= 0
    dy[dst[live]] = w[live, None] * dout[np.nonzero(live)[0] // K]
    want = np.stack([dy[a:b].T @ hq[a:b] for a, b in zip(off[:-1], off[1:])])
    assert_close(np64(lay.dw2), want, BF16_TOL, "dw2")
    other = np.stack([dy[a:b].T @ h[a:b] for a, b in zip(off[:-1], off[1:])])
    assert_close(np64(plain.dw2), other, BF16_TOL, "dw2 of the saved h")

    def loss(w2):
        y = np.concatenate([hq[a:b] @ m.T for a, b, m in zip(off[:-1], off[1:], w2)])
        y = np.concatenate([y, np.zeros((h.shape[0] - len(y), d))])
        out = np.zeros((T, d))
        np.add.at(out, np.nonzero(live)[0] // K, w[live, None] * y[dst[live]])
        return (out * dout).sum()

    rng = np.random.default_rng(1)
    for _ in range(10):
        e, i, j = rng.integers(E + S), rng.integers(d), rng.integers(f)
        hi, lo = w2.copy(), w2.copy()
        hi[e, i, j] += 0.5
        lo[e, i, j] -= 0.5
        diff = loss(hi) - loss(lo)                     # the forward is linear in W2
        assert abs(diff - want[e, i, j]) <= 1e-9 * np.abs(want).max()
    # stage by stage, and into fp32 accumulators
    ref = lay.dw2.clone()
    lay.dw2.zero_()
    lay.gemm_stage(moe.MOE_GEMM_WGRAD)
    a13, a2 = torch.zeros(E + S, 2 * f, d, device=DEV), torch.zeros(E + S, d, f, device=DEV)
    lay.wgrad_accumulate(a13, a2)
    torch.cuda.synchronize()
    assert torch.equal(lay.dw2, ref)
    assert_close(np64(a2), want, BF16_TOL, "dw2 accumulated")
