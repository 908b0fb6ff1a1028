"""MoELayer with other gates, dropout and 4-bit integer experts: whole steps against 64-bit ones made by autograd, masks
that advance and replay, and a layer trained with a gate served in 4 bits with the same."""
import sys

import pytest
import torch

from tests import _plain_gated as pl

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _say(*a):
    print("[gpu-gated-layer]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


def _inputs(T, d, E, f, t, seed=1):
    g = torch.Generator().manual_seed(seed)
    shapes = dict(logits=((T, E), 1.0), x=((T, d), 1.0), w13=((E, 2 * f, d), 1.2 / d ** 0.5), w2=((E, d, f), f ** -0.5),
                  dout=((T, d), 1.0), residual=((T, d), 1.0))
    out = {n: torch.randn(*s, generator=g) * c for n, (s, c) in shapes.items()}
    return {n: (v if n == "logits" else v.to(t)).to(DEV) for n, v in out.items()}


def _reference(lay, v, act, limit, hp, op, rng):
    """The layer's step in 64 bits, token by token and slot by slot, from its formulas; gradients by autograd, the
    gate weights' too."""
    T, K, f, d = lay.T, lay.K, lay.f, lay.d
    w = {n: v[n].cpu().double().requires_grad_(True) for n in ("x", "w13", "w2", "logits")}
    idx = lay.s_idx.cpu().long()
    top = torch.softmax(torch.gather(w["logits"], 1, idx[:, :lay.k]), 1)
    gates = torch.cat([top, torch.ones(T, lay.S, dtype=torch.float64)], 1)
    dst = lay.s_dst.cpu().long().view(T, K)
    hf = pl.factors(lay.n_rows * f, hp, *rng[0]).view(lay.n_rows, f)
    outs = []
    for t in range(T):
        o = torch.zeros(d, dtype=torch.float64)
        for j in range(K):
            if dst[t, j] < 0:
                continue
            e = idx[t, j]
            gu = w["w13"][e] @ w["x"][t]
            if limit:
                # which elements the limit stops is decided on g and u as saved: of the bf16 ones 2^-8 of the density
                # at each limit (0.3) round onto it from beyond, 2e-3 of all, and pass their gradient
                saved = gu.detach().to(v["x"].dtype).double()
                gu = torch.where((saved <= limit) & ((saved >= -limit) | (torch.arange(2 * f) < f)), gu,
                                 saved.clamp(-limit, limit))
            g, u = gu[:f], gu[f:]
            o = o + gates[t, j] * (w["w2"][e] @ (pl.act(act, g) * u * hf[dst[t, j]]))
        outs.append(o)
    out = torch.stack(outs) * pl.factors(T * d, op, *rng[1]).view(T, d)
    grads = torch.autograd.grad((out * v["dout"].cpu().double()).sum(), [w["x"], w["w13"], w["w2"], w["logits"]])
    return out.detach() + v["residual"].cpu().double(), grads


CASES = [("gelu", 0.0, 0.0, 0.0, 0, 0), ("gelu_tanh", 0.0, 0.2, 0.1, 0, 0), ("silu", 1.0, 0.0, 0.3, 1, 0),
         ("silu", 0.0, 0.4, 0.0, 0, 20), ("relu", 0.0, 0.1, 0.1, 2, 20)]


@pytest.mark.parametrize("t", [BF, torch.float32])
@pytest.mark.parametrize("act,limit,hp,op,S,C", CASES)
def test_step(moe, act, limit, hp, op, S, C, t):
    """fp32 to 2e-5 of the size (sums of at most 200 terms with 2^-23 each); bf16 to 3e-2 (five roundings of 2^-8 on the
    way, gates amplify by at most 2, and relu and the limit flip units within a rounding of their kink)."""
    from routing_grouped_gemm_amd.layer import MoELayer
    T, d, E, f, k = 48, 64, 4, 72, 2
    _say(act, limit, hp, op, S, C, t)
    v = _inputs(T, d, E + S, f, t)
    v["logits"] = v["logits"][:, :E].contiguous()
    dt = moe.MOE_F32 if t is torch.float32 else moe.MOE_BF16
    lay = MoELayer(T, d, E, f, k, dt, capacity=C, n_shared=S, act=pl.ACTS.index(act), limit=limit, h_dropout=hp,
                   out_dropout=op, seed=31)
    lay.set_weights(v["w13"], v["w2"])
    for step in (1, 2):
        out = lay.forward(v["logits"], v["x"], residual=v["residual"])
        dx, dw13, dw2 = lay.backward(v["dout"])
        got = dict(out=out, dx=dx, dw13=dw13, dw2=dw2)
        if dt == moe.MOE_BF16 and not S:
            got["dlogits"] = lay.gate_grad(v["dout"])
        torch.cuda.synchronize()
        ref, (rx, r13, r2, rl) = _reference(lay, v, act, limit, hp, op, ((31, step), (31, (1 << 62) + step)))
        for n, r in dict(out=ref, dx=rx, dw13=r13, dw2=r2, dlogits=rl).items():
            if n not in got:
                continue
            err = float((got[n].cpu().double() - r).norm() / r.norm())
            assert err <= (3e-2 if t is BF else 2e-5), (n, err, step)
        again = lay.forward(v["logits"], v["x"], residual=v["residual"], same_mask=True).clone()
        assert torch.equal(again, out)
    lay.training = False
    out = lay.forward(v["logits"], v["x"], residual=v["residual"])
    ref, _ = _reference(lay, v, act, limit, 0.0, 0.0, ((0, 0), (0, 0)))
    assert float((out.cpu().double() - ref).norm() / ref.norm()) <= (3e-2 if t is BF else 2e-5)


def test_stage_by_stage_and_accumulated_weight_gradients(moe):
    """The stages by themselves give what forward and backward give, and the weight gradient adds into fp32."""
    from routing_grouped_gemm_amd.layer import MoELayer
    T, d, E, f, k = 300, 128, 4, 128, 2
    v = _inputs(T, d, E, f, BF)
    lay = MoELayer(T, d, E, f, k, act=moe.MOE_ACT_GELU, limit=2.0, h_dropout=0.2, seed=5)
    lay.set_weights(v["w13"], v["w2"])
    lay.forward(v["logits"], v["x"])
    lay.backward(v["dout"])
    names = ("gu", "h", "y_perm", "dgu", "dx_perm", "dw13", "dw2")
    want = {n: getattr(lay, n).clone() for n in names}
    for n in names:
        getattr(lay, n).fill_(0)
    for op in range(5):
        lay.gemm_stage(op)
    for n in names:
        assert torch.equal(getattr(lay, n), want[n]), n
    a, b = torch.ones_like(lay.dw13, dtype=torch.float32), torch.ones_like(lay.dw2, dtype=torch.float32)
    lay.wgrad_accumulate(a, b)
    torch.testing.assert_close(a.to(BF), (want["dw13"].float() + 1).to(BF), rtol=2 ** -6, atol=2 ** -6)
    torch.testing.assert_close(b.to(BF), (want["dw2"].float() + 1).to(BF), rtol=2 ** -6, atol=2 ** -6)


@pytest.mark.parametrize("dt", ["BF16", "MXFP8", "MXFP4"])
def test_replayed_steps_draw_the_masks_of_eager_ones(moe, dt):
    """A captured step advances its masks by itself: replay n is the eager step n from the same seed, eager work between."""
    from routing_grouped_gemm_amd.layer import MoELayer
    T, d, E, f, k = 128, 256, 4, 128, 2
    v = _inputs(T, d, E, f, BF)
    kw = dict(act=moe.MOE_ACT_RELU, h_dropout=0.3) if dt == "BF16" else {}
    lays = [MoELayer(T, d, E, f, k, getattr(moe, "MOE_" + dt), out_dropout=0.2, seed=77, **kw) for _ in range(2)]
    for lay in lays:
        lay.set_weights(v["w13"], v["w2"])

    def step(lay):
        lay.forward(v["logits"], v["x"], residual=v["residual"])
        lay.backward(v["dout"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(lays[0])
    torch.cuda.synchronize()
    step(lays[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(lays[0])
    seen = []
    for n in range(4):
        for t in (lays[0].out, lays[0].dx, lays[0].dw2):
            t.fill_(0)
        graph.replay()
        step(lays[1])
        torch.cuda.synchronize()
        for name in ("out", "dx", "dw13", "dw2"):
            assert torch.equal(getattr(lays[0], name), getattr(lays[1], name)), (n, name)
        seen.append(lays[0].out.clone())
    assert not any(torch.equal(a, b) for i, a in enumerate(seen) for b in seen[:i])


@pytest.mark.parametrize("T,S", [(1, 0), (1, 1), (3, 2), (40, 1), (200, 0)])
@pytest.mark.parametrize("zeros", [False, True])
def test_served_in_four_bits(moe, T, S, zeros):
    """The INT4 layer against a bf16 layer of the same gate on the decoded weights: the same products but for bf16's
    rounding of the weights (2^-8 of each) and of h and y, all below 2e-2 of the output."""
    from routing_grouped_gemm_amd.layer import MoELayer
    d, E, f, k, group = 256, 6, 128, 2, 32
    v = _inputs(T, d, E + S, f, BF)
    v["logits"] = v["logits"][:, :E].contiguous()
    kw = dict(n_shared=S, act=moe.MOE_ACT_GELU_TANH, limit=3.0)
    lay = MoELayer(T, d, E, f, k, moe.MOE_INT4, group=group, zeros=zeros, **kw)
    lay.set_weights(v["w13"], v["w2"])
    dec = []
    for c, s, z in (lay.w13_4, lay.w2_4):
        w = torch.empty(*c.shape[:2], 2 * c.shape[2], dtype=BF, device=DEV)
        moe.moe_dequantize_int4(c.flatten(0, 1), s.flatten(0, 1), None if z is None else z.flatten(0, 1), group, w.flatten(0, 1))
        dec.append(w)
    ref = MoELayer(T, d, E, f, k, **kw)
    ref.set_weights(*dec)
    a, b = lay.forward(v["logits"], v["x"]).float(), ref.forward(v["logits"], v["x"]).float()
    assert float((a - b).norm() / b.norm()) <= 2e-2
    assert int(lay.dev_err) == 0
    # held in 4 bits elsewhere, and refreshed in place
    other = MoELayer(T, d, E, f, k, moe.MOE_INT4, group=group, zeros=zeros, **kw)
    other.set_weights_int4(lay.w13_4, lay.w2_4)
    assert torch.equal(other.forward(v["logits"], v["x"]).float(), a)
    lay.w13_4[1].mul_(0)
    assert not bool(other.forward(v["logits"], v["x"]).any()) or zeros is None
