"""Padding rows of a layout with as many rows as there are routed pairs (capacity factor 1: E * C == T * k),
where some experts drop pairs and others have empty rows: the empty rows are zero-filled, and what an earlier
batch left there reaches no gradient."""
import sys

import numpy as np
import pytest
import torch

import moe_synth
import oracle
from tests._chain import BF16_TOL, assert_close, np64, oracle_layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _say(*a):
    print("[gpu-padding]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


T, D, E, F, K = 120, 256, 4, 128, 2
C = T * K // E


def _skewed(seed):
    inp = moe_synth.make_inputs(T=T, d=D, E=E, f=F, k=K, seed=seed)
    inp["logits"][:, 0] += 2.0
    return inp


@pytest.mark.parametrize("dtype", ["MOE_F32", "MOE_BF16", "MOE_MXFP8", "MOE_MXFP4"])
def test_empty_rows_are_zero(moe, dtype):
    _say("rows", dtype)
    inp = _skewed(1)
    r = oracle.route(inp["logits"].numpy(), K, C)
    n = r["n_rows"]
    assert n == T * K
    empty = torch.from_numpy(r["src_slot"] < 0).to(DEV)
    assert 0 < int(empty.sum()) < n
    dt = getattr(moe, dtype)
    x = inp["x"].to(DEV) if dt != moe.MOE_F32 else inp["x"].float().to(DEV)
    width = {"MOE_F32": D * 4, "MOE_BF16": D * 2, "MOE_MXFP8": D, "MOE_MXFP4": D // 2}[dtype]
    raw = torch.full((n, width), 0x55, dtype=torch.uint8, device=DEV)
    out = raw if dtype.startswith("MOE_MX") else raw.view(x.dtype)
    scales = torch.full((n, D // 32), 0x55, dtype=torch.uint8, device=DEV) if dtype.startswith("MOE_MX") else None
    moe.moe_permute(dt, x, K, torch.from_numpy(r["dst_row"]).to(DEV), out,
                    src_slot=torch.from_numpy(r["src_slot"]).to(DEV), x_perm_scales=scales)
    torch.cuda.synchronize()
    assert not bool(raw[empty].any())
    assert bool((raw[~empty] != 0x55).any(1).all())
    if scales is not None:
        assert not bool(scales[empty].any())


def test_an_earlier_batch_leaves_nothing_in_the_gradients(moe):
    _say("layer bf16")
    from routing_grouped_gemm_amd.layer import MoELayer
    lay = MoELayer(T, D, E, F, K, moe.MOE_BF16, capacity=C)
    for seed, shift in ((2, 0), (3, 1)):           # another expert is the full one
        inp = _skewed(seed)
        inp["logits"] = inp["logits"].roll(shift, 1).contiguous()
        g = {n: inp[n].to(DEV) for n in ("logits", "x", "w13", "w2", "dout")}
        lay.set_weights(g["w13"], g["w2"])
        lay.forward(g["logits"], g["x"])
        lay.backward(g["dout"])
    torch.cuda.synchronize()
    ref = oracle_layer(inp, K, capacity=C)
    for n in ("out", "dx", "dw13", "dw2"):
        assert_close(np64(getattr(lay, n)), ref[n], BF16_TOL, n)


@pytest.mark.parametrize("dtype", ["MOE_MXFP8", "MOE_MXFP4"])
def test_an_earlier_batch_leaves_nothing_in_the_mx_gradients(moe, dtype):
    """The second batch of one layer against the only batch of another whose rows start as zeros."""
    _say("layer", dtype)
    from routing_grouped_gemm_amd.layer import MoELayer
    used, clean = (MoELayer(T, D, E, F, K, getattr(moe, dtype), capacity=C) for _ in range(2))
    for seed in (2, 3):
        inp = _skewed(seed)
        inp["logits"] = inp["logits"].roll(seed, 1).contiguous()
        g = {n: inp[n].to(DEV) for n in ("logits", "x", "w13", "w2", "dout")}
        used.set_weights(g["w13"], g["w2"])
        used.forward(g["logits"], g["x"])
        used.backward(g["dout"])
    clean.set_weights(g["w13"], g["w2"])
    clean._alloc_bwd()
    for t in (clean.x_perm, clean.x_perm_scales, clean.dy_perm, clean.gu, clean.h):
        t.zero_()
    clean.forward(g["logits"], g["x"])
    clean.backward(g["dout"])
    torch.cuda.synchronize()
    for n in ("out", "dx", "dw13", "dw2"):
        assert torch.equal(getattr(used, n), getattr(clean, n)), n
        assert np.isfinite(np64(getattr(used, n))).all()
