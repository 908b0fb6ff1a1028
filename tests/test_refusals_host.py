"""CPU checks that tensors of another type, size or place than a call reads are refused before anything is launched: a
kernel given them would read or write past their ends.  No kernel runs."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import routing_grouped_gemm_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return m


T, D, E, F, K = 8, 128, 4, 128, 2
BF, F32 = torch.bfloat16, torch.float32
TYPES = {"F32": F32, "BF16": BF, "MXFP8": BF}


def _weights(t):
    return torch.zeros(E, 2 * F, D, dtype=t), torch.zeros(E, D, F, dtype=t)


def _layer(m, name, monkeypatch):
    from routing_grouped_gemm_amd import layer
    monkeypatch.setattr(layer, "moe_quantize_mxfp8", lambda *a: None)     # (its tensors are on the CPU)
    return layer.MoELayer(T, D, E, F, K, getattr(m, "MOE_" + name), device="cpu")


@pytest.mark.parametrize("bad", ["w13 type", "w2 type", "w13 half", "w13 short", "w2 short", "w13 place", "w2 place",
                                 "w13 strided"])
@pytest.mark.parametrize("name", TYPES)
def test_weights_of_another_kind_leave_the_earlier_ones(m, name, bad, monkeypatch):
    if (name, bad) == ("MXFP8", "w13 strided"):
        pytest.skip("the MXFP8 caches are made from a dense copy of such weights")
    lay = _layer(m, name, monkeypatch)
    t = TYPES[name]
    had = _weights(t)
    lay.set_weights(*had)
    which, how = bad.split()
    w = dict(zip(("w13", "w2"), _weights(t)))
    w[which] = {"type": lambda v: v.to(F32 if t is BF else BF), "half": lambda v: v.half(), "short": lambda v: v[1:],
                "place": lambda v: v.to("meta"), "strided": lambda v: v.repeat(1, 1, 2)[..., ::2]}[how](w[which])
    with pytest.raises(ValueError, match=which):
        lay.set_weights(**w)
    assert lay.w13 is had[0] and lay.w2 is had[1]


@pytest.mark.parametrize("name", TYPES)
def test_weights_of_any_shape_with_their_elements_are_taken(m, name, monkeypatch):
    lay = _layer(m, name, monkeypatch)
    w13, w2 = (w.flatten(0, 1) for w in _weights(TYPES[name]))
    lay.set_weights(w13, w2)
    assert lay.w13 is w13 and lay.w2 is w2


@pytest.mark.parametrize("at", range(4))
@pytest.mark.parametrize("how", ["type", "short", "place", "strided"])
def test_four_bit_weights_of_another_kind_leave_the_earlier_ones(m, at, how):
    from routing_grouped_gemm_amd.layer import MoELayer
    lay = MoELayer(T, D, E, F, K, m.MOE_MXFP4, device="cpu")

    def codes():
        return [torch.zeros(E, n, dtype=torch.uint8) for n in (F * D, 2 * F * D // 32, D * F // 2, D * F // 32)]
    had = codes()
    lay.set_weights_mxfp4(*had)
    w = codes()
    w[at] = {"type": lambda v: v.to(torch.int16), "short": lambda v: v[1:], "place": lambda v: v.to("meta"),
             "strided": lambda v: v.repeat(1, 2)[:, ::2]}[how](w[at])
    with pytest.raises(ValueError):
        lay.set_weights_mxfp4(*w)
    assert all(a is b for a, b in zip((lay.w13_q, lay.w13_s, lay.w2_q, lay.w2_s), had))
