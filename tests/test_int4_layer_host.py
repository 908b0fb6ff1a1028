"""CPU checks of the 4-bit integer layer's weights: which tensors a quantisation writes and which calls are refused.  No
kernel runs: the quantiser is replaced."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import routing_grouped_gemm_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return m


T, D, E, F, K, G = 8, 128, 4, 192, 2, 64
BF = torch.bfloat16


def _weights():
    return torch.ones(E, 2 * F, D, dtype=BF), torch.ones(E, D, F, dtype=BF)


@pytest.fixture
def made(m, monkeypatch):
    """What the quantiser is called with."""
    from routing_grouped_gemm_amd import layer
    calls = []
    monkeypatch.setattr(layer, "moe_quantize_int4", lambda *a: calls.append(a))
    return calls


@pytest.mark.parametrize("zeros", [False, True])
def test_requantized_in_place(m, made, zeros):
    """The tensors that a captured forward reads take the new codes, whoever made them."""
    from routing_grouped_gemm_amd.layer import MoELayer
    lay = MoELayer(T, D, E, F, K, m.MOE_INT4, device="cpu", group=G, zeros=zeros)
    lay.set_weights(*_weights())
    other = MoELayer(T, D, E, F, K, m.MOE_INT4, device="cpu", group=G, zeros=zeros)
    other.set_weights_int4(lay.w13_4, lay.w2_4)
    held = lay.w13_4, lay.w2_4
    first = made[:]
    for one in (lay, other):
        del made[:]
        w13, w2 = _weights()
        one.requantize_weights(w13, w2)
        assert (one.w13_4, one.w2_4) == held
        assert len(made) == 2
        for (src, group, codes, scales, z), before, w, n in zip(made, first, (w13, w2), (D, F)):
            assert src.data_ptr() == w.data_ptr() and src.shape[1] == n and group == G
            for t, b in zip((codes, scales, z), before[2:]):
                assert (t is None and b is None and not zeros) or (t.data_ptr() == b.data_ptr() and t.shape == b.shape)


def test_requantize_refusals(m, made):
    from routing_grouped_gemm_amd.layer import MoELayer
    w13, w2 = _weights()
    lay = MoELayer(T, D, E, F, K, m.MOE_INT4, device="cpu", group=G)
    with pytest.raises(ValueError):
        lay.requantize_weights(w13, w2)                     # no weights yet
    lay.set_weights(w13, w2)
    del made[:]
    for a in ((), (w13,), (w13, w2.float()), (w13[1:], w2), (w13.to("meta"), w2), (w2, w13)):
        with pytest.raises(ValueError):
            lay.requantize_weights(*a)
    assert not made
    for dtype in (m.MOE_F32, m.MOE_BF16):
        with pytest.raises(ValueError):
            MoELayer(T, D, E, F, K, dtype, device="cpu").requantize_weights()
    with pytest.raises(ValueError):
        MoELayer(T, D, E, 128, K, m.MOE_MXFP4, device="cpu").requantize_weights(w13, w2)
