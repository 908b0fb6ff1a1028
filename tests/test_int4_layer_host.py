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


# T, E, d, f, k at and past each limit
LIMITS = [(8, 4, 128, 128, 2), (1 << 22, 8, 256, 128, 1), ((1 << 22) - 1, 8, 256, 128, 1), (1 << 20, 8, 128, 128, 8),
          ((1 << 20) - 1, 8, 128, 128, 8), (1, 8, 1 << 20, 2048, 1), (1, 8, 1 << 20, 1984, 1), (1, 8, 1 << 21, 64, 1),
          (1, 8, 64, (1 << 20) + 64, 1), (8, 1024, 64, 64, 8), (8, 1025, 64, 64, 8), (8, 16, 64, 64, 9), (1, 8, 64, 1 << 20, 8)]


@pytest.mark.parametrize("T,E,d,f,k", LIMITS)
def test_sizes_past_the_limits_are_refused_when_the_layer_is_made(m, T, E, d, f, k):
    """As the call refuses them: with good sizes it gets as far as the workspace that is missing here."""
    import ctypes

    from routing_grouped_gemm_amd import layer
    P = 0x10000
    w = ctypes.byref(m.MoeInt4(P, P, None))
    rc = m.load().moe_int4_ffn(ctypes.byref(m.MoeGlu(0, 0.0, 0.0, None)), P, T, k, P, P, P, P, P, E, d, f, 64, w, w, P, None,
                               0, None, None)
    assert rc in (m.MOE_EINVAL, m.MOE_EWORKSPACE)
    ok = rc == m.MOE_EWORKSPACE
    assert layer.int4_sizes_ok(T, E, d, f, k) == ok
    if not ok:
        for S in ((0, 1) if k > 1 else (0,)):
            with pytest.raises(ValueError):
                layer.MoELayer(T, d, E - S, f, k - S, m.MOE_INT4, device="cpu", group=64, n_shared=S)


def test_forward_without_weights_is_refused(m):
    from routing_grouped_gemm_amd.layer import MoELayer
    lay = MoELayer(T, D, E, F, K, m.MOE_INT4, device="cpu", group=G)
    with pytest.raises(ValueError, match="weights"):
        lay.forward(torch.zeros(T, E), torch.zeros(T, D, dtype=BF))
