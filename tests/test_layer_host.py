"""CPU checks of MoELayer's bookkeeping: what a refused call leaves behind.  No kernel runs: the layer's
buffers are host tensors, and the calls that would launch are refused or replaced."""
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


def _codes():
    u8 = dict(dtype=torch.uint8)
    return (torch.zeros(E, 2 * F, D // 2, **u8), torch.zeros(E, 2 * F, D // 32, **u8), torch.zeros(E, D, F // 2, **u8),
            torch.zeros(E, D, F // 32, **u8))


@pytest.mark.parametrize("bad", ["w13 fp32", "w2 fp32", "w13 short", "w2 short", "host"])
def test_refused_weights_leave_the_earlier_ones(m, bad):
    from routing_grouped_gemm_amd.layer import MoELayer
    lay = MoELayer(T, D, E, F, K, m.MOE_MXFP4, device="cpu")
    codes = _codes()
    lay.set_weights_mxfp4(*codes)
    w = {"w13": torch.ones(E, 2 * F, D, dtype=torch.bfloat16), "w2": torch.ones(E, D, F, dtype=torch.bfloat16)}
    if bad != "host":
        name, how = bad.split()
        w[name] = w[name].float() if how == "fp32" else w[name][1:]
    with pytest.raises(ValueError):
        lay.set_weights(w["w13"], w["w2"])
    assert all(a is b for a, b in zip((lay.w13_q, lay.w13_s, lay.w2_q, lay.w2_s), codes))
    assert lay.w13 is None and lay.w2 is None
    assert not any(bool(c.any()) for c in codes)


def test_decode_h_is_refused_where_there_is_no_4_bit_h(m):
    from routing_grouped_gemm_amd.layer import MoELayer
    for dtype in (m.MOE_F32, m.MOE_BF16, m.MOE_MXFP8):
        with pytest.raises(ValueError):
            MoELayer(T, D, E, F, K, dtype, device="cpu", decode_h=True)
    with pytest.raises(ValueError):
        MoELayer(T, D, E, F, K, m.MOE_MXFP4, device="cpu", save=False, decode_h=True)
