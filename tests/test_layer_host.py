"""CPU checks of MoELayer's bookkeeping: what a refused call leaves behind, which buffers outlive a call.
No kernel runs: the layer's buffers are host tensors, and the calls that would launch are refused or replaced."""
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


def test_balance_buffers_outlive_other_numbers_of_sequences(m, monkeypatch):
    """What a balance_loss writes to stays allocated while the layer lives (a captured one replays into it)
    when later calls have other numbers of sequences, and does not grow with every new number."""
    import weakref

    from routing_grouped_gemm_amd import layer
    refs = []

    def record(logits, topk_idx, cb, cz, losses, counts, probs, lse, tokens, ws, seg_off=None, mask=None, dev_err=None):
        n = counts.shape[0]
        assert counts.shape == (n, E) and probs.shape == (n, E) and tokens.shape == (n + 1,) and losses.shape == (2,)
        assert all(t.is_contiguous() for t in (counts, probs, tokens, ws))
        assert ws.numel() >= m.moe_balance_workspace_bytes(T, E, n)
        refs.append([weakref.ref(t if t._base is None else t._base) for t in (losses, counts, probs, tokens, ws)])

    monkeypatch.setattr(layer, "moe_balance_loss", record)
    lay = layer.MoELayer(T, D, E, F, K, m.MOE_BF16, device="cpu")
    logits = torch.zeros(T, E)
    for n in (4, 1, 3, 4, 7, 2, 300, 5, 1):
        lay.balance_loss(logits, 0.1, 0.0, seg_off=None if n == 1 else torch.zeros(n + 1, dtype=torch.int32))
    assert all(r() is not None for call in refs for r in call)
    assert len({id(r()) for call in refs for r in call}) == 1 + 3 * 4    # losses; sets for 4, 8 and 512 sequences


def test_balance_workspace_grows_with_the_sequences(m):
    """A workspace for more sequences serves fewer."""
    for T_ in (0, 1, 63, 64, 1000, 16391, 1 << 20, 1 << 30):
        for E_ in (1, 8, 130, 1024):
            sizes = [m.moe_balance_workspace_bytes(T_, E_, n) for n in list(range(1, 70)) + [100, 999, 5000, 1 << 16, 1 << 20]]
            assert sizes == sorted(sizes), (T_, E_)


def test_src_slot_of_another_length_is_refused(m):
    """moe_permute reads a slot for each row of x_perm."""
    x, dst = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    out = torch.zeros(8, 64, dtype=torch.bfloat16)
    for n in (7, 9):
        with pytest.raises(ValueError):
            m.moe_permute(m.MOE_BF16, x, 2, dst, out, src_slot=torch.zeros(n, dtype=torch.int32))
