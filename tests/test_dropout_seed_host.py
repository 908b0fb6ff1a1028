"""CPU checks of the seeds that layers drop by."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import routing_grouped_gemm_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return m


def _layer(m, **kw):
    from routing_grouped_gemm_amd.layer import MoELayer
    return MoELayer(8, 64, 4, 64, 2, m.MOE_BF16, device="cpu", **kw)


@pytest.mark.parametrize("kw", [dict(h_dropout=0.1), dict(out_dropout=0.1)])
def test_layers_without_a_seed_drop_different_elements(m, kw):
    seeds = [int(_layer(m, **kw).rng[0, 0]) for _ in range(20)]
    assert len(set(seeds)) == 20 and all(0 <= s < 2 ** 62 for s in seeds)


def test_torch_seeds_repeat_them(m):
    def three():
        torch.manual_seed(5)
        return [_layer(m, out_dropout=0.1).rng.tolist() for _ in range(3)]
    assert three() == three()


def test_a_given_seed_is_taken(m):
    for seed in (0, 7, -3, 2 ** 63 - 1):
        assert _layer(m, h_dropout=0.1, seed=seed).rng.tolist() == [[seed, 0], [seed, 1 << 62]]


def test_layers_without_dropout_draw_nothing(m):
    torch.manual_seed(1)
    want = torch.rand(3)
    torch.manual_seed(1)
    _layer(m)
    _layer(m, act=m.MOE_ACT_RELU)
    _layer(m, out_dropout=0.2, seed=4)
    assert torch.equal(torch.rand(3), want)
