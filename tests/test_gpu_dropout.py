"""Dropout and the combine with dropout against 64-bit values: masks element for element, sums within their rounding."""
import sys

import pytest
import torch

from tests import _plain_gated as pl

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}    # a rounding's half step, relative


def _say(*a):
    print("[gpu-dropout]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


def _rng(seed, step):
    return torch.tensor([seed, step], dtype=torch.int64, device=DEV)


def _type(moe, t):
    return moe.MOE_F32 if t is torch.float32 else moe.MOE_BF16


def _rand(seed, t, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(t)


def _check(got, want, size, t, adds):
    """|got - want| within the last rounding and `adds` fp32 roundings of terms of magnitude `size`."""
    err = (got.cpu().double() - want).abs()
    tol = HALF[t] * want.abs() + (adds * 2.0 ** -24) * size * (1 + HALF[t]) + 1e-38
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-30)).max())


SIZES = [(1, 8), (1, 2048), (3, 24), (63, 72), (257, 128), (5003, 40), (128, 4096)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", SIZES)
def test_dropout(moe, T, d, t, residual):
    _say(T, d, t, residual)
    d = d if t is torch.bfloat16 else d - 4                 # fp32: rows that end inside a generator block
    x, res = _rand(1, t, T, d), _rand(2, t, T, d) * 3 if residual else None
    for p, seed, step in ((0.1, 3, 0), (0.5, -2, 2 ** 63 - 1), (0.999999, 2 ** 40 + 1, 5), (2.0 ** -18, 1, 1), (0.0, 0, 0)):
        out = torch.full((T, d), float("nan"), dtype=t, device=DEV)
        moe.moe_dropout(_type(moe, t), x.to(DEV), p, _rng(seed, step) if p else None, out,
                        residual=None if res is None else res.to(DEV))
        f = pl.factors(T * d, p, seed, step).view(T, d)
        v = x.double() * f
        r = res.double() if residual else torch.zeros_like(v)
        # two fp32 roundings (of the factor, of the product) and that of the sum
        _check(out, v + r, v.abs() + r.abs(), t, 3)
        if not residual:
            assert torch.equal(out.cpu() == 0, (f == 0) | (x == 0))


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_dropped_infinities_are_zero_and_kept_ones_pass(moe, t):
    x = torch.full((64, 64), float("inf"), dtype=t)
    x[1::2] = float("nan")
    out = torch.empty_like(x, device=DEV)
    moe.moe_dropout(_type(moe, t), x.to(DEV), 0.3, _rng(4, 4), out)
    keep = pl.factors(64 * 64, 0.3, 4, 4).view(64, 64) > 0
    want = torch.where(keep, x, torch.zeros((), dtype=t))
    assert torch.equal(torch.nan_to_num(out.cpu(), nan=-1.0), torch.nan_to_num(want, nan=-1.0))


def test_in_place_and_residual_in_place(moe):
    x, res = _rand(1, torch.bfloat16, 33, 64).to(DEV), _rand(2, torch.bfloat16, 33, 64).to(DEV)
    want = torch.empty_like(x)
    moe.moe_dropout(moe.MOE_BF16, x, 0.2, _rng(1, 2), want, residual=res)
    a, b = x.clone(), res.clone()
    moe.moe_dropout(moe.MOE_BF16, a, 0.2, _rng(1, 2), a, residual=res)
    moe.moe_dropout(moe.MOE_BF16, x, 0.2, _rng(1, 2), b, residual=b)
    assert torch.equal(a, want) and torch.equal(b, want)


def test_past_32_bits(moe):
    """More than 2^32 elements: the element number's upper bits reach the generator's counter and the addresses."""
    n = 2 ** 32 + 2 ** 20
    _say("elements", n)
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    moe.moe_dropout(moe.MOE_BF16, x, 0.25, _rng(8, 1), x)
    for first in (0, 2 ** 31 - 512, 2 ** 32 - 512, n - 1024):
        f = pl.factors(1024, 0.25, 8, 1, first=first)
        assert torch.equal(x[first:first + 1024].cpu(), f.to(torch.bfloat16)), first


CASES = [(1, 1, 8), (5, 3, 24), (64, 2, 2048), (300, 4, 128), (37, 8, 4096), (129, 5, 72)]


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,d", CASES)
def test_combine(moe, T, k, d, t):
    _say("combine", T, k, d, t)
    d = d if t is torch.bfloat16 else d - 4
    g = torch.Generator().manual_seed(T)
    n = T * k + 3
    y, res = _rand(1, t, n, d), _rand(2, t, T, d)
    dst = torch.randperm(n, generator=g)[:T * k].to(torch.int32)
    if T > 4:
        dst[::7] = -1
        dst[3 * k:4 * k] = -1                               # a token with no row at all
    w = torch.rand(T * k, generator=g)
    for p, weights, r in ((0.1, w, res), (0.5, None, None), (0.0, w, res), (0.3, w, None)):
        out = torch.full((T, d), float("nan"), dtype=t, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        moe.moe_combine_dropout(_type(moe, t), y.to(DEV), dst.to(DEV), None if weights is None else weights.to(DEV), k, p,
                                _rng(9, T) if p else None, out, residual=None if r is None else r.to(DEV), dev_err=err)
        terms = y.double()[dst.clamp(min=0).long()] * (dst >= 0).double()[:, None]
        terms = (terms * (1 if weights is None else weights.double()[:, None])).view(T, k, d)
        f = pl.factors(T * d, p, 9, T).view(T, d)
        rr = torch.zeros(T, d, dtype=torch.float64) if r is None else r.double()
        _check(out, terms.sum(1) * f + rr, terms.abs().sum(1) * f + rr.abs(), t, k + 3)
        assert int(err) == 0
        if r is not None:                                   # the residual's own buffer takes the result
            same = r.to(DEV)
            moe.moe_combine_dropout(_type(moe, t), y.to(DEV), dst.to(DEV), w.to(DEV), k, p, _rng(9, T) if p else None, same,
                                    residual=same)
            assert torch.equal(same, out)


def test_combine_without_dropout_is_the_plain_combine(moe):
    T, k, d = 200, 4, 256
    y, dst = _rand(1, torch.bfloat16, T * k, d).to(DEV), torch.randperm(T * k, dtype=torch.int32).to(DEV)
    w = torch.rand(T, k).to(DEV)
    a, b = torch.empty(T, d, dtype=torch.bfloat16, device=DEV), torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    moe.moe_unpermute_combine(moe.MOE_BF16, y, dst, w, k, a)
    moe.moe_combine_dropout(moe.MOE_BF16, y, dst, w, k, 0.0, None, b)
    assert torch.equal(a, b)


def test_combine_flags_rows_out_of_range(moe):
    y = torch.ones(4, 64, dtype=torch.bfloat16, device=DEV)
    dst = torch.tensor([0, 4, -1, 3], dtype=torch.int32, device=DEV)
    out, err = torch.empty(2, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_combine_dropout(moe.MOE_BF16, y, dst, None, 2, 0.0, None, out, dev_err=err)
    assert int(err) == moe.MOE_ERR_ROW_RANGE and bool((out == 1).all())


def test_backward_is_the_transpose(moe):
    """<dout, drop(x)> = <drop(dout), x> term by term: the factors are symmetric, so the two sums have the same terms."""
    x, dout = _rand(1, torch.float32, 100, 64).to(DEV), _rand(2, torch.float32, 100, 64).to(DEV)
    a, b = torch.empty_like(x), torch.empty_like(x)
    moe.moe_dropout(moe.MOE_F32, x, 0.4, _rng(5, 6), a)
    moe.moe_dropout(moe.MOE_F32, dout, 0.4, _rng(5, 6), b)
    torch.testing.assert_close(dout.double() * a.double(), b.double() * x.double(), rtol=2.0 ** -21, atol=0)


def test_replays_draw_new_masks(moe):
    """A captured call reads seed and step when it runs."""
    x, out, rng = torch.ones(64, 64, device=DEV), torch.empty(64, 64, device=DEV), _rng(11, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_dropout(moe.MOE_F32, x, 0.5, rng, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_dropout(moe.MOE_F32, x, 0.5, rng, out)
        rng[1].add_(1)
    for step in range(4):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu().double(), pl.factors(64 * 64, 0.5, 11, step).view(64, 64)), step
