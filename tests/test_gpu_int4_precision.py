"""What 4-bit integer experts keep of h between their products: eleven significant bits, whatever its size, so that an
output is off by its own rounding and little more."""
import pytest
import torch

from tests import _plain_gated as pl
from tests.test_gpu_int4 import GATE, Ffn, _say, moe  # noqa: F401  (moe: the fixture)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
E, K = 8, 2
# slot by slot, tiles of 16 rows, tiles of 64 rows (with 8 experts of 2 slots)
FORMS = [1, 5, 40, 200]


def _bound(c):
    """want [T, d] in 64 bits, and how far what is rounded to the output may be from it.  h: fp16's half step 2^-11 of
    each element, and 2^-24 / 2^7 of the row's largest where that leaves the smallest of them none; a group's sum of h has
    parts below 2^-24 / 2^7 of the row's largest cut off, times at most 31.  The fp32 sums as in Ffn._mm, the gates' GATE."""
    x, f, group = c.x.double(), c.f, c.group
    want = torch.zeros(c.T, c.d, dtype=torch.float64)
    off = torch.zeros_like(want)
    for e in range(c.E):
        t, j = torch.nonzero(c.route["topk_idx"] == e, as_tuple=True)
        if not t.numel():
            continue
        gu, dg = c._mm(x[t], 0, e)
        g, u = pl.limited(gu[:, :f], gu[:, f:], c.limit)
        lg, lu = pl.limited(gu[:, :f] - dg[:, :f], gu[:, f:].abs() - dg[:, f:], c.limit)
        dgl, dul = (g - lg).clamp(min=0), (u.abs() - lu.abs()).clamp(min=0)     # (nothing where the limit holds both)
        if not c.limit:
            dgl, dul = dg[:, :f], dg[:, f:]
        a = pl.act(c.act, g)
        h = a * u
        dh = 1.13 * dgl * (u.abs() + dul) + a.abs() * dul + (GATE if c.act != "relu" else 2.0 ** -23) * h.abs()
        largest = h.abs().amax(1, keepdim=True)
        dh = dh * (1 + 2.0 ** -11) + 2.0 ** -11 * h.abs() + 2.0 ** -32 * largest
        y, dy = c._mm(h, 1, e)
        w, s = c.values(1, e)
        dy = dy * 1.01 + dh @ w.abs().t() + 31 * 2.0 ** -31 * largest * s[:, ::group].sum(1)
        cw = c.route["topk_w"].double()[t, j][:, None]
        want.index_add_(0, t, cw * y)
        off.index_add_(0, t, cw * (dy + 2.0 ** -20 * y.abs()))
    return want, off


def _close(out, want, off):
    """A value within `off` of want, rounded to bf16: as far from want as its own rounding, and at most twice `off` more (a
    value on the other side of a midpoint rounds the other way, where want is within `off` of the midpoint)."""
    err = (out.double() - want).abs()
    own = (want.to(BF).double() - want).abs()
    assert bool((err <= own + 2 * off + 1e-35).all()), float(((err - own) / (off + 1e-35)).max())


def _positive(c):
    """Weights of the down product that are all positive (codes 9..15, zero 8): errors of one sign in h add up."""
    codes, s, _ = c.w[1]
    codes = codes | 0x88
    codes = codes | torch.where(codes & 0x07 == 0, 0x01, 0) | torch.where(codes & 0x70 == 0, 0x10, 0)
    c.w[1] = (codes.to(torch.uint8), s, None)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("act,limit", [("relu", (1 + 2.0 ** -8 + 2.0 ** -11) ** 0.5), ("silu", 1.5), ("gelu", 1.5),
                                       ("gelu_tanh", 1.5)])
@pytest.mark.parametrize("T", FORMS)
def test_clamped_gates(moe, T, act, limit, group):  # noqa: F811
    """Every g and u past the limit: all elements of h are one number, L^2 = 1 + 2^-8 + 2^-11 with relu, which bf16 would
    round by 3e-3 and with it every output."""
    _say("clamped", T, act, group)
    c = Ffn(moe, T, E, 256, 256, K, group, False, act=act, limit=limit, seed=T, x=torch.ones(T, 256))
    codes, s, _ = c.w[0]
    c.w[0] = (torch.full_like(codes, 0xFF), torch.full_like(s, 1.0), None)
    _positive(c)
    want, off = _bound(c)
    assert float((off / want.abs()).max()) < 2.0 ** -10     # (far below the bf16 step of h: this is what the test is for)
    _close(c.run(), want, off)


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("act,limit", [("relu", 0.0), ("gelu", 1.5), ("silu", 0.0)])
@pytest.mark.parametrize("T", FORMS)
def test_random_rows(moe, T, act, limit, group, zeros):  # noqa: F811
    c = Ffn(moe, T, E, 384, 128, K, group, zeros, act=act, limit=limit, seed=T)
    _close(c.run(), *_bound(c))


@pytest.mark.parametrize("T", FORMS)
def test_rows_of_any_size(moe, T):  # noqa: F811
    """Tokens from 2^-40 to 2^40 (with relu h from 2^-80 to 2^80), and tokens of zeros: each to its own size."""
    c = Ffn(moe, T, E, 256, 160, K, 32, True, act="relu", seed=3)
    p = torch.linspace(-40, 40, T).round() if T > 1 else torch.tensor([-40.0])
    c.x = (c.x.float() * torch.exp2(p)[:, None]).to(BF)
    if T > 4:
        c.x[3] = 0
    out = c.run()
    _close(out, *_bound(c))
    assert T <= 4 or not bool(out[3].any())


@pytest.mark.parametrize("step", [1, 2, 3])
@pytest.mark.parametrize("T", FORMS)
def test_rows_of_elements_of_many_sizes(moe, T, step):  # noqa: F811
    """The up product's rows fall by 2^-step from one 32 columns of h to the next, the down product's scales grow by as
    much: the smallest elements, 2^-21 of a row's largest, count as much as that."""
    c = Ffn(moe, T, E, 128, 256, K, 32, False, act="relu", seed=8)
    f = c.f
    fall = torch.exp2(-step * (torch.arange(f) // 32).float())
    codes, s, _ = c.w[0]
    s = s.clone()
    s[:, f:] = (s[:, f:].float() * fall[None, :, None]).to(BF)
    c.w[0] = (codes, s, None)
    codes, s, _ = c.w[1]
    c.w[1] = (codes, (s.float() / fall[::32][None, None, :]).to(BF), None)
    _close(c.run(), *_bound(c))


@pytest.mark.parametrize("T", FORMS)
def test_infinite_and_nan_h_stay_in_their_rows(moe, T):  # noqa: F811
    """g u past fp32's largest number: that token is not finite, the others are as without it."""
    c = Ffn(moe, T, E, 128, 128, K, 64, False, act="relu", seed=2)
    clean = c.run()
    at = T // 2
    c.x[at] = (c.x[at].float().sign() * 2.0 ** 66).to(BF)
    out = c.run()
    rest = torch.arange(T) != at
    assert torch.equal(out[rest], clean[rest]) and not bool(torch.isfinite(out[at]).any())


def test_long_rows_of_h(moe):  # noqa: F811
    """Rows longer than the threads that look for their largest element: it is the last one, the first one, one between."""
    for f, T in ((480, 20), (512, 300), (1984, 20), (2080, 300), (8128, 20), (8256, 40)):
        f = -(-f // 32) * 32
        c = Ffn(moe, T, 2, 64, f, 1, 32, False, act="relu", seed=f)
        codes, s, _ = c.w[0]
        s = s.clone()
        for e, col in ((0, f - 1), (1, 0)):
            s[e, f + col] = (s[e, f + col].float() * 2.0 ** 18).to(BF)
        s[0, f + f // 2 + 1] = (s[0, f + f // 2 + 1].float() * 2.0 ** 10).to(BF)
        c.w[0] = (codes, s, None)
        _close(c.run(), *_bound(c))
