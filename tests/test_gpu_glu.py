"""Gated blocks of every gate, with a limit and dropout, forward and backward: each stage against its formula in 64
bits on the very tensors that the stage read, so that a bound holds for one stage's roundings alone."""
import sys

import pytest
import torch

from tests import _plain_gated as pl

pytestmark = pytest.mark.gpu
DEV = "cuda"
# relative error of a gate and of each term of its slope: fp32 from the mathematical library (a few 2^-24, and 2^-23
# times the argument of exp, at most 100), bf16 from the hardware's exp2 and reciprocal and a polynomial of 1e-6
GATE = {torch.float32: 2.0 ** -16, torch.bfloat16: 2.0 ** -14}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# Where 1 / (1 + exp(-z)) is below fp32's smallest normal number 2^-126 it may come out as 0: a gate g s is then off by up
# to 2^-126 |g|, a slope s (1 + g (1 - s) dz/dg), with dz/dg at most 1.6 + 0.22 * 144 < 2^6, by up to 2^-120 (1 + |g|).
# (The bound was relative alone at first, and a product dh u s of s = 1e-39 and |dh u| = 2e4 came out as 0.)
TINY = 2.0 ** -120


def _say(*a):
    print("[gpu-glu]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


def _within(name, got, want, tol):
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol + 1e-35).all()), (name, float((err / (tol + 1e-35)).max()))


def _mm(a, b):
    """a @ b in 64 bits, and the bound of its fp32 sum: a rounding of at most 2^-23 of the sum of the magnitudes for each
    of the K additions (the matrix unit may cut off rather than round)."""
    return a @ b, (a.shape[1] + 4) * 2.0 ** -23 * (a.abs() @ b.abs())


class Block:
    """Inputs of one block of E experts on the CPU in 64 bits and on the device, and its outputs."""

    def __init__(self, moe, counts, d, f, t, act, limit, p, seed=1, capacity=0, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        E, self.d, self.f, self.t = len(counts), d, f, t
        self.limit, self.act, self.p, self.moe, self.capacity = limit, act, p, moe, capacity
        self.dt = moe.MOE_F32 if t is torch.float32 else moe.MOE_BF16
        self.cuts = [e * capacity for e in range(E + 1)] if capacity else [0] + torch.tensor(counts).cumsum(0).tolist()
        R = self.R = self.cuts[-1] + (0 if capacity else 5)  # rows behind the last group, left as they are
        self.rng = (977 + seed, 2 ** 33 + seed)
        dev = {}
        for n, shape, s in (("x", (R, d), scale), ("w13", (E, 2 * f, d), 1.2 / d ** 0.5), ("w2", (E, d, f), 1 / f ** 0.5),
                            ("dy", (R, d), 1.0)):
            dev[n] = (torch.randn(*shape, generator=g) * s).to(t).to(DEV)
        for n, shape in (("gu", (R, 2 * f)), ("h", (R, f)), ("y", (R, d)), ("dgu", (R, 2 * f)), ("dx", (R, d)),
                         ("dw13", (E, 2 * f, d)), ("dw2", (E, d, f))):
            dev[n] = torch.full(shape, 7.0, dtype=t, device=DEV)
        self.dev = dev
        self.off = torch.tensor(self.cuts, dtype=torch.int32, device=DEV)
        self.ws = torch.empty(max(moe.moe_gemm_workspace_bytes(self.dt, E, R, d, f), 16), dtype=torch.uint8, device=DEV)
        rng = torch.tensor(self.rng, dtype=torch.int64, device=DEV)
        self.gate = moe.glu(pl.ACTS.index(act), limit, p, rng if p else None)

    def forward(self):
        v = self.dev
        self.moe.moe_grouped_glu_fwd(self.dt, self.gate, v["x"], v["w13"], v["w2"], self.off, self.capacity, v["gu"],
                                     v["h"], v["y"])

    def backward(self):
        v = self.dev
        self.moe.moe_grouped_glu_bwd(self.dt, self.gate, v["dy"], v["x"], v["gu"], v["h"], v["w13"], v["w2"], self.off,
                                     self.capacity, v["dgu"], v["dx"], v["dw13"], v["dw2"], ws=self.ws)

    def check(self):
        torch.cuda.synchronize()
        v = {n: w.cpu().double() for n, w in self.dev.items()}
        f, t, end = self.f, self.t, self.cuts[-1]
        half, rel = HALF[t], GATE[t]
        fac = pl.factors(self.R * f, self.p, *self.rng).view(self.R, f)
        for e, (a, b) in enumerate(zip(self.cuts[:-1], self.cuts[1:])):
            r = slice(a, b)
            w13, w2, fc = v["w13"][e], v["w2"][e], fac[r]
            # gu, and h from the unrounded g and u
            gu, tol = _mm(v["x"][r], w13.t())
            _within("gu", self.dev["gu"][r], gu, half * gu.abs() + tol * (1 + half))
            g, u = pl.limited(gu[:, :f], gu[:, f:], self.limit)
            ac = pl.act(self.act, g)
            # a slope is at most 1.13 for any of the gates
            spread = 1.13 * tol[:, :f] * (u.abs() + tol[:, f:]) + ac.abs() * tol[:, f:] + rel * (ac * u).abs() + TINY * (g * u).abs()
            _within("h", self.dev["h"][r], fc * ac * u, half * fc * (ac * u).abs() + fc * spread * 1.01)
            assert bool((v["h"][r][fc == 0] == 0).all())
            # y from the stored h; dh, dgu from the stored gu
            y, tol = _mm(v["h"][r], w2.t())
            _within("y", self.dev["y"][r], y, half * y.abs() + tol * 1.01)
            dh, tol = _mm(v["dy"][r], w2)
            g0, u0 = v["gu"][r][:, :f], v["gu"][r][:, f:]
            g, u = pl.limited(g0, u0, self.limit)
            ac, terms = pl.act(self.act, g), pl.slope_terms(self.act, g)
            sl, sl_size = sum(terms), sum(s.abs() for s in terms)
            L = self.limit or float("inf")
            on_g, on_u = fc * (g0 <= L), fc * (u0.abs() <= L)
            dg, du = dh * u * sl * on_g, dh * ac * on_u
            tg = on_g * ((tol * sl.abs() + rel * dh.abs() * sl_size + TINY * dh.abs() * (1 + g.abs())) * u.abs()) * 1.01
            tu = on_u * ((tol + rel * dh.abs()) * ac.abs() + TINY * (dh * g).abs()) * 1.01
            _within("dg", self.dev["dgu"][r][:, :f], dg, half * dg.abs() + tg)
            _within("du", self.dev["dgu"][r][:, f:], du, half * du.abs() + tu)
            # the products of the stored dgu
            dx, tol = _mm(v["dgu"][r], w13)
            _within("dx", self.dev["dx"][r], dx, half * dx.abs() + tol * 1.01)
            dw, tol = _mm(v["dgu"][r].t(), v["x"][r])
            _within("dw13", self.dev["dw13"][e], dw, half * dw.abs() + tol * 1.01)
            dw, tol = _mm(v["dy"][r].t(), v["h"][r])
            _within("dw2", self.dev["dw2"][e], dw, half * dw.abs() + tol * 1.01)
        for n in ("gu", "h", "y", "dgu", "dx"):
            assert bool((v[n][end:] == 7).all()), f"{n}: rows behind the last group were written"


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("limit,p", [(0.0, 0.0), (1.0, 0.0), (0.0, 0.3), (1.5, 0.1)])
@pytest.mark.parametrize("act", pl.ACTS)
@pytest.mark.parametrize("t", [BF, F32])
def test_gates(moe, t, act, limit, p):
    _say(t, act, limit, p)
    b = Block(moe, [37, 0, 1, 70], 72, 136, t, act, limit, p)
    b.forward()
    b.backward()
    b.check()


@pytest.mark.parametrize("counts,d,f", [([1], 8, 8), ([0, 0, 3], 64, 24), ([64, 65, 63], 64, 128), ([128, 129], 128, 256),
                                        ([256, 300, 5], 192, 264), ([513], 256, 320)])
def test_tiles(moe, counts, d, f):
    """Row counts at and beside every tile height, K with and without a tail, columns that end inside tiles."""
    _say(counts, d, f)
    b = Block(moe, counts, d, f, BF, "gelu", 1.5, 0.2, seed=len(counts))
    b.forward()
    b.backward()
    b.check()


def test_padded_layout(moe):
    b = Block(moe, [0] * 3, 64, 64, BF, "gelu_tanh", 0.0, 0.1, capacity=40)
    b.forward()
    b.backward()
    b.check()


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("act", pl.ACTS)
def test_far_arguments(moe, act, t):
    """Gates from -infinity's side to infinity's: |g| up to a few hundred, where exponentials over- and underflow."""
    b = Block(moe, [40, 25], 64, 64, t, act, 0.0, 0.0, scale=100.0)
    b.forward()
    b.backward()
    b.check()


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("act", range(4))
def test_huge_finite_gates(moe, act, t):
    """g of 1e20 and -1e20: a(g) is g or 0 and the slopes 1 or 0, with no NaN from an overflow on the way."""
    R, n = 4, 8
    x = torch.zeros(R, n)
    x[:, 0] = torch.tensor([1.0, -1.0, 1.0, -1.0])
    w13 = torch.zeros(1, 2 * n, n)
    w13[0, :n, 0], w13[0, n:, 0] = 1e20, torch.tensor([1.0, -1.0] * 4)
    w2 = torch.eye(n)[None]
    v = {k: w.to(t).to(DEV) for k, w in dict(x=x, w13=w13, w2=w2, dy=torch.ones(R, n)).items()}
    o = {k: torch.empty(R, c, dtype=t, device=DEV) for k, c in dict(gu=2 * n, h=n, y=n, dgu=2 * n, dx=n).items()}
    dw13, dw2 = torch.empty_like(v["w13"]), torch.empty_like(v["w2"])
    off, ws = torch.tensor([0, R], dtype=torch.int32, device=DEV), torch.empty(256, dtype=torch.uint8, device=DEV)
    dt, gate = (moe.MOE_F32 if t is F32 else moe.MOE_BF16), moe.glu(act, limit=1e30)
    moe.moe_grouped_glu_fwd(dt, gate, v["x"], v["w13"], v["w2"], off, 0, o["gu"], o["h"], o["y"])
    moe.moe_grouped_glu_bwd(dt, gate, v["dy"], v["x"], o["gu"], o["h"], v["w13"], v["w2"], off, 0, o["dgu"], o["dx"], dw13,
                            dw2, ws=ws)
    g, u = o["gu"][:, :n].cpu().double(), o["gu"][:, n:].cpu().double()
    want = torch.where(g > 0, g * u, 0.0)
    assert torch.equal(o["h"].cpu().double(), want)
    assert torch.equal(o["dgu"][:, :n].cpu().double(), torch.where(g > 0, u, 0.0))
    assert torch.equal(o["dgu"][:, n:].cpu().double(), torch.where(g > 0, g, 0.0))


@pytest.mark.parametrize("t", [BF, F32])
def test_limits_themselves_have_slope_one(moe, t):
    """g and u exactly at the limit pass their gradient, beyond it none; a NaN passes through."""
    n = 8
    gu = torch.tensor([[2.0, 2.5, -2.0, -2.5, 2.0, 1.0, 1.0, float("nan")],
                       [1.0, 1.0, 1.0, 1.0, 2.0, -2.0, 2.5, 1.0]]).reshape(1, 16)
    w2, dy = torch.eye(n)[None].to(t).to(DEV), torch.ones(1, n, dtype=t, device=DEV)
    guv, dgu, off = gu.to(t).to(DEV), torch.empty(1, 16, dtype=t, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    tens = moe.gemm_tensors(dy_perm=dy, w2=w2, gu=guv, dgu=dgu)
    moe.moe_grouped_glu_op(moe.MOE_GEMM_DGRAD_DOWN, moe.MOE_F32 if t is F32 else moe.MOE_BF16,
                           moe.glu(moe.MOE_ACT_RELU, limit=2.0), tens, off, 0, 1, 1, n, n)
    dg, du = dgu.cpu().float()[0, :n], dgu.cpu().float()[0, n:]
    assert dg[:7].tolist() == [1.0, 0.0, 0.0, 0.0, 2.0, -2.0, 2.0]
    assert du[:7].tolist() == [2.0, 2.0, 0.0, 0.0, 2.0, 1.0, 0.0] and bool(torch.isnan(du[7]))


def test_dropped_nan_and_infinity_leave_zeros(moe):
    """Rows of infinities and NaN: dropped elements of h and of its gradients are 0."""
    b = Block(moe, [16], 64, 64, BF, "silu", 0.0, 0.5)
    b.dev["x"][3] = float("nan")
    b.dev["x"][5] = float("inf")
    b.forward()
    b.dev["dy"][4] = float("nan")
    b.backward()
    out = pl.factors(b.R * 64, 0.5, *b.rng).view(b.R, 64)[:16] == 0
    assert bool((b.dev["h"][:16].cpu()[out] == 0).all())
    assert bool((b.dev["dgu"][:16, :64].cpu()[out] == 0).all()) and bool((b.dev["dgu"][:16, 64:].cpu()[out] == 0).all())
    assert bool(torch.isnan(b.dev["h"][3].cpu()[~out[3]]).all()) and bool(torch.isnan(b.dev["dgu"][4].float()).any())


@pytest.mark.parametrize("t", [BF, F32])
def test_the_plain_form_is_the_swiglu_call(moe, t):
    """silu, no limit, p = 0: bit for bit moe_grouped_gemm_fwd and _bwd."""
    b = Block(moe, [70, 300, 0, 9], 128, 192, t, "silu", 0.0, 0.0)
    b.forward()
    b.backward()
    mine = {n: b.dev[n].clone() for n in ("gu", "h", "y", "dgu", "dx", "dw13", "dw2")}
    v = b.dev
    moe.moe_grouped_gemm_fwd(b.dt, v["x"], v["w13"], v["w2"], b.off, 0, v["gu"], v["h"], v["y"])
    moe.moe_grouped_gemm_bwd(b.dt, v["dy"], v["x"], v["gu"], v["h"], v["w13"], v["w2"], b.off, 0, v["dgu"], v["dx"],
                             v["dw13"], v["dw2"], ws=b.ws)
    for n, w in mine.items():
        assert torch.equal(w, v[n]), n


@pytest.mark.parametrize("act", pl.ACTS)
def test_gradient_against_differences(moe, act):
    """fp32: <dy, y> along a random direction of x and of the weights.  The direction's second and third derivatives are
    of order 1, so a step of 2^-6 leaves 2^-12 of them, and the fp32 sums of about 1e3 terms 2^-24 * 1e3 / 2^-6 = 2^-8 of
    one term; relu has kinks, each within a step of them for a share of 2^-6 of the units."""
    t, step = F32, 2.0 ** -6
    b = Block(moe, [20, 12], 64, 64, t, act, 0.0, 0.2)
    b.forward()
    b.backward()
    v = b.dev
    grads = {"x": v["dx"].clone(), "w13": v["dw13"].clone(), "w2": v["dw2"].clone()}
    for n in ("x", "w13", "w2"):
        g = torch.Generator().manual_seed(3)
        way = torch.randn(v[n].shape, generator=g).to(DEV) * v[n][:20].std()
        if n == "x":
            way[32:] = 0
        at, vals = v[n].clone(), []
        for s in (step, -step):
            v[n].copy_(at + s * way)
            b.forward()
            vals.append(float((v["y"][:32].double() * v["dy"][:32].double()).sum()))
        v[n].copy_(at)
        got = float((grads[n][:32].double() * way[:32].double()).sum())
        size = float((grads[n][:32].double() * way[:32].double()).square().sum().sqrt())
        assert abs((vals[0] - vals[1]) / (2 * step) - got) <= (0.05 if act != "relu" else 0.25) * size, n


def test_two_streams_at_once(moe):
    """Blocks with different gates and masks, launched on two streams without a wait between: each as alone."""
    bs = [Block(moe, [300, 200], 128, 256, BF, a, 0.0, p, seed=s) for a, p, s in (("gelu", 0.1, 4), ("relu", 0.4, 5))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for b, s in zip(bs, streams):
            with torch.cuda.stream(s):
                b.forward()
                b.backward()
    torch.cuda.synchronize()
    for b in bs:
        b.check()


@pytest.mark.parametrize("d,f", [(64, 5120), (5120, 64)])
def test_tiles_of_large_launches(moe, d, f):
    """Enough tiles for the tallest ones, with every height of a group's last one."""
    _say("large", d, f)
    b = Block(moe, [300, 64, 128, 513, 0, 40], d, f, BF, "gelu_tanh", 1.5, 0.2, seed=6)
    b.forward()
    b.backward()
    b.check()


@pytest.mark.parametrize("d,f", [(512, 1024), (1024, 448), (448, 1152)])
@pytest.mark.parametrize("plain", [False, True])
def test_a_group_alone_has_the_same_bits(moe, d, f, plain):
    """The height of a launch's tiles changes no bit: a group by itself, and sixteen times over."""
    m, E, n = moe, 16, 333
    _say("alone", d, f, plain)
    g = torch.Generator(DEV).manual_seed(3)

    def make(*shape, s=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * s).to(BF)
    one = dict(x_perm=make(n, d), dy_perm=make(n, d), w13=make(1, 2 * f, d, s=d ** -0.5), w2=make(1, d, f, s=f ** -0.5))
    gate = m.glu() if plain else m.glu(m.MOE_ACT_GELU, 1.0)      # (a mask is the row's, and these are other rows)
    outs = []
    for reps in (1, E):
        t = {k: v.repeat(reps, *[1] * (v.dim() - 1)).contiguous() for k, v in one.items()}
        R = n * reps
        t.update({k: torch.full((R, w), 7.0, dtype=BF, device=DEV)
                  for k, w in (("gu", 2 * f), ("h", f), ("y_perm", d), ("dgu", 2 * f), ("dx_perm", d))})
        off = torch.arange(0, R + 1, n, dtype=torch.int32, device=DEV)
        args = m.gemm_tensors(**t)
        for op in (m.MOE_GEMM_GATE_UP, m.MOE_GEMM_DOWN, m.MOE_GEMM_DGRAD_DOWN, m.MOE_GEMM_DGRAD_GATE_UP):
            if plain:
                m.moe_grouped_gemm_op(op, m.MOE_BF16, args, off, 0, reps, R, d, f)
            else:
                m.moe_grouped_glu_op(op, m.MOE_BF16, gate, args, off, 0, reps, R, d, f)
        outs.append(t)
    torch.cuda.synchronize()
    for k in ("gu", "h", "y_perm", "dgu", "dx_perm"):
        a, b = outs[0][k], outs[1][k].view(E, n, -1)
        assert bool((a == b).all()), k
