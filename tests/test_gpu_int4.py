"""4-bit integer experts: the quantiser and its inverse bit for bit, the feed-forward against 64-bit sums of the very
codes within a bound from its roundings, probes that read single weights out, routes with dropped and foreign slots."""
import sys

import numpy as np
import pytest
import torch

from tests import _plain_gated as pl

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
GATE = 2.0 ** -14       # relative error of a gate (hardware exp2 and reciprocal, a polynomial of 1e-6)


def _say(*a):
    print("[gpu-int4]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


def _quantize(moe, w, group, zeros):
    rows, K = w.shape
    codes = torch.full((rows, K // 2), 0x77, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, K // group), 3.0, dtype=BF, device=DEV)
    z = torch.full((rows, K // group), 99, dtype=torch.uint8, device=DEV) if zeros else None
    moe.moe_quantize_int4(w.to(DEV), group, codes, scales, z)
    return codes, scales, z


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,groups", [(1, 1), (3, 5), (130, 9), (1031, 2)])
def test_quantizer_bit_exact(moe, rows, groups, group, zeros):
    _say("quantise", rows, groups, group, zeros)
    K = group * groups
    g = torch.Generator().manual_seed(rows + group)
    w = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    w = w.to(BF)
    w[0, :group] = 0                                        # an empty group
    if rows > 2:
        w[1, :group] = w[1, :group].abs()                   # one sign only: the zero point at an end
        w[2, :group] = -w[2, :group].abs()
    if rows > 100:
        w[3, :group] = torch.linspace(-7.5, 7.5, group).to(BF)            # ties
        w[4, :group] = torch.tensor([0.5, 1.5, 2.5, 7.0] * (group // 4)).to(BF)
        w[5, :group] = torch.tensor([-8.0, 7.0] * (group // 2)).to(BF)
        w[6, 0] = float("nan")
        w[7, group - 1] = float("-inf")
        w[8, :group] = 1e-39                                # below the smallest scale
        w[9, :group] = torch.tensor([3.3e38, -3.3e38] * (group // 2)).to(BF)
        w[10, :group] = torch.tensor([1e-30, 1e30] * (group // 2)).to(BF)
    codes, scales, z = _quantize(moe, w, group, zeros)
    q, s, zz = pl.int4_quantize(w.double().numpy(), group, zeros)
    assert torch.equal(codes.cpu(), torch.from_numpy(pl.int4_pack(q)))
    assert np.array_equal(scales.cpu().double().numpy(), s, equal_nan=True)
    if zeros:
        assert torch.equal(z.cpu(), torch.from_numpy(zz))
    back = torch.full((rows, K), 5.0, dtype=BF, device=DEV)
    moe.moe_dequantize_int4(codes, scales, z, group, back)
    want = torch.from_numpy(pl.int4_values(q, s, zz, group)).float().to(BF)   # 12 bits: exact in fp32
    assert torch.equal(torch.nan_to_num(back.cpu(), nan=-77.0), torch.nan_to_num(want, nan=-77.0))


def test_codec_of_no_rows(moe):
    moe.moe_quantize_int4(torch.empty(0, 64, dtype=BF, device=DEV), 32, torch.empty(0, 32, dtype=torch.uint8, device=DEV),
                          torch.empty(0, 2, dtype=BF, device=DEV))
    moe.moe_dequantize_int4(torch.empty(0, 32, dtype=torch.uint8, device=DEV), torch.empty(0, 2, dtype=BF, device=DEV), None,
                            32, torch.empty(0, 64, dtype=BF, device=DEV))


def test_codec_past_32_bits(moe):
    """More than 2^32 elements: the last rows are those of a quantiser of their own."""
    rows, K = (1 << 20) + 96, 4096
    w = torch.empty(rows, K, dtype=BF, device=DEV)
    for a in range(0, rows, 1 << 18):
        w[a:a + (1 << 18)].normal_(generator=torch.Generator(DEV).manual_seed(a + 1))
    codes, scales, z = _quantize(moe, w, 128, True)
    c2, s2, z2 = _quantize(moe, w[-100:], 128, True)
    assert torch.equal(codes[-100:], c2) and torch.equal(scales[-100:], s2) and torch.equal(z[-100:], z2)
    moe.moe_dequantize_int4(codes, scales, z, 128, w)
    back = torch.empty(100, K, dtype=BF, device=DEV)
    moe.moe_dequantize_int4(c2, s2, z2, 128, back)
    assert torch.equal(w[-100:], back)


# ------------------------------------------------------------------ the feed-forward
def _route(T, E, k, seed, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) - skew * torch.arange(E)
    top = torch.topk(logits, k, dim=1)
    idx = top.indices.reshape(-1)
    order = torch.argsort(idx, stable=True)
    dst = torch.empty_like(order)
    dst[order] = torch.arange(T * k)
    off = torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(idx, minlength=E).cumsum(0)])
    return dict(topk_idx=top.indices.int(), topk_w=torch.softmax(top.values, 1), dst_row=dst.int(), src_slot=order.int(),
                group_off=off.int())


class Ffn:
    def __init__(self, moe, T, E, d, f, k, group, zeros, act="silu", limit=0.0, seed=0, skew=0.0, x=None):
        g = torch.Generator().manual_seed(seed)
        self.moe, self.group, self.act, self.limit = moe, group, act, limit
        self.T, self.E, self.d, self.f, self.k = T, E, d, f, k
        self.x = (torch.randn(T, d, generator=g) + 0.3).to(BF) if x is None else x.to(BF)   # a mean: long sums of x
        self.route = _route(T, E, k, seed, skew)
        self.w = []
        for N, K in ((2 * f, d), (d, f)):
            codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)     # every code, every zero point
            scales = (torch.rand(E, N, K // group, generator=g) * 0.3 / K ** 0.5).to(BF)
            z = torch.randint(0, 16, (E, N, K // group), generator=g, dtype=torch.uint8) if zeros else None
            self.w.append((codes, scales, z))

    def run(self, **over):
        r = {n: t.to(DEV) for n, t in self.route.items()}
        w13, w2 = (tuple(None if t is None else t.to(DEV) for t in w) for w in self.w)
        ws = torch.full((self.moe.moe_int4_workspace_bytes(self.T * self.k, self.d, self.f),), 0xFF, dtype=torch.uint8,
                        device=DEV)                        # NaN in every type: nothing is read before it is written
        out = torch.full((self.T, self.d), float("nan"), dtype=BF, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.moe.moe_int4_ffn(self.moe.glu(pl.ACTS.index(self.act), self.limit), self.x.to(DEV), r["topk_idx"], r["topk_w"],
                              r["dst_row"], r["src_slot"], r["group_off"], self.group, w13, w2, out, ws, dev_err=self.err)
        torch.cuda.synchronize()
        return out.cpu()

    def values(self, which, e):
        codes, s, z = self.w[which]
        q = torch.stack([codes[e] & 15, codes[e] >> 4], -1).view(codes.shape[1], -1).double()
        z = 8.0 if z is None else z[e].double().repeat_interleave(self.group, 1)
        return (q - z) * s[e].double().repeat_interleave(self.group, 1), s[e].double().repeat_interleave(self.group, 1)

    def _mm(self, x, which, e):
        """x W^T in 64 bits and the bound of its fp32 sums: within a group |x| (16 + q) and (16 + z) |x| are at most 31 |x|,
        each summed with group + 4 roundings of 2^-23, and scaled; then the groups' sums."""
        w, s = self.values(which, e)
        n = w.shape[1] // self.group
        return x @ w.t(), 2.0 ** -23 * ((2 * 31 * (self.group + 4)) * (x.abs() @ s.t()) + (n + 12) * (x.abs() @ w.abs().t()))

    def check(self, out, live=None):
        x, f = self.x.double(), self.f
        want = torch.zeros(self.T, self.d, dtype=torch.float64)
        tol = torch.zeros_like(want)
        for e in range(self.E):
            hit = self.route["topk_idx"] == e
            if live is not None:
                hit = hit & live
            t, j = torch.nonzero(hit, as_tuple=True)
            if not t.numel():
                continue
            gu, dg = self._mm(x[t], 0, e)
            g, u = pl.limited(gu[:, :f], gu[:, f:], self.limit)
            a = pl.act(self.act, g)
            h = a * u
            dh = 1.13 * dg[:, :f] * (u.abs() + dg[:, f:]) + a.abs() * dg[:, f:] + GATE * h.abs()
            dh = dh + 2.0 ** -8 * (h.abs() + dh)            # h is stored in bf16
            y, dy = self._mm(h, 1, e)
            w = self.values(1, e)[0].abs()
            dy = dy * 1.01 + dh @ w.t()
            c = self.route["topk_w"].double()[t, j][:, None]
            want.index_add_(0, t, c * y)
            tol.index_add_(0, t, c * (dy + 2.0 ** -20 * y.abs()))
        err = (out.double() - want).abs()
        tol = tol + 2.0 ** -8 * want.abs() + 1e-35
        assert bool((err <= tol).all()), float((err / tol).max())
        # the bound adds every rounding up as if all had one sign; the roundings of h, y and out alone leave
        # 2^-8 / sqrt(3) of the size each, so twice their joint size is far from a lost or doubled group
        size = float(want.square().mean().sqrt())
        if size:
            assert float(err.square().mean().sqrt()) <= 2.0 ** -7 * 2 * size


SHAPES = [
    # T, E, d, f, k
    (1, 1, 32, 32, 1), (1, 8, 160, 96, 2), (1, 128, 512, 384, 8), (2, 4, 64, 96, 2), (3, 3, 288, 64, 3),
    (5, 64, 256, 256, 4), (17, 2, 128, 160, 1), (33, 1, 96, 128, 1), (40, 4, 1056, 32, 2), (67, 16, 512, 320, 4),
    (130, 3, 256, 224, 2), (300, 8, 192, 128, 4), (64, 1, 128, 128, 1), (65, 1, 128, 128, 1),
]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,E,d,f,k", SHAPES)
def test_ffn(moe, T, E, d, f, k, group, zeros):
    d, f = (-(-v // group) * group for v in (d, f))
    _say("ffn", T, E, d, f, k, group, zeros)
    c = Ffn(moe, T, E, d, f, k, group, zeros, act=pl.ACTS[(T + group) % 4], limit=2.0 if zeros else 0.0, seed=T)
    c.check(c.run())
    assert int(c.err) == 0


@pytest.mark.parametrize("T,E,d,f", [(1, 2, 4352, 64), (10, 2, 4352, 4480), (40, 1, 4352, 4224), (7, 200, 64, 64),
                                     (300, 1024, 128, 32)])
def test_long_rows_and_many_experts(moe, T, E, d, f):
    """Sums longer than a workgroup's share of one step, and more experts than lanes."""
    c = Ffn(moe, T, E, d, f, 1, 32, True, seed=T)
    c.check(c.run())


@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("T", [1, 20, 70])
def test_a_nan_scale_keeps_to_its_column(moe, T, group):
    """Rows that end inside a chunk of 128 codes: what follows is the next row's first group, whose NaN scale makes that
    row's column NaN and no other."""
    c = Ffn(moe, T, 2, 160 if group == 32 else 192, 160 if group == 32 else 192, 2, group, False, seed=6)
    clean = c.run()
    for e in range(2):
        c.w[1][1][e, 77, 0] = float("nan")
    out = c.run()
    keep = torch.arange(c.d) != 77
    assert torch.equal(out[:, keep], clean[:, keep]) and bool(torch.isnan(out[:, 77]).all())


@pytest.mark.parametrize("T", [1, 2, 90])
@pytest.mark.parametrize("act", pl.ACTS)
def test_gates(moe, act, T):
    c = Ffn(moe, T, 4, 256, 128, 2, 64, True, act=act, limit=1.0, seed=3)
    c.check(c.run())


@pytest.mark.parametrize("T", [60, 500])
def test_skewed_route_with_empty_experts(moe, T):
    c = Ffn(moe, T, 32, 128, 128, 2, 32, True, seed=5, skew=1.0)
    assert int((c.route["group_off"].diff() == 0).sum()) > 5
    c.check(c.run())


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("T", [1, 4, 70])
def test_single_weights_read_out(moe, T, group, zeros):
    """A token with one element reads one column of W13 out: relu(g) u of exact g and u, through a W2 that is the identity
    (code 9, zero 8, scale 1 on the diagonal), so the output is h but for the roundings of h, y and out (2^-8 each) and
    of the fp32 sums: h_c = sum h (16 + q) - 24 sum h over a group, either sum at most 25 sum |h| in group + 4 roundings of
    2^-23 (so not bit for bit, as first written here).  A misplaced code, scale or zero point of any lane, group or
    chunk shows."""
    E, d, f = 1, 384, 384
    for first in range(0, d, 47):
        col = [(first + 5 * t) % d for t in range(T)]
        x = torch.zeros(T, d)
        x[torch.arange(T), torch.tensor(col)] = 1.0
        c = Ffn(moe, T, E, d, f, 1, group, zeros, act="relu", seed=first, x=x)
        codes = torch.full((E, d, f), 8, dtype=torch.uint8)
        codes[0, torch.arange(d), torch.arange(f)] = 9
        c.w[1] = (codes[..., 0::2] | (codes[..., 1::2] << 4), torch.ones(E, d, f // group, dtype=BF),
                  torch.full((E, d, f // group), 8, dtype=torch.uint8) if zeros else None)
        out = c.run()
        w = c.values(0, 0)[0][:, torch.tensor(col)].t()
        want = w[:, :f].clamp(min=0) * w[:, f:]
        sums = want.abs().view(T, -1, group).sum(-1).repeat_interleave(group, 1)
        tol = 3.02 * 2.0 ** -8 * want.abs() + 50 * (group + 4) * 2.0 ** -23 * sums * 1.01
        assert bool(((out.double() - want).abs() <= tol).all()), first


def test_dropped_slots(moe):
    """Slots with dst_row < 0 add nothing, a token with none of its slots gets zeros."""
    for T in (1, 2, 50):
        c = Ffn(moe, T, 8, 128, 128, 3, 64, False, seed=2)
        live = torch.ones(T, 3, dtype=torch.bool)
        live[::2, 1] = False
        live[T // 2] = False
        dst = c.route["dst_row"].view(T, 3)
        dst[~live] = -1
        c.check(c.run(), live)
        assert int(c.err) == 0


@pytest.mark.parametrize("T", [1, 30])
def test_foreign_rows_are_flagged(moe, T):
    """A destination past the rows, and (one token) an expert past the experts: flagged, and their slots add nothing."""
    c = Ffn(moe, T, 8, 128, 128, 2, 64, False, seed=2)
    live = torch.ones(T, 2, dtype=torch.bool)
    live[0, 1] = False
    c.route["dst_row"][1] = T * 2 + 5
    c.check(c.run(), live)
    assert int(c.err) == moe.MOE_ERR_ROW_RANGE
    if T == 1:
        for bad in (8, -1, 2 ** 30):
            c = Ffn(moe, T, 8, 128, 128, 2, 64, False, seed=2)
            keep = c.route["topk_idx"].clone()
            c.route["topk_idx"][0, 1] = bad
            out = c.run()
            c.route["topk_idx"] = keep
            c.check(out, live)
            assert int(c.err) == moe.MOE_ERR_ROW_RANGE


def test_no_tokens(moe):
    c = Ffn(moe, 1, 4, 64, 64, 2, 32, False)
    c.T, c.x = 0, c.x[:0]
    c.route = {n: t[:0] if n != "group_off" else t * 0 for n, t in c.route.items()}
    assert c.run().shape == (0, 64)


def test_a_token_with_a_nan_or_an_infinity_keeps_to_itself(moe):
    for T in (20, 70):
        c = Ffn(moe, T, 2, 128, 128, 2, 64, False, seed=2)
        clean = c.run()
        c.x[3, 5], c.x[9, 100] = float("nan"), float("inf")
        out = c.run()
        rest = [t for t in range(T) if t not in (3, 9)]
        assert torch.equal(out[rest], clean[rest]) and bool(torch.isnan(out[[3, 9]]).all())


def test_codes_of_the_quantizer(moe):
    """The quantiser's own codes go through: the outputs are those of the dequantised weights in bf16 products, within
    the roundings of either."""
    T, E, d, f, k, group = 48, 4, 256, 128, 2, 64
    g = torch.Generator().manual_seed(8)
    c = Ffn(moe, T, E, d, f, k, group, True, seed=1)
    for i, (N, K) in enumerate(((2 * f, d), (d, f))):
        codes, s, z = _quantize(moe, (torch.randn(E * N, K, generator=g) / K ** 0.5).to(BF), group, True)
        c.w[i] = (codes.view(E, N, -1).cpu(), s.view(E, N, -1).cpu(), z.view(E, N, -1).cpu())
    c.check(c.run())


def test_streams_and_replays(moe):
    """Two calls on two streams with their own workspaces, and one captured: each replay bit for bit the eager call."""
    cs = [Ffn(moe, 24, 8, 256, 128, 2, 64, True, seed=4), Ffn(moe, 1, 8, 256, 128, 2, 128, False, seed=5),
          Ffn(moe, 200, 8, 256, 128, 2, 32, False, seed=6)]
    want = [c.run() for c in cs]
    args = []
    for c in cs:
        r = {n: t.to(DEV) for n, t in c.route.items()}
        w = [tuple(None if t is None else t.to(DEV) for t in w) for w in c.w]
        args.append((moe.glu(pl.ACTS.index(c.act), c.limit), c.x.to(DEV), r["topk_idx"], r["topk_w"], r["dst_row"],
                     r["src_slot"], r["group_off"], c.group, *w, torch.empty(c.T, c.d, dtype=BF, device=DEV),
                     torch.empty(moe.moe_int4_workspace_bytes(c.T * c.k, c.d, c.f), dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(4):
        for a, s in zip(args, streams):
            moe.moe_int4_ffn(*a, stream=s)
    torch.cuda.synchronize()
    for a, w in zip(args, want):
        assert torch.equal(a[-2].cpu(), w)
    for a, w in zip(args, want):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_int4_ffn(*a)
        for _ in range(3):
            a[-2].zero_()
            a[-1].fill_(0xFF)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(a[-2].cpu(), w)


@pytest.mark.parametrize("T", [30, 100])
@pytest.mark.parametrize("bad", [8, -1, 2 ** 30])
def test_foreign_experts_are_flagged_in_batches(moe, T, bad):
    """An expert past the experts, in the forms for many tokens: flagged, and its slot adds nothing."""
    c = Ffn(moe, T, 8, 128, 128, 2, 64, False, seed=2)
    live = torch.ones(T, 2, dtype=torch.bool)
    live[3, 1] = False
    keep = c.route["topk_idx"].clone()
    c.route["topk_idx"][3, 1] = bad
    out = c.run()
    c.route["topk_idx"] = keep
    c.check(out, live)
    assert int(c.err) == moe.MOE_ERR_ROW_RANGE


def _reroute(c, idx):
    order = torch.argsort(idx.reshape(-1), stable=True)
    dst = torch.empty_like(order)
    dst[order] = torch.arange(order.numel())
    off = torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(idx.reshape(-1), minlength=c.E).cumsum(0)])
    c.route.update(topk_idx=idx.int(), dst_row=dst.int(), src_slot=order.int(), group_off=off.int())


@pytest.mark.parametrize("T", [1, 5, 60])
def test_the_same_expert_twice(moe, T):
    c = Ffn(moe, T, 6, 128, 96, 3, 32, True, seed=9)
    _reroute(c, torch.arange(T)[:, None].expand(T, 3) % 2 * 5)
    c.check(c.run())


@pytest.mark.parametrize("T", [1, 4, 40])
def test_eight_slots_of_a_thousand_experts(moe, T):
    c = Ffn(moe, T, 1024, 64, 32, 8, 32, True, seed=T)
    c.check(c.run())


@pytest.mark.parametrize("T", [1, 20, 90])
def test_parameters_at_odd_addresses(moe, T):
    """Scales at any even address, zero points at any."""
    c = Ffn(moe, T, 3, 128, 64, 2, 32, True, seed=5)
    c.check(c.run())
    want = c.run()
    for i, (codes, s, z) in enumerate(c.w):
        wide_s = torch.full((s.numel() + 9,), float("nan"), dtype=BF, device=DEV)
        wide_z = torch.full((z.numel() + 9,), 255, dtype=torch.uint8, device=DEV)
        s2, z2 = wide_s[1:1 + s.numel()].view(s.shape), wide_z[3:3 + z.numel()].view(z.shape)
        s2.copy_(s)
        z2.copy_(z)
        c.w[i] = (codes, s2, z2)
    assert torch.equal(c.run(), want)


def _big(moe, T, E, d, f, k, group):
    """A call on the device whose codes are random bytes, scales 2^-7 and zero points 8."""
    g = torch.Generator(DEV).manual_seed(1)
    w = []
    for N, K in ((2 * f, d), (d, f)):
        codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8, device=DEV)
        w.append((codes, torch.full((E, N, K // group), 2.0 ** -7 if K < 1024 else 2.0 ** -11, dtype=BF, device=DEV), None))
    x = torch.empty(T, d, dtype=BF, device=DEV)
    for a in range(0, T, 1 << 18):
        x[a:a + (1 << 18)].normal_(generator=g)
    r = _route(T, E, k, 3)
    out = torch.empty(T, d, dtype=BF, device=DEV)
    ws = torch.empty(moe.moe_int4_workspace_bytes(T * k, d, f), dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_int4_ffn(moe.glu(), x, *(r[n].to(DEV) for n in ("topk_idx", "topk_w", "dst_row", "src_slot", "group_off")), group,
                     *w, out, ws, dev_err=err)
    assert int(err) == 0
    return x, r, w, out


def _big_values(w, e, rows):
    codes, s, _ = w
    c = codes[e, rows]
    return (torch.stack([c & 15, c >> 4], -1).flatten(1).double() - 8) * float(s.flatten()[0])


def _big_check(x, r, w, out, tokens):
    """Some tokens in 64 bits.  The bounds of Ffn.check with one scale: fp32 sums of K terms below 31 |x| s each, in
    two steps, then the roundings of h and of the output."""
    f, d = w[1][0].shape[2] * 2, x.shape[1]
    for t in tokens:
        want = torch.zeros(d, dtype=torch.float64, device=DEV)
        tol = torch.zeros_like(want)
        v = x[t].double()
        for j in range(r["topk_idx"].shape[1]):
            e, c = int(r["topk_idx"][t, j]), float(r["topk_w"][t, j])
            gu, mag = [], []
            for a in range(0, 2 * f, 128):
                m = _big_values(w[0], e, slice(a, min(a + 128, 2 * f)))
                gu.append(m @ v)
                mag.append(m.abs() @ v.abs())
            gu, mag = torch.cat(gu), torch.cat(mag)
            s = float(w[0][1].flatten()[0])
            eps = 2.0 ** -23 * (2 * 31 * 132 * s * float(v.abs().sum()) + (d // 32 + 12) * mag)
            g, u, dg, du = gu[:f], gu[f:], eps[:f], eps[f:]
            h = g * torch.sigmoid(g) * u
            dh = 1.13 * dg * (u.abs() + du) + (g * torch.sigmoid(g)).abs() * du + GATE * h.abs()
            dh = dh + 2.0 ** -8 * (h.abs() + dh)
            for a in range(0, d, 1 << 16):
                m = _big_values(w[1], e, slice(a, min(a + (1 << 16), d)))
                y = m @ h
                s = float(w[1][1].flatten()[0])
                dy = 2.0 ** -23 * (2 * 31 * 132 * s * float(h.abs().sum()) + (f // 32 + 12) * (m.abs() @ h.abs())) * 1.01
                dy = dy + m.abs() @ dh
                want[a:a + (1 << 16)] += c * y
                tol[a:a + (1 << 16)] += c * (dy + 2.0 ** -20 * y.abs())
        err = (out[t].double() - want).abs()
        tol += 2.0 ** -8 * want.abs() + 1e-35
        assert bool((err <= tol).all()), (t, float((err / tol).max()))
        assert float(err.norm()) <= 2.0 ** -6 * float(want.norm())


def test_as_many_tokens_as_32_bits_hold(moe):
    """x and h of just under 2^31 bytes, fp32 expert outputs past 2^32."""
    T = 2 ** 23 - 1
    _say("int4 many tokens")
    x, r, w, out = _big(moe, T, 8, 128, 128, 1, 64)
    _big_check(x, r, w, out, [0, 1, T // 2, T - 2, T - 1])
    src = r["src_slot"][torch.tensor([0, T - 1, T // 3])]
    _big_check(x, r, w, out, src.tolist())


@pytest.mark.parametrize("T", [1, 9, 70])
def test_the_widest_rows(moe, T):
    """d of 2^20: offsets into an expert's codes up to 2^30, 8192 chunks of K."""
    _say("int4 wide rows", T)
    x, r, w, out = _big(moe, T, 2, 2 ** 20, 1024, 2 if T < 20 else 1, 128)
    _big_check(x, r, w, out, sorted({0, T // 2, T - 1}))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,d,f", [(12, 3200, 2688), (30, 2176, 3712), (9, 4096, 1152), (20, 640, 1920)])
def test_workgroups_of_every_length(moe, T, d, f, group):
    """K shared by 3 to 16 waves, one step a tile."""
    c = Ffn(moe, T, 3, d, f, 2, group, True, seed=T)
    c.check(c.run())
