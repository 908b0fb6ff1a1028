"""GPU parity of the MXFP4 path against plain 64-bit implementations.

Codes and scales (quantiser, dispatch) must match bit for bit, decoded values
exactly.  The products' tolerances count roundings: an fp32 sum of K products
is off by at most K additions' roundings of at most 2^-23 of sum |a b| each
(the matrix unit may truncate, so a whole unit), and the stored bf16 by half a
step, 2^-8 of the value.
"""
import sys

import numpy as np
import pytest
import torch

import moe_synth
import oracle
from tests import _plain
from tests._chain import BF16_TOL, assert_close, np64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _say(*a):
    print("[gpu-mx4]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


def _bf16(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(*shape, generator=g) * scale
    v[..., ::97] *= 64.0
    return v.to(torch.bfloat16)


def _quantize(moe, x):
    rows, K = x.shape
    codes = torch.full((rows, K // 2), 0xAA, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, K // 32), 0xAA, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_mxfp4(x.to(DEV), codes, scales)
    return codes, scales


# ------------------------------------------------------------------ codec
def _special(rows, K):
    v = torch.randn(rows, K, generator=torch.Generator().manual_seed(9))
    v[0, 3] = float("nan")
    v[1, 40] = float("inf")
    v[1, 41] = float("-inf")
    v[2, 0] = float("inf")
    v[2, 1] = float("nan")
    v[3, :32] = 0.0
    v[4, 32:64] = -0.0
    v[5, 5] = 3.3895e38                                       # the largest bf16
    v[6, 32:64] *= 1e-37
    v[7, :32] = 2.0 ** -133                                   # the smallest subnormal
    v[8, :32] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] * 4) * 2.0 ** -11     # every midpoint
    v[9, :32] = -torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] * 4) * 2.0 ** 60
    v[10, :32] = 6.0                                          # a maximum that just fits, and one that just does not
    v[11, :32] = 6.03125
    v[12, 0:32] = 2.0 ** -126 * 1.5
    return v.to(torch.bfloat16)


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (77, 256), (513, 1152), (64, 4096)])
def test_quantize_bit_exact(moe, rows, K):
    _say("quantize", rows, K)
    x = _bf16((rows, K), rows + K, 0.02)
    codes, scales = _quantize(moe, x)
    back = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_dequantize_mxfp4(codes, scales, back)
    torch.cuda.synchronize()
    c, s = _plain.mxfp4_quantize(np64(x))
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    np.testing.assert_array_equal(np64(back), _plain.mxfp4_decode(c, s))


def test_quantize_special_values(moe):
    _say("quantize-special")
    x = _special(16, 64)
    codes, scales = _quantize(moe, x)
    back = torch.empty(16, 64, dtype=torch.bfloat16, device=DEV)
    moe.moe_dequantize_mxfp4(codes, scales, back)
    torch.cuda.synchronize()
    v = np64(x)
    c, s = _plain.mxfp4_quantize(v)
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    got = np64(back)
    assert np.isnan(got[0, :32]).all() and not np.isnan(got[0, 32:]).any()
    assert np.isnan(got[1, 32:]).all() and not np.isnan(got[1, :32]).any()    # nor do 4 bits hold infinities
    # the largest bf16 is 3.98 * 2^126, of which 4 * 2^126 = 2^128 is the nearest: past bf16's range
    assert s[5, 0] == 126 + 127 and c[5, 2] >> 4 == 6 and got[5, 5] == np.inf
    want = _plain.mxfp4_decode(c, s)
    want[np.abs(want) > 3.4e38] = np.sign(want[np.abs(want) > 3.4e38]) * np.inf
    np.testing.assert_array_equal(got, want)


def test_dequantize_every_code_and_scale(moe):
    _say("dequantize-all")
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(256, 1)       # K = 512: 16 blocks a row
    scales = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, 16)
    back = torch.empty(256, 512, dtype=torch.bfloat16, device=DEV)
    moe.moe_dequantize_mxfp4(codes.to(DEV), scales.to(DEV), back)
    torch.cuda.synchronize()
    want = _plain.mxfp4_decode(codes.numpy(), scales.numpy())
    want[np.abs(want) > 3.4e38] = np.sign(want[np.abs(want) > 3.4e38]) * np.inf
    np.testing.assert_array_equal(np64(back), want)


@pytest.mark.parametrize("T,d,E,k,C", [(1, 32, 4, 1, 0), (67, 1152, 8, 8, 0), (700, 256, 6, 2, 0), (300, 128, 5, 2, 90)])
def test_dispatch_bit_exact(moe, T, d, E, k, C):
    _say("dispatch", T, d, E, k, C)
    logits = moe_synth.router_logits(T, E, seed=T + d)
    x = _bf16((T, d), T * 3 + d)
    r = oracle.route(logits.numpy(), k, C)
    n = r["n_rows"]
    codes = torch.full((n, d // 2), 0xAA, dtype=torch.uint8, device=DEV)
    scales = torch.full((n, d // 32), 0xAA, dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dst, src = torch.from_numpy(r["dst_row"]).to(DEV), torch.from_numpy(r["src_slot"]).to(DEV)
    moe.moe_permute(moe.MOE_MXFP4, x.to(DEV), k, dst, codes, src_slot=src, x_perm_scales=scales, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    c, s = _plain.mxfp4_quantize(np64(x))
    live = r["src_slot"] >= 0
    want_c, want_s = np.zeros((n, d // 2), np.uint8), np.zeros((n, d // 32), np.uint8)
    want_c[live], want_s[live] = c[r["src_slot"][live] // k], s[r["src_slot"][live] // k]
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)          # rows of the padding are zero
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)


@pytest.mark.parametrize("T,d,E,k,C", [(70, 2048, 6, 3, 0), (70, 2080, 9, 8, 0), (120, 4128, 4, 2, 50), (5, 2016, 5, 5, 0)])
def test_dispatch_of_wide_rows(moe, T, d, E, k, C):
    """Rows on both sides of a workgroup per token, vectors that end inside its second pass, padding."""
    test_dispatch_bit_exact(moe, T, d, E, k, C)


def test_dispatch_flags_rows_out_of_range(moe):
    _say("dispatch-range")
    x = _bf16((4, 64), 1)
    codes = torch.full((8, 32), 0xAA, dtype=torch.uint8, device=DEV)
    scales = torch.full((8, 2), 0xAA, dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dst = torch.tensor([0, 1, 2, 8, 1 << 30, 5, -1, 7], dtype=torch.int32, device=DEV)
    moe.moe_permute(moe.MOE_MXFP4, x.to(DEV), 2, dst, codes, x_perm_scales=scales, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == moe.MOE_ERR_ROW_RANGE
    c, _ = _plain.mxfp4_quantize(np64(x))
    got = codes.cpu().numpy()
    for row, tok in ((0, 0), (1, 0), (2, 1), (5, 2), (7, 3)):
        np.testing.assert_array_equal(got[row], c[tok])
    for row in (3, 4, 6):
        assert (got[row] == 0xAA).all()


def test_quantize_past_the_cache(moe):
    """From 256 MB of source on the accesses stream: the same codes as of its halves."""
    _say("quantize-stream")
    rows, K = 33001, 4128
    x = torch.randn(rows, K, generator=torch.Generator(DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    codes, scales = _quantize(moe, x)
    back = torch.empty_like(x)
    moe.moe_dequantize_mxfp4(codes, scales, back)
    for sl in (slice(0, 15000), slice(15000, 30000), slice(30000, rows)):
        c, s = _quantize(moe, x[sl].contiguous())
        b = torch.empty_like(x[sl])
        moe.moe_dequantize_mxfp4(c, s, b)
        assert torch.equal(codes[sl], c) and torch.equal(scales[sl], s) and torch.equal(back[sl], b)


def test_quantize_and_dispatch_past_32_bits(moe):
    """More elements than 2^32, more workgroups than a grid has: the last rows are those of small calls."""
    _say("quantize-dispatch-long")
    rows, K = (1 << 20) + 1003, 4224
    x = torch.empty(rows, K, dtype=torch.bfloat16, device=DEV)
    base = torch.randn(1009, K, generator=torch.Generator(DEV).manual_seed(2), device=DEV).to(torch.bfloat16)
    for a in range(0, rows, 1009):
        n = min(1009, rows - a)
        x[a:a + n] = base[:n]
    bc, bs = _quantize(moe, base)
    idx = torch.arange(rows, device=DEV) % 1009
    ends = torch.cat([torch.arange(0, 5000), torch.arange(rows - 5000, rows)]).to(DEV)
    mid = torch.randint(0, rows, (5000,), generator=torch.Generator(DEV).manual_seed(3), device=DEV)
    pick = torch.cat([ends, mid])
    codes, scales = _quantize(moe, x)
    assert torch.equal(codes[pick], bc[idx[pick]]) and torch.equal(scales[pick], bs[idx[pick]])
    back = torch.zeros_like(x)
    moe.moe_dequantize_mxfp4(codes, scales, back)
    small = torch.empty_like(base)
    moe.moe_dequantize_mxfp4(bc, bs, small)
    assert torch.equal(back[pick], small[idx[pick]])
    del back
    for d in (K, 128):                        # a workgroup per token, and by vectors
        T = rows * K // d
        dst = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)
        codes.fill_(0xAA)
        moe.moe_permute(moe.MOE_MXFP4, x.view(T, d), 1, dst, codes.view(T, d // 2), x_perm_scales=scales.view(T, d // 32))
        want_c, want_s = bc.view(-1, d // 2), bs.view(-1, d // 32)
        tok = torch.cat([torch.arange(0, 9000), torch.arange(T - 9000, T)]).to(DEV)
        per = want_c.shape[0]
        assert torch.equal(codes.view(T, d // 2)[T - 1 - tok], want_c[tok % per])
        assert torch.equal(scales.view(T, d // 32)[T - 1 - tok], want_s[tok % per])


def test_tensors_of_the_host_are_refused(moe):
    q = _case(moe, [4], 256, 128)
    x = _bf16((4, 256), 1).to(DEV)
    dst = torch.arange(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_permute(moe.MOE_MXFP4, x, 1, dst, q["x"], x_perm_scales=q["xs"])
    y = torch.empty(4, 256, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm_fwd(moe.MOE_MXFP4, q["x"], q["w13"], q["w2"], q["off"], 0, None, None, y,
                                 x_perm_scales=q["xs"], w13_scales=q["w13s"], w2_scales=q["w2s"],
                                 ws=torch.empty(1 << 16, dtype=torch.uint8))


# ------------------------------------------------------------------ products
def _case(moe, sizes, d, f, seed=1, xscale=1.0, capacity=0, special=None):
    """Operands of groups of the given sizes, with rows before and behind when off says so."""
    E = len(sizes)
    R = E * capacity if capacity else sum(sizes)
    x = _bf16((R, d), seed, xscale)
    if special:
        special(x)
    w13 = _bf16((E * 2 * f, d), seed + 1, 0.05 if d > 512 else 0.1)
    w2 = _bf16((E * d, f), seed + 2, 0.05)
    q = {}
    for n, t in (("x", x), ("w13", w13), ("w2", w2)):
        q[n], q[n + "s"] = _quantize(moe, t)
    q["w13"], q["w13s"] = q["w13"].view(E, 2 * f, d // 2), q["w13s"].view(E, 2 * f, d // 32)
    q["w2"], q["w2s"] = q["w2"].view(E, d, f // 2), q["w2s"].view(E, d, f // 32)
    q["off"] = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=DEV)
    return q


def _forward(moe, q, d, f, capacity=0, save=True, ws=None):
    E, R = q["w13"].shape[0], q["x"].shape[0]
    bf = dict(dtype=torch.bfloat16, device=DEV)
    gu = torch.full((R, 2 * f), 123.0, **bf) if save else None
    h = torch.full((R, f), 123.0, **bf) if save else None
    y = torch.full((R, d), 123.0, **bf)
    if ws is None:
        ws = torch.full((max(moe.moe_gemm_workspace_bytes(moe.MOE_MXFP4, E, R, d, f), 1),), 0xFF, dtype=torch.uint8,
                        device=DEV)
    moe.moe_grouped_gemm_fwd(moe.MOE_MXFP4, q["x"], q["w13"], q["w2"], q["off"], capacity, gu, h, y,
                             x_perm_scales=q["xs"], w13_scales=q["w13s"], w2_scales=q["w2s"], ws=ws)
    return gu, h, y


def _check(q, gu, h, y, sizes, d, f, rows0=0, capacity=0):
    """gu from the operands, h from this gu's definition, y from the h the GPU stored."""
    x = _plain.mxfp4_decode(q["x"].cpu(), q["xs"].cpu())
    w13 = _plain.mxfp4_decode(q["w13"].cpu(), q["w13s"].cpu())
    w2 = _plain.mxfp4_decode(q["w2"].cpu(), q["w2s"].cpu())
    gu, h, y = np64(gu), np64(h), np64(y)
    at = rows0
    for e, n in enumerate(sizes):
        a = e * capacity if capacity else at
        n = capacity if capacity else n
        sl = slice(a, a + n)
        ref = x[sl] @ w13[e].T
        acc = d * 2.0 ** -23 * (np.abs(x[sl]) @ np.abs(w13[e]).T)      # the fp32 sums of g and u
        tol = 2.0 ** -8 * np.abs(ref) + acc
        assert np.all(np.abs(gu[sl] - ref) <= tol), f"gu of group {e}"
        g, u, dg, du = ref[:, :f], ref[:, f:], acc[:, :f], acc[:, f:]
        href = _plain.silu(g) * u
        # |silu'| <= 1.1, |silu| <= |g|; the logistic's exponential and reciprocal are good to 2^-20
        htol = (2.0 ** -8 + 2.0 ** -20) * np.abs(href) + 1.1 * (np.abs(u) + du) * dg + (np.abs(g) + dg) * du
        assert np.all(np.abs(h[sl] - href) <= htol), f"h of group {e}"
        hq = _plain.mxfp4_qdq(h[sl]) if n else h[sl]
        yref = hq @ w2[e].T
        ytol = 2.0 ** -8 * np.abs(yref) + f * 2.0 ** -23 * (np.abs(hq) @ np.abs(w2[e]).T)
        assert np.all(np.abs(y[sl] - yref) <= ytol), f"y of group {e}"
        at += n
    return at


SIZES = [
    # sizes of the groups, d, f
    ([1], 128, 128), ([1, 0, 1], 256, 128), ([0, 0, 5], 128, 384), ([3, 1, 2, 1], 640, 256),
    ([16, 17, 15], 512, 256), ([33, 0, 64, 65], 256, 384), ([129, 128, 127], 384, 128), ([257, 1, 300], 256, 256),
    ([200, 511], 1152, 640), ([70, 0, 260, 90], 128, 128), ([1, 2], 4096, 1536), ([40, 10], 2176, 1280),
    # few rows over many experts: skewed (several 16- and 64-row groups of one expert), and K of several panels
    ([0] * 20 + [63] + [0] * 20, 256, 128), ([1] * 3 + [0] * 60 + [130, 1], 640, 256), ([2, 1], 8448, 2176),
    ([0, 17, 0, 0, 0, 0, 1, 0], 384, 4224), ([1, 0] * 70, 128, 128),
]


@pytest.mark.parametrize("sizes,d,f", SIZES)
def test_products(moe, sizes, d, f):
    _say("products", sizes, d, f)
    q = _case(moe, sizes, d, f, seed=sum(sizes) + d)
    gu, h, y = _forward(moe, q, d, f)
    torch.cuda.synchronize()
    _check(q, gu, h, y, sizes, d, f)
    # without the saved activations: the same bits
    _, _, y2 = _forward(moe, q, d, f, save=False)
    gu3, h3, y3 = _forward(moe, q, d, f)
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(y3, y) and torch.equal(gu3, gu) and torch.equal(h3, h)


# enough column tiles that 256-row tiles are taken: every length of that loop
# (an odd and an even number of 128-k halves up to its steady state and past
# it) for the gate/up stage (K = d), then for the down stage (K = f)
@pytest.mark.parametrize("d,f", [(128, 1536), (256, 1536), (384, 1536), (512, 1536), (640, 1536), (768, 1536),
                                 (1024, 1536), (1152, 1536), (1280, 1536), (1408, 1536), (2176, 1536), (4096, 128),
                                 (4096, 384), (4096, 640), (3968, 896)])
def test_products_with_large_tiles(moe, d, f):
    _say("products-large-tiles", d, f)
    sizes = [257, 0, 512, 700, 255, 1000]
    q = _case(moe, sizes, d, f, seed=d + f)
    gu, h, y = _forward(moe, q, d, f)
    _, _, y2 = _forward(moe, q, d, f, save=False)
    torch.cuda.synchronize()
    _check(q, gu, h, y, sizes, d, f)
    assert torch.equal(y2, y)


def test_products_past_32_bits(moe):
    """More than 2^32 outputs: a block of rows over and over gives the same bits everywhere, up to the last row."""
    _say("products-long")
    n, reps, d, f = 512, 4200, 256, 1024
    q = _case(moe, [n], d, f)
    q["x"], q["xs"] = q["x"].repeat(reps, 1), q["xs"].repeat(reps, 1)
    q["off"] = torch.tensor([0, n * reps], dtype=torch.int32, device=DEV)
    assert n * reps * 2 * f > 1 << 32
    gu, h, y = _forward(moe, q, d, f)
    torch.cuda.synchronize()
    for t in (gu, h, y):
        b = t.view(reps, n, -1)
        for i in (1, reps // 2, reps - 2, reps - 1):
            assert torch.equal(b[i], b[0]), i
    q["x"], q["xs"] = q["x"][:n].contiguous(), q["xs"][:n].contiguous()
    _check(q, gu[:n], h[:n], y[:n], [n], d, f)


def test_products_padded(moe):
    _say("products-padded")
    C, d, f, E = 70, 256, 128, 3
    q = _case(moe, [C] * E, d, f, capacity=C)
    gu, h, y = _forward(moe, q, d, f, capacity=C)
    torch.cuda.synchronize()
    _check(q, gu, h, y, [C] * E, d, f, capacity=C)


@pytest.mark.parametrize("before,behind", [(0, 40), (5, 300)])
def test_rows_outside_every_group_stay(moe, before, behind):
    _say("products-outside", before, behind)
    sizes, d, f = [20, 0, 30], 256, 128
    q = _case(moe, [before] + sizes + [behind], d, f)
    for n in ("w13", "w13s", "w2", "w2s"):
        q[n] = q[n][1:4].contiguous()
    q["off"] = q["off"][1:5].contiguous()
    gu, h, y = _forward(moe, q, d, f)
    torch.cuda.synchronize()
    assert _check(q, gu, h, y, sizes, d, f, rows0=before) == before + 50
    for t in (gu, h, y):
        assert bool((t[:before] == 123).all()) and bool((t[before + 50:] == 123).all())


def test_corrupt_offsets_stay_inside(moe):
    _say("products-offsets")
    d, f = 128, 128
    q = _case(moe, [10, 20, 30], d, f)
    for off in ([0, 10, 5, 60], [-7, 10, 30, 1 << 30], [60, 60, 60, 60], [50, 40, 30, 20]):
        q["off"] = torch.tensor(off, dtype=torch.int32, device=DEV)
        _forward(moe, q, d, f)
        torch.cuda.synchronize()


def test_no_rows(moe):
    q = _case(moe, [3, 4], 128, 128)
    for n in ("x", "xs"):
        q[n] = q[n][:0]
    q["off"].zero_()
    _forward(moe, q, 128, 128)
    torch.cuda.synchronize()


def test_nan_and_infinity_stay_in_their_rows(moe):
    _say("products-nan")

    def special(x):
        x[3, 5] = float("nan")
        x[70, 200] = float("inf")
    sizes, d, f = [66, 30], 256, 128
    q = _case(moe, sizes, d, f, special=special)
    gu, h, y = _forward(moe, q, d, f)
    clean = _case(moe, sizes, d, f)
    gu0, h0, y0 = _forward(moe, clean, d, f)
    torch.cuda.synchronize()
    assert bool(gu[3].isnan().all()) and bool(y[3].isnan().all())
    assert not bool(gu[70].isfinite().any())
    keep = torch.ones(96, dtype=torch.bool, device=DEV)
    keep[3] = keep[70] = False
    for a, b in ((gu, gu0), (h, h0), (y, y0)):
        assert torch.equal(a[keep], b[keep])


def test_extreme_scales(moe):
    """Blocks near the ends of the scale range multiply to ordinary numbers."""
    _say("products-scales")
    sizes, d, f = [20], 256, 128
    q = _case(moe, sizes, d, f)
    q["xs"] = (q["xs"].to(torch.int32) + 100).clamp(max=254).to(torch.uint8)
    q["w13s"] = (q["w13s"].to(torch.int32) - 100).clamp(min=0).to(torch.uint8)
    gu, h, y = _forward(moe, q, d, f)
    torch.cuda.synchronize()
    _check(q, gu, h, y, sizes, d, f)


def test_stages_are_the_forward(moe):
    _say("products-stages")
    sizes, d, f = [30, 70, 0, 200], 512, 384
    q = _case(moe, sizes, d, f)
    gu, h, y = _forward(moe, q, d, f)
    R, E = sum(sizes), len(sizes)
    gu2, h2, y2 = torch.empty_like(gu), torch.empty_like(h), torch.empty_like(y)
    ws = torch.empty(moe.moe_gemm_workspace_bytes(moe.MOE_MXFP4, E, R, d, f), dtype=torch.uint8, device=DEV)
    t = moe.gemm_tensors(x_perm=q["x"], x_perm_scales=q["xs"], w13=q["w13"], w13_scales=q["w13s"], w2=q["w2"],
                         w2_scales=q["w2s"], gu=gu2, h=h2, y_perm=y2, ws=ws)
    for op in (moe.MOE_GEMM_GATE_UP, moe.MOE_GEMM_DOWN):
        moe.moe_grouped_gemm_op(op, moe.MOE_MXFP4, t, q["off"], 0, E, R, d, f)
    torch.cuda.synchronize()
    assert torch.equal(gu2, gu) and torch.equal(h2, h) and torch.equal(y2, y)


def test_strided_tensors_are_refused(moe):
    q = _case(moe, [4], 256, 128)
    y = torch.empty(4, 512, dtype=torch.bfloat16, device=DEV)[:, ::2]
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm_fwd(moe.MOE_MXFP4, q["x"], q["w13"], q["w2"], q["off"], 0, None, None, y,
                                 x_perm_scales=q["xs"], w13_scales=q["w13s"], w2_scales=q["w2s"], ws=ws)
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4(y, q["x"], q["xs"])


# ------------------------------------------------------------------ the layer
@pytest.mark.parametrize("T,d,E,f,k,S,C", [(300, 256, 6, 256, 2, 0, 0), (64, 128, 8, 128, 2, 1, 0),
                                           (257, 384, 4, 128, 1, 0, 90), (1, 256, 8, 128, 4, 0, 0)])
def test_layer_forward_backward(moe, T, d, E, f, k, S, C):
    """The layer's MXFP4 forward, and its backward: the bf16 one of the oracle on the decoded operands."""
    _say("layer", T, d, E, f, k, S, C)
    from routing_grouped_gemm_amd.layer import MoELayer
    inp = moe_synth.make_inputs(T=T, d=d, E=E + S, f=f, k=k, seed=T + E)
    inp["logits"] = inp["logits"][:, :E].contiguous()
    inp["x"] = (inp["x"].float() * 50).to(torch.bfloat16)
    g = {n: inp[n].to(DEV) for n in ("logits", "x", "w13", "w2", "dout")}
    lay = MoELayer(T, d, E, f, k, moe.MOE_MXFP4, capacity=C, n_shared=S)
    lay.set_weights(g["w13"], g["w2"])
    out = lay.forward(g["logits"], g["x"])
    dx, dw13, dw2 = lay.backward(g["dout"])
    torch.cuda.synchronize()
    assert int(lay.dev_err) == 0
    go = lay.s_off.cpu().numpy().astype(np.int32)
    if C and not S:
        go = (np.arange(E + 1) * C).astype(np.int32)
    xq = _plain.mxfp4_decode(lay.x_perm.cpu(), lay.x_perm_scales.cpu())
    w13 = _plain.mxfp4_qdq(np64(inp["w13"]).reshape(-1, d)).reshape(E + S, 2 * f, d)
    w2 = _plain.mxfp4_qdq(np64(inp["w2"]).reshape(-1, f)).reshape(E + S, d, f)
    np.testing.assert_array_equal(np64(lay.w13_d), w13)
    np.testing.assert_array_equal(np64(lay.w2_d), w2)
    dst, w = lay.s_dst.cpu().numpy(), lay.s_w.cpu().numpy()
    xt = _plain.mxfp4_qdq(np64(inp["x"]))
    live = dst >= 0
    np.testing.assert_array_equal(xq[dst[live]], xt[np.nonzero(live)[0] // (k + S)])
    gu, h, _ = oracle.ffn_fwd(xq, w13, w2, go, oracle.BF16)
    assert_close(np64(lay.gu), gu, BF16_TOL, "gu")
    assert_close(np64(lay.h), h, BF16_TOL, "h")
    y = np.zeros_like(xq)
    hq = _plain.mxfp4_qdq(np64(lay.h))
    for e in range(E + S):
        y[go[e]:go[e + 1]] = hq[go[e]:go[e + 1]] @ w2[e].T
    assert_close(np64(lay.y_perm), y, BF16_TOL, "y_perm")
    assert_close(np64(out), oracle.combine(np64(lay.y_perm), dst, w, T, k + S, oracle.BF16), BF16_TOL, "out")
    dy = oracle.permute(np64(inp["dout"]), dst, k + S, xq.shape[0], row_scale=w, round_mode=oracle.BF16)
    _, dxp, rdw13, rdw2 = oracle.ffn_bwd(dy, xq, np64(lay.gu), np64(lay.h), w13, w2, go, oracle.BF16)
    assert_close(np64(dx), oracle.combine(dxp, dst, None, T, k + S, oracle.BF16), BF16_TOL, "dx")
    assert_close(np64(dw13), rdw13, BF16_TOL, "dw13")
    assert_close(np64(dw2), rdw2, BF16_TOL, "dw2")
    # stage by stage, and the weight gradient into fp32 accumulators
    ref = {n: getattr(lay, n).clone() for n in ("y_perm", "dx_perm", "dw13", "dw2")}
    for op in range(5):
        lay.gemm_stage(op)
    torch.cuda.synchronize()
    for n, v in ref.items():
        assert torch.equal(getattr(lay, n), v), n
    a13 = torch.zeros(E + S, 2 * f, d, device=DEV)
    a2 = torch.zeros(E + S, d, f, device=DEV)
    lay.wgrad_accumulate(a13, a2)
    torch.cuda.synchronize()
    assert_close(np64(a13), rdw13, BF16_TOL, "dw13 accumulated")
    assert_close(np64(a2), rdw2, BF16_TOL, "dw2 accumulated")
    # weights that come in 4 bits; no saved activations: the same output
    serve = MoELayer(T, d, E, f, k, moe.MOE_MXFP4, capacity=C, n_shared=S, save=False)
    serve.set_weights_mxfp4(lay.w13_q, lay.w13_s, lay.w2_q, lay.w2_s)
    assert torch.equal(serve.forward(g["logits"], g["x"]), out)
    serve.gemm_stage(moe.MOE_GEMM_GATE_UP)
    serve.gemm_stage(moe.MOE_GEMM_DOWN)
    assert torch.equal(serve.y_perm, lay.y_perm)
    with pytest.raises(RuntimeError):
        serve.backward(g["dout"])


def test_codes_given_to_a_layer_are_not_made_anew(moe):
    """Weights given in 4 bits after bf16 ones: no call writes the old weights' codes into them."""
    from routing_grouped_gemm_amd.layer import MoELayer
    T, d, E, f, k = 20, 128, 4, 128, 2
    inp = moe_synth.make_inputs(T=T, d=d, E=E, f=f, k=k, seed=3)
    lay = MoELayer(T, d, E, f, k, moe.MOE_MXFP4)
    lay.set_weights(inp["w13"].to(DEV), inp["w2"].to(DEV))
    codes = [t.clone() for t in (lay.w13_q, lay.w13_s, lay.w2_q, lay.w2_s)]
    codes[0].zero_()
    lay.set_weights_mxfp4(*codes)
    with pytest.raises(ValueError):
        lay.requantize_weights()
    assert not bool(codes[0].any())
    out = lay.forward(inp["logits"].to(DEV), inp["x"].to(DEV))
    torch.cuda.synchronize()
    assert not bool(out.any())                       # silu(0) * 0
    lay.set_weights(inp["w13"].to(DEV), inp["w2"].to(DEV))
    lay.requantize_weights()
    assert bool(lay.w13_q.any()) and not bool(codes[0].any())


def test_two_layers_two_streams_and_graphs(moe):
    """Forwards of two layers captured in two graphs and replayed on two streams at once, with eager
    steps in between, give the eager results."""
    _say("graphs")
    from routing_grouped_gemm_amd.layer import MoELayer
    T, d, E, f, k = 200, 256, 6, 256, 2
    lays, ins, refs, graphs = [], [], [], []
    for i in range(2):
        inp = moe_synth.make_inputs(T=T, d=d, E=E, f=f, k=k, seed=50 + i)
        g = {n: inp[n].to(DEV) for n in ("logits", "x", "w13", "w2", "dout")}
        lay = MoELayer(T, d, E, f, k, moe.MOE_MXFP4)
        lay.set_weights(g["w13"], g["w2"])

        def step(lay=lay, g=g):
            lay.forward(g["logits"], g["x"])
            lay.backward(g["dout"])
        step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
        lays.append((lay, step, side))
        ins.append(g)
        graphs.append(gr)
    for rep in range(3):
        refs = []
        for (lay, step, _), g in zip(lays, ins):
            g["x"].copy_((torch.randn(T, d, generator=torch.Generator().manual_seed(rep)) * 3).to(torch.bfloat16))
            step()
            torch.cuda.synchronize()
            refs.append({n: getattr(lay, n).clone() for n in ("out", "y_perm", "gu", "dx", "dw13", "dw2")})
            for n in refs[-1]:
                getattr(lay, n).fill_(0)
        torch.cuda.synchronize()
        for gr, (_, _, side) in zip(graphs, lays):
            with torch.cuda.stream(side):
                gr.replay()
        torch.cuda.synchronize()
        for (lay, _, _), ref in zip(lays, refs):
            for n, v in ref.items():
                assert torch.equal(getattr(lay, n), v), (rep, n)
