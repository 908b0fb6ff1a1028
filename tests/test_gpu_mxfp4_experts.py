"""MXFP4 products of many experts: the tile kernels' schedule for more than 128 experts, at each tile height, against
64-bit values.  The tolerances are those of a sum of K products in fp32 (2^-23 of sum |a b| for each addition) and of
the stored bf16 (2^-8 of the value)."""
import sys

import numpy as np
import pytest
import torch

from tests import _plain
from tests._chain import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _say(*a):
    print("[gpu-mx4-experts]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


def _qdq(v):
    """MXFP4 there and back of v [rows, K], as _plain.mxfp4_qdq, all blocks at once."""
    b = np.asarray(v, np.float64).reshape(-1, 32)
    m, e = np.frexp(np.abs(b).max(1, keepdims=True))
    s = np.exp2(np.where(m > 0, np.clip(e - 3 + (m > 0.75), -127, 127), -127).astype(np.float64))
    a = np.abs(b) / s
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return (np.copysign(np.rint(a / step) * step * s, b)).reshape(np.shape(v))


def _quantize(moe, shape, seed, scale):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn(*shape, generator=g, device=DEV) * scale).to(torch.bfloat16)
    K = shape[-1]
    codes = torch.empty(*shape[:-1], K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(*shape[:-1], K // 32, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_mxfp4(x.view(-1, K), codes.view(-1, K // 2), scales.view(-1, K // 32))
    return codes, scales


def _row_tiles(n, E, bm):
    e = min(E, n)
    return e + (n - e) // bm


def _form(n, E, K, n_out, gate_up):
    """Which form the host's rule takes: 'few', or the tiles' rows."""
    e = min(E, n)
    wgs, one = _row_tiles(n, E, 64) * (n_out // 32), 256 * (2 if K <= 2048 else 1)
    if wgs <= 256 if n > 32 * e else wgs <= one if n > 16 * e else 2 * wgs <= 3 * one:
        return "few"
    ntn = n_out // 128 if gate_up else -(-n_out // 256)
    return next((bm for bm in (64, 128) if _row_tiles(n, E, bm) * ntn <= 256), 256)


def _sizes(E, mean, seed):
    """Ragged: a tenth empty, a tenth of one row, tile heights and their neighbours, one expert with many rows."""
    rng = np.random.default_rng(seed)
    s = rng.integers(1, 2 * mean, E)
    s[rng.random(E) < 0.1] = 0
    s[rng.random(E) < 0.1] = 1
    for i, v in enumerate((63, 64, 65, 127, 128, 129)):
        s[(i * 37 + E // 2) % E] = min(v, 3 * mean)
    s[-1] = 3 * mean
    return s


@pytest.mark.parametrize("E,mean,d,f,capacity,up,down", [
    (129, 20, 256, 128, 0, 64, 64), (150, 24, 128, 128, 0, 64, 64), (130, 90, 256, 128, 0, 128, 128),
    (180, 0, 256, 128, 27, 64, 64), (135, 0, 256, 128, 110, 128, 128), (300, 160, 256, 256, 0, 256, 256),
    (1024, 34, 128, 128, 0, 256, 256), (1000, 40, 640, 256, 0, 256, 256), (257, 0, 384, 256, 70, 256, 256),
])
def test_products_of_many_experts(moe, E, mean, d, f, capacity, up, down):
    _say(E, mean, d, f, capacity)
    sizes = np.full(E, capacity) if capacity else _sizes(E, mean, E)
    R = int(sizes.sum())
    assert _form(R, E, d, f, True) == up and _form(R, E, f, d, False) == down
    x, xs = _quantize(moe, (R, d), E, 1.0)
    w13, w13s = _quantize(moe, (E, 2 * f, d), E + 1, d ** -0.5)
    w2, w2s = _quantize(moe, (E, d, f), E + 2, f ** -0.5)
    off = np.concatenate([[0], np.cumsum(sizes)])
    gu, h, y = (torch.full((R, n), 123.0, dtype=torch.bfloat16, device=DEV) for n in (2 * f, f, d))
    ws = torch.full((moe.moe_gemm_workspace_bytes(moe.MOE_MXFP4, E, R, d, f),), 0xFF, dtype=torch.uint8, device=DEV)
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    if capacity:
        offsets.zero_()                                  # only its length counts
    moe.moe_grouped_gemm_fwd(moe.MOE_MXFP4, x, w13, w2, offsets, capacity, gu, h, y, x_perm_scales=xs, w13_scales=w13s,
                             w2_scales=w2s, ws=ws)
    torch.cuda.synchronize()
    gu, h, y = np64(gu), np64(h), np64(y)
    xv, xsc, w13, w13s, w2, w2s = (t.cpu().numpy() for t in (x, xs, w13, w13s, w2, w2s))
    for e in range(E):
        sl = slice(int(off[e]), int(off[e + 1]))
        if sl.start == sl.stop:
            continue
        a, b = _plain.mxfp4_decode(xv[sl], xsc[sl]), _plain.mxfp4_decode(w13[e], w13s[e])
        ref, acc = a @ b.T, d * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)
        assert np.all(np.abs(gu[sl] - ref) <= 2.0 ** -8 * np.abs(ref) + acc), ("gu", e)
        g, u, dg, du = ref[:, :f], ref[:, f:], acc[:, :f], acc[:, f:]
        href = _plain.silu(g) * u
        htol = (2.0 ** -8 + 2.0 ** -20) * np.abs(href) + 1.1 * (np.abs(u) + du) * dg + (np.abs(g) + dg) * du
        assert np.all(np.abs(h[sl] - href) <= htol), ("h", e)
        hq, c = _qdq(h[sl]), _plain.mxfp4_decode(w2[e], w2s[e])
        yref = hq @ c.T
        assert np.all(np.abs(y[sl] - yref) <= 2.0 ** -8 * np.abs(yref) + f * 2.0 ** -23 * (np.abs(hq) @ np.abs(c).T)), ("y", e)


def test_block_codec_is_the_plain_one():
    rng = np.random.default_rng(1)
    v = _plain.bf16_round(rng.standard_normal((30, 96)) * np.exp2(rng.integers(-40, 40, (30, 1)).astype(float)))
    v[3, :32] = 0
    v[4, :8] = [6, 0.25, -0.75, 1.25, 1.75, 2.5, 3.5, -5]
    v[4, 8:32] = 0
    np.testing.assert_array_equal(_qdq(v), _plain.mxfp4_qdq(v))
