"""CPU checks of the dropout, gated block and 4-bit integer calls: the plain implementations against published values,
differences and brute force, and the refusals of every entry point.  No kernel runs: each call fails validation."""
import ctypes
import os

import numpy as np
import pytest
import torch

from tests import _plain_gated as pl

P = 0x10000          # 16-byte aligned, never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def m():
    import routing_grouped_gemm_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return m


# ------------------------------------------------------------------ the plain implementations
def test_philox_known_answers():
    """The three answers published with the generator: counter and key all zeros, all ones, and digits of pi."""
    assert pl.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert pl.philox([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert pl.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_philox_blocks_are_the_scalar_ones():
    seed, step = 0x123456789ABCDEF0, 0xFEDCBA9876543210
    at = [0, 1, 7, 2 ** 32 - 1, 2 ** 32, 2 ** 37 + 5]
    got = pl.philox_blocks(np.array(at, np.uint64), seed, step)
    for b, w in zip(at, got):
        assert list(map(int, w)) == pl.philox([b & 0xFFFFFFFF, b >> 32, step & 0xFFFFFFFF, step >> 32],
                                              [seed & 0xFFFFFFFF, seed >> 32])


@pytest.mark.parametrize("p", [0.1, 0.5])
def test_mask_rate_and_mean(p):
    """n independent elements: the kept share is within five standard deviations, the factors' mean 1 as near."""
    n = 1 << 16
    f = pl.factors(n, p, 5, 9)
    q = 1 - pl.threshold(p) / 65536
    assert abs(float((f > 0).double().mean()) - q) < 5 * (q * (1 - q) / n) ** 0.5
    assert float(f.max()) * q == pytest.approx(1, rel=1e-12)
    assert not torch.equal(f, pl.factors(n, p, 5, 10)) and not torch.equal(f, pl.factors(n, p, 6, 9))
    assert torch.equal(f[37:1037], pl.factors(1000, p, 5, 9, first=37))


@pytest.mark.parametrize("name", pl.ACTS)
def test_gate_slopes_are_the_differences(name):
    """Central differences with step 1e-5 in 64 bits: error about step^2 * third derivative / 6 + 2^-52 / step < 1e-9."""
    g = torch.cat([torch.linspace(-8, 8, 1601, dtype=torch.float64) + 0.003, torch.tensor([1.0, -1.2784], dtype=torch.float64)])
    d = (pl.act(name, g + 1e-5) - pl.act(name, g - 1e-5)) / 2e-5
    assert float((sum(pl.slope_terms(name, g)) - d).abs().max()) < 1e-9


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_codes_are_the_nearest(group, zeros):
    """Every code is one of those nearest to its value among the sixteen of its group, up to the clipping that a scale
    rounded down leaves: at most half a scale and 2^-8 of fifteen of them."""
    v = torch.randn(7, 3 * group, generator=torch.Generator().manual_seed(group)).to(torch.bfloat16).double().numpy()
    v[0, :group] = 0
    v[1, group:2 * group] = np.abs(v[1, group:2 * group])
    q, s, z = pl.int4_quantize(v, group, zeros)
    back = pl.int4_values(q, s, z, group)
    off = np.abs(back - v) / np.repeat(s, group, 1)
    assert (off <= 0.5 + (1.0 if zeros else 0.5)).all() and np.quantile(off, 0.99) <= 0.6
    levels = (np.arange(16)[None, None] - z[..., None].astype(float)) * s[..., None]
    best = np.abs(np.repeat(levels, group, 1) - v[..., None]).min(-1)
    assert (np.abs(back - v) <= best * (1 + 1e-12) + (np.repeat(s, group, 1) * 0.5 + 1e-300 if zeros else 0)).all()


# ------------------------------------------------------------------ refusals of the C calls
def test_dropout_refusals(m):
    lib = m.load()

    def call(dtype=m.MOE_BF16, x=P, res=None, n=64, p=0.1, rng=P, out=P):
        return lib.moe_dropout(dtype, x, res, n, p, rng, out, None)
    assert call(dtype=m.MOE_MXFP8) == m.MOE_EUNSUPPORTED
    assert call(n=-8) == call(n=1 << 40) == m.MOE_EINVAL
    for p in (1.0, -0.1, float("nan"), float("inf"), 2.0):
        assert call(p=p) == m.MOE_EINVAL, p
    assert call(rng=None) == call(x=None) == call(out=None) == m.MOE_EINVAL
    assert call(rng=P + 4) == m.MOE_EINVAL
    assert call(n=60) == call(x=P + 8) == call(res=P + 2) == call(out=P + 8) == m.MOE_EALIGN
    assert call(dtype=m.MOE_F32, n=62) == m.MOE_EALIGN
    assert call(n=0) == m.MOE_OK and call(n=0, p=0.0, rng=None, x=None, out=None) == m.MOE_OK


def test_combine_dropout_refusals(m):
    lib = m.load()

    def call(dtype=m.MOE_BF16, y=P, dst=P, w=P, res=P, T=4, k=2, d=64, n=8, p=0.1, rng=P, out=P):
        return lib.moe_combine_dropout(dtype, y, dst, w, res, T, k, d, n, p, rng, out, None, None)
    assert call(dtype=m.MOE_MXFP4) == m.MOE_EUNSUPPORTED
    assert call(T=-1) == call(k=0) == call(k=9) == call(d=0) == call(n=-1) == call(T=1 << 30, k=4) == m.MOE_EINVAL
    assert call(p=1.0) == call(rng=None) == call(dst=None) == call(out=None) == call(y=None) == m.MOE_EINVAL
    assert call(d=60) == call(y=P + 8) == call(res=P + 8) == call(out=P + 8) == m.MOE_EALIGN
    assert call(T=0, dst=None, out=None) == m.MOE_OK


def _glu(m, act=1, limit=0.0, p=0.0, rng=None):
    return ctypes.byref(m.MoeGlu(act, limit, p, rng))


BAD_FORMS = [dict(act=-1), dict(act=4), dict(limit=-1.0), dict(limit=float("nan")), dict(limit=float("inf")),
             dict(p=1.0), dict(p=float("nan")), dict(p=0.5), dict(p=0.5, rng=P + 4)]


def test_glu_refusals(m):
    lib = m.load()

    def fwd(g, dtype=m.MOE_BF16, d=64, x=P):
        return lib.moe_grouped_glu_fwd(dtype, g, x, P, P, P, 0, 2, 8, d, 64, P, P, P, None)

    def bwd(g, dtype=m.MOE_BF16, ws=256, dw2=P):
        return lib.moe_grouped_glu_bwd(dtype, g, P, P, P, P, P, P, P, 0, 2, 8, 64, 64, P, P, P, dw2, P, ws, None)

    def op(g, o=0, dtype=m.MOE_BF16):
        t = m.gemm_tensors(x_perm=P, w13=P, gu=P)      # no h
        return lib.moe_grouped_glu_op(o, dtype, g, ctypes.byref(t), P, 0, 2, 8, 64, 64, None)
    for kw in BAD_FORMS:
        assert fwd(_glu(m, **kw)) == bwd(_glu(m, **kw)) == op(_glu(m, **kw)) == m.MOE_EINVAL, kw
    for call in (fwd, bwd, op):
        assert call(None) == m.MOE_EINVAL
        for dt in (m.MOE_MXFP8, m.MOE_MXFP4, 9):
            assert call(_glu(m), dtype=dt) == m.MOE_EUNSUPPORTED
    assert fwd(_glu(m), d=60) == m.MOE_EALIGN and fwd(_glu(m), x=P + 8) == m.MOE_EALIGN
    assert fwd(_glu(m), x=None) == bwd(_glu(m), dw2=None) == m.MOE_EINVAL
    assert bwd(_glu(m), ws=255) == m.MOE_EWORKSPACE
    assert op(_glu(m)) == op(_glu(m), o=5) == op(_glu(m), o=-1) == m.MOE_EINVAL


def test_int4_codec_refusals(m):
    lib = m.load()

    def q(src=P, rows=4, K=128, g=64, codes=P, scales=P, zeros=None):
        return lib.moe_quantize_int4(src, rows, K, g, codes, scales, zeros, None)

    def dq(codes=P, scales=P, zeros=None, rows=4, K=128, g=64, dst=P):
        return lib.moe_dequantize_int4(codes, scales, zeros, rows, K, g, dst, None)
    for f in (q, dq):
        assert f(rows=-1) == f(K=0) == f(rows=1 << 31) == f(rows=1 << 30, K=1024) == m.MOE_EINVAL
        assert f(g=16) == f(g=0) == f(g=256) == m.MOE_EUNSUPPORTED
        assert f(K=96) == f(codes=P + 4) == f(scales=P + 1) == m.MOE_EALIGN
        assert f(codes=None) == f(scales=None) == m.MOE_EINVAL
        assert f(rows=0) == m.MOE_OK
    assert q(src=P + 8) == dq(dst=P + 8) == m.MOE_EALIGN
    assert q(src=None) == dq(dst=None) == m.MOE_EINVAL


def test_int4_ffn_refusals(m):
    lib = m.load()
    full = dict(codes=P, scales=P, zeros=None)

    def call(g=None, x=P, T=4, k=2, idx=P, w=P, dst=P, src=P, off=P, E=4, d=128, f=64, group=64, w13=full, w2=full, out=P,
             ws=P, wsb=1 << 20):
        a, b = (None if v is None else ctypes.byref(m.MoeInt4(v["codes"], v["scales"], v["zeros"])) for v in (w13, w2))
        return lib.moe_int4_ffn(g or _glu(m), x, T, k, idx, w, dst, src, off, E, d, f, group, a, b, out, ws, wsb, None, None)
    for kw in BAD_FORMS:
        assert call(g=_glu(m, **kw)) == m.MOE_EINVAL, kw
    assert call(g=_glu(m, p=0.5, rng=P)) == m.MOE_EUNSUPPORTED
    assert call(T=-1) == call(k=0) == call(k=9) == call(E=0) == call(E=1025) == call(T=1 << 30, k=4) == m.MOE_EINVAL
    assert call(d=0) == call(f=0) == call(d=1 << 21) == call(f=1 << 21) == m.MOE_EINVAL
    assert call(group=48) == m.MOE_EUNSUPPORTED and call(group=128) == call(d=96) == m.MOE_EALIGN
    for n in ("x", "idx", "w", "dst", "src", "off", "w13", "w2", "out"):
        assert call(**{n: None}) == m.MOE_EINVAL, n
    for n in ("w13", "w2"):
        assert call(**{n: dict(full, codes=None)}) == call(**{n: dict(full, scales=None)}) == m.MOE_EINVAL
        assert call(**{n: dict(full, codes=P + 8)}) == call(**{n: dict(full, scales=P + 1)}) == m.MOE_EALIGN
    assert call(x=P + 8) == call(out=P + 8) == m.MOE_EALIGN
    need = m.moe_int4_workspace_bytes(8, 128, 64)
    assert call(wsb=need - 1) == call(ws=None) == call(ws=P + 8) == m.MOE_EWORKSPACE
    assert call(T=0) == m.MOE_OK


def test_int4_workspace(m):
    assert m.moe_int4_workspace_bytes(-1, 64, 64) == m.moe_int4_workspace_bytes(4, 0, 64) == 0
    assert m.moe_int4_workspace_bytes(1 << 31, 64, 64) == m.moe_int4_workspace_bytes(4, 64, 1 << 21) == 0
    assert m.moe_int4_workspace_bytes(1000, 4096, 1536) >= 1000 * (4096 + 1536) * 2


# ------------------------------------------------------------------ refusals of the Python calls
def test_python_refusals(m):
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    x = torch.zeros(4, 64, dtype=bf)
    rng = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        m.moe_dropout(m.MOE_BF16, x, 0.1, rng, x)                      # not on a GPU
    with pytest.raises(ValueError):
        m.moe_dropout(m.MOE_BF16, x, 0.1, rng.int(), x)
    with pytest.raises(ValueError):
        m.moe_dropout(m.MOE_BF16, x, 0.1, rng, x.float())
    with pytest.raises(ValueError):
        m.moe_dropout(m.MOE_BF16, x[:, ::2], 0.1, rng, x[:, ::2])      # strided
    with pytest.raises(m.MoeError):
        m.moe_dropout(m.MOE_MXFP8, x, 0.1, rng, x)
    with pytest.raises(ValueError):
        m.glu(m.MOE_ACT_GELU, p=0.1, rng=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        m.moe_combine_dropout(m.MOE_BF16, x, torch.zeros(7, dtype=i32), None, 2, 0.1, rng, x)
    idx = torch.zeros(4, 2, dtype=i32)
    w = [(torch.zeros(3, n, k // 2, dtype=u8), torch.zeros(3, n, k // 64, dtype=bf), None) for n, k in ((128, 64), (64, 64))]

    def ffn(**kw):
        a = dict(gate=m.glu(), x=x, topk_idx=idx, topk_w=idx.float(), dst_row=idx.view(-1), src_slot=idx.view(-1),
                 group_off=torch.zeros(4, dtype=i32), group=64, w13=w[0], w2=w[1], out=x, ws=torch.zeros(1 << 16, dtype=u8))
        a.update(kw)
        m.moe_int4_ffn(**a)
    for kw in (dict(), dict(x=x.float()), dict(topk_idx=idx.long()), dict(dst_row=idx.view(-1)[:7]), dict(w13=w[1]),
               dict(w2=(w[1][0], w[1][1].float(), None)), dict(w2=(w[1][0], w[1][1], w[1][0])), dict(out=x[:3]),
               dict(src_slot=idx.view(-1).long())):
        with pytest.raises(ValueError):
            ffn(**kw)
    with pytest.raises(m.MoeError):
        ffn(group=16)


@pytest.mark.parametrize("kw", [dict(act=4), dict(act=-1), dict(limit=-1.0), dict(limit=float("nan")), dict(h_dropout=1.0),
                                dict(out_dropout=-0.1), dict(h_dropout=float("nan")),
                                dict(dtype="MXFP8", act=1), dict(dtype="MXFP4", limit=1.0), dict(dtype="MXFP8", h_dropout=0.1),
                                dict(dtype="INT4", h_dropout=0.1), dict(dtype="INT4", out_dropout=0.1),
                                dict(dtype="INT4", capacity=8), dict(dtype="INT4", group=16), dict(dtype="INT4", d=96)])
def test_layer_refusals(m, kw):
    from routing_grouped_gemm_amd.layer import MoELayer
    kw = dict(kw)
    dtype = getattr(m, "MOE_" + kw.pop("dtype", "BF16"))
    with pytest.raises(ValueError):
        MoELayer(8, kw.pop("d", 128), 4, 128, 2, dtype, device="cpu", **kw)


def test_int4_layer_refusals(m):
    from routing_grouped_gemm_amd.layer import MoELayer
    lay = MoELayer(8, 128, 4, 128, 2, m.MOE_INT4, device="cpu", group=64, zeros=True)
    u8, bf = torch.uint8, torch.bfloat16

    def w(N, K, g=64, z=True):
        return (torch.zeros(4, N, K // 2, dtype=u8), torch.zeros(4, N, K // g, dtype=bf),
                torch.zeros(4, N, K // g, dtype=u8) if z else None)
    lay.set_weights_int4(w(256, 128), w(128, 128))
    had = lay.w13_4, lay.w2_4
    for a, b in ((w(256, 128, 32), w(128, 128)), (w(256, 128), w(256, 128)), (w(128, 128), w(128, 128))):
        with pytest.raises(ValueError):
            lay.set_weights_int4(a, b)
    with pytest.raises(ValueError):
        lay.set_weights(torch.zeros(4, 256, 128, dtype=bf), torch.zeros(4, 128, 128))
    assert (lay.w13_4, lay.w2_4) == had
    with pytest.raises(ValueError):
        lay.gemm_stage(m.MOE_GEMM_GATE_UP)
    with pytest.raises(RuntimeError):
        lay.backward(torch.zeros(8, 128, dtype=bf))
    with pytest.raises(ValueError):
        MoELayer(8, 128, 4, 128, 2, device="cpu").set_weights_int4(w(256, 128), w(128, 128))


def test_int4_layer_parts_are_refused(m):
    from routing_grouped_gemm_amd.layer import MoELayer
    lay = MoELayer(8, 128, 4, 128, 2, m.MOE_INT4, device="cpu", group=64)
    x = torch.zeros(8, 128, dtype=torch.bfloat16)
    for call in (lambda: lay.permute(x), lay.gemm_fwd, lay.combine, lambda: lay.gate_grad(x)):
        with pytest.raises(ValueError):
            call()
    codes = torch.zeros(4, 256, 64, dtype=torch.uint8), torch.zeros(4, 256, 2, dtype=torch.bfloat16)
    down = torch.zeros(4, 128, 64, dtype=torch.uint8), torch.zeros(4, 128, 2, dtype=torch.bfloat16), None
    for bad in (codes, (codes[0], None, None), (None, codes[1], None)):
        with pytest.raises(ValueError):
            lay.set_weights_int4(bad, down)
