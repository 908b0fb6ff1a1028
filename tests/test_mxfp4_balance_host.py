"""CPU checks: the plain MXFP4 codec and balance loss the GPU tests compare
with, and the refusals of the C entry points (nothing is launched: every call
fails validation, or has nothing to do)."""
import ctypes
import os

import numpy as np
import pytest
import torch

from tests import _plain

FAKE = 0x10000          # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def m():
    import routing_grouped_gemm_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return m


# ------------------------------------------------------------------ the plain implementations
def test_plain_codec_properties():
    rng = np.random.default_rng(1)
    v = _plain.bf16_round(rng.standard_normal((40, 96)) * np.exp2(rng.integers(-120, 120, (40, 1))))
    v[3, :32] = 0
    q = _plain.mxfp4_qdq(v)
    codes, scales = _plain.mxfp4_quantize(v)
    top = np.abs(v.reshape(40, 3, 32)).max(-1)
    s = 2.0 ** (scales.astype(np.float64) - 127)
    assert np.all(top <= 6 * s)                                     # the maximum never overflows
    assert np.all((top > 3 * s) | (scales == 0))                    # and the next smaller power would
    # nearest: no representable value is nearer
    grid = np.concatenate([_plain.E2M1, -_plain.E2M1])
    cand = grid * s[..., None, None]
    d = np.abs(cand - v.reshape(40, 3, 32, 1)).min(-1)
    assert np.array_equal(np.abs(q - v).reshape(40, 3, 32), d)
    # a midpoint takes the value with the even code: 0.25 0.75 1.25 1.75 2.5 3.5 5
    w = np.zeros((1, 32))
    w[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    assert list(_plain.mxfp4_qdq(w)[0, :8]) == [6, 0, 1, 1, 2, 2, 4, 4]
    # values that are representable under their own scale come back
    assert np.array_equal(_plain.mxfp4_qdq(q), q)


def test_plain_balance_against_autograd_and_differences():
    rng = np.random.default_rng(2)
    T, E, k = 19, 6, 2
    x = rng.standard_normal((T, E)) * 2
    idx = np.argsort(-x, 1)[:, :k]
    seg, mask = [1, 7, 7, 16], (rng.random(T) > 0.3).astype(np.uint8)
    cb, cz, dl = 0.7, 0.3, (1.5, -0.5)
    r = _plain.balance(x, idx, cb, cz, seg, mask, dl)
    # torch, written another way
    xt = torch.tensor(x, requires_grad=True)
    on = np.zeros(T, bool)
    on[seg[0]:seg[-1]] = True
    on &= mask != 0
    N = on.sum()
    bal = 0
    for a, b in zip(seg[:-1], seg[1:]):
        sel = [t for t in range(a, b) if on[t]]
        if sel:
            hits = torch.bincount(torch.tensor(idx[sel]).reshape(-1), minlength=E).double()
            bal = bal + len(sel) / N * E * (hits / hits.sum() * torch.softmax(xt[sel], 1).mean(0)).sum()
    z = (torch.logsumexp(xt[torch.tensor(on)], 1) ** 2).sum() / N
    np.testing.assert_allclose(r["losses"], [cb * bal.item(), cz * z.item()], rtol=1e-12)
    (g,) = torch.autograd.grad(dl[0] * cb * bal + dl[1] * cz * z, xt)
    np.testing.assert_allclose(r["grad"], g.numpy(), rtol=1e-9, atol=1e-14)
    # central differences, the counts held
    eps = 1e-6
    for t, e in [(0, 0), (3, 2), (8, 5), (15, 1), (18, 4)]:
        hi, lo = x.copy(), x.copy()
        hi[t, e] += eps
        lo[t, e] -= eps
        d = (np.dot(_plain.balance(hi, idx, cb, cz, seg, mask, dl, r["counts"])["losses"], dl)
             - np.dot(_plain.balance(lo, idx, cb, cz, seg, mask, dl, r["counts"])["losses"], dl)) / (2 * eps)
        assert abs(d - r["grad"][t, e]) <= 1e-7 + 1e-6 * abs(d)
    # at even load the balance loss is its coefficient, whatever the counts' total
    even = _plain.balance(np.zeros((12, 4)), np.arange(24).reshape(12, 2) % 4, cb, 0.0)
    np.testing.assert_allclose(even["losses"][0], cb, rtol=1e-12)


# ------------------------------------------------------------------ refusals
def test_mxfp4_quantiser_validation(m):
    lib = m.load()
    P = FAKE
    for fn in (lib.moe_quantize_mxfp4, lambda a, r, k, b, c, s: lib.moe_dequantize_mxfp4(b, c, r, k, a, s)):
        assert fn(P, -1, 64, P, P, None) == m.MOE_EINVAL
        assert fn(P, 1 << 31, 64, P, P, None) == m.MOE_EINVAL
        assert fn(P, 1 << 30, 1 << 20, P, P, None) == m.MOE_EINVAL
        assert fn(P, 10, 0, P, P, None) == m.MOE_EINVAL
        assert fn(None, 10, 64, P, P, None) == m.MOE_EINVAL
        assert fn(P, 10, 64, None, P, None) == m.MOE_EINVAL
        assert fn(P, 10, 64, P, None, None) == m.MOE_EINVAL
        assert fn(P, 10, 48, P, P, None) == m.MOE_EALIGN
        assert fn(P + 8, 10, 64, P, P, None) == m.MOE_EALIGN
        assert fn(P, 10, 64, P + 4, P, None) == m.MOE_EALIGN
        assert fn(None, 0, 64, None, None, None) == m.MOE_OK          # nothing to do


def test_mxfp4_permute_validation(m):
    lib = m.load()
    P = FAKE

    def call(x=P, d=64, scale=None, xs=P, n_rows=20, src=None, xp=P):
        return lib.moe_permute(m.MOE_MXFP4, x, 10, d, 2, P, src, scale, n_rows, xp, xs, None, None)
    assert call(d=48) == m.MOE_EALIGN
    assert call(x=P + 8) == m.MOE_EALIGN
    assert call(xp=P + 8) == m.MOE_EALIGN
    assert call(scale=P) == m.MOE_EUNSUPPORTED
    assert call(xs=None) == m.MOE_EINVAL
    assert call(n_rows=24) == m.MOE_EINVAL                            # padded: needs src_slot


def test_mxfp4_gemm_validation(m):
    lib = m.load()
    P = FAKE
    wsb = lib.moe_gemm_workspace_bytes(m.MOE_MXFP4, 8, 100, 128, 256)
    assert wsb >= 100 * 256 * 17 // 32

    def fwd(goff=P, C=0, n_rows=100, d=128, f=256, xp=P, xs=P, w13=P, ws13=P, w2=P, ws2=P, gu=P, h=P, y=P, ws=P,
            wsb=wsb):
        return lib.moe_grouped_gemm_fwd(m.MOE_MXFP4, xp, xs, w13, ws13, w2, ws2, goff, C, 8, n_rows, d, f, gu, h, y,
                                        ws, wsb, None)
    assert fwd(d=192) == m.MOE_EALIGN
    assert fwd(f=64) == m.MOE_EALIGN
    assert fwd(d=(1 << 20) + 128) == m.MOE_EINVAL
    assert fwd(f=(1 << 20) + 128) == m.MOE_EINVAL
    assert fwd(goff=None) == m.MOE_EINVAL
    assert fwd(C=10) == m.MOE_EINVAL
    for name in ("xp", "xs", "w13", "ws13", "w2", "ws2", "y"):
        assert fwd(**{name: None}) == m.MOE_EINVAL, name
        assert fwd(**{name: P + 4}) == m.MOE_EALIGN, name
    assert fwd(gu=P + 8) == m.MOE_EALIGN
    assert fwd(h=P + 8) == m.MOE_EALIGN
    for ws, b in ((None, wsb), (P, wsb - 1), (P + 8, wsb)):
        assert fwd(ws=ws, wsb=b) == m.MOE_EWORKSPACE
    # no backward of its own
    assert lib.moe_grouped_gemm_bwd(m.MOE_MXFP4, P, P, P, P, P, P, P, P, P, P, 0, 8, 100, 128, 256, P, P, P, P, P,
                                    1 << 30, None) == m.MOE_EUNSUPPORTED
    t = m.MoeGemmTensors(**{n: P for n in m.GEMM_TENSOR_FIELDS})
    t.ws_bytes = wsb

    def op(o, **over):
        tt = m.MoeGemmTensors.from_buffer_copy(t)
        for n, v in over.items():
            setattr(tt, n, v)
        return lib.moe_grouped_gemm_op(o, m.MOE_MXFP4, ctypes.byref(tt), P, 0, 8, 100, 128, 256, None)
    for o in (m.MOE_GEMM_DGRAD_DOWN, m.MOE_GEMM_DGRAD_GATE_UP, m.MOE_GEMM_WGRAD):
        assert op(o) == m.MOE_EUNSUPPORTED
    assert op(m.MOE_GEMM_GATE_UP, x_perm=None) == m.MOE_EINVAL
    assert op(m.MOE_GEMM_GATE_UP, w13=None) == m.MOE_EINVAL
    assert op(m.MOE_GEMM_GATE_UP, x_perm_scales=None) == m.MOE_EINVAL
    assert op(m.MOE_GEMM_GATE_UP, w13_scales=P + 4) == m.MOE_EALIGN
    assert op(m.MOE_GEMM_GATE_UP, gu=P + 8) == m.MOE_EALIGN
    assert op(m.MOE_GEMM_GATE_UP, ws=None) == m.MOE_EWORKSPACE
    assert op(m.MOE_GEMM_DOWN, w2_scales=None) == m.MOE_EINVAL
    assert op(m.MOE_GEMM_DOWN, y_perm=None) == m.MOE_EINVAL
    assert op(m.MOE_GEMM_DOWN, y_perm=P + 8) == m.MOE_EALIGN
    assert op(m.MOE_GEMM_DOWN, ws_bytes=wsb - 1) == m.MOE_EWORKSPACE
    assert op(m.MOE_GEMM_GATE_UP, dw13_f32=P, dw2_f32=P) == m.MOE_EUNSUPPORTED


def test_balance_validation(m):
    lib = m.load()
    P = FAKE
    assert lib.moe_balance_workspace_bytes(-1, 8, 1) == 0
    assert lib.moe_balance_workspace_bytes(10, 1025, 1) == 0
    assert lib.moe_balance_workspace_bytes(10, 8, 0) == 0
    wsb = lib.moe_balance_workspace_bytes(100, 8, 3)
    assert wsb > 0

    def fwd(lg=P, idx=P, seg=P, S=3, T=100, E=8, k=2, losses=P, counts=P, probs=P, tokens=P, ws=P, wsb=wsb):
        return lib.moe_balance_loss(lg, idx, None, seg, S, T, E, k, 0.1, 0.1, losses, counts, probs, None, tokens, ws,
                                    wsb, None, None)
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=1), dict(S=0),
                dict(S=(1 << 20) + 1), dict(seg=None), dict(lg=None), dict(idx=None), dict(losses=None),
                dict(counts=None), dict(probs=None), dict(tokens=None), dict(T=1 << 30)):
        assert fwd(**bad) == m.MOE_EINVAL, bad
    for ws, b in ((None, wsb), (P, wsb - 1), (P + 4, wsb)):
        assert fwd(ws=ws, wsb=b) == m.MOE_EWORKSPACE

    def bwd(lg=P, seg=P, S=3, T=100, E=8, counts=P, tokens=P, dl=P):
        return lib.moe_balance_loss_bwd(lg, None, seg, S, T, E, counts, tokens, 0.1, 0.1, None, None, dl, None)
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(S=0), dict(seg=None), dict(lg=None), dict(counts=None),
                dict(tokens=None), dict(dl=None)):
        assert bwd(**bad) == m.MOE_EINVAL, bad
    assert bwd(T=0, lg=None, dl=None) == m.MOE_OK


def test_balance_refuses_token_numbers_that_leave_32_bits(m):
    lib = m.load()
    P, T = FAKE, (1 << 30) + 1
    assert lib.moe_balance_workspace_bytes(T - 1, 1, 1) > 0 and lib.moe_balance_workspace_bytes(T, 1, 1) == 0
    assert lib.moe_balance_loss(P, P, None, None, 1, T, 1, 1, 0.1, 0.1, P, P, P, None, P, P, 1 << 40, None,
                                None) == m.MOE_EINVAL
    assert lib.moe_balance_loss_bwd(P, None, None, 1, T, 1, P, P, 0.1, 0.1, None, None, P, None) == m.MOE_EINVAL


def test_python_calls_refuse_what_is_not_dense(m):
    """The Python entry points check types, shapes and strides before anything is passed on."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    with pytest.raises(ValueError):                       # not on a GPU
        m.moe_dequantize_mxfp4(u8(4, 32), u8(4, 2), x)
    with pytest.raises(ValueError):
        m._dense("x", x[:, ::2], torch.bfloat16, 4, 32)
    with pytest.raises(ValueError):                       # another shape, another type
        m._dense("x", x, torch.bfloat16, 4, 32)
    with pytest.raises(ValueError):
        m._dense("x", x, torch.float32, 4, 64)
    # MXFP4 calls: what lies on the host, a destination per slot
    dst = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError):
        m.moe_permute(m.MOE_MXFP4, x, 2, dst, u8(8, 32), x_perm_scales=u8(8, 2))
    with pytest.raises(ValueError):
        m.moe_permute(m.MOE_MXFP4, x, 2, dst[:7], u8(8, 32), x_perm_scales=u8(8, 2))
    off = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        m.moe_grouped_gemm_fwd(m.MOE_MXFP4, u8(4, 64), u8(1, 256, 64), u8(1, 128, 64), off, 0, None, None,
                               torch.zeros(4, 128, dtype=torch.bfloat16), x_perm_scales=u8(4, 4),
                               w13_scales=u8(1, 256, 4), w2_scales=u8(1, 128, 4), ws=u8(4096))
