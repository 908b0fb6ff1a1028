"""MXFP4 calls that the interface allows and a layer does not make: one saved activation without the other, no tokens
into a padded layout, weights with a NaN scale, two forwards on two streams at once."""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _say(*a):
    print("[gpu-mx4-calls]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


def _operand(moe, shape, seed, scale):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn(*shape, generator=g, device=DEV) * scale).to(torch.bfloat16)
    K = shape[-1]
    codes = torch.empty(*shape[:-1], K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(*shape[:-1], K // 32, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_mxfp4(x.view(-1, K), codes.view(-1, K // 2), scales.view(-1, K // 32))
    return codes, scales


def _case(moe, sizes, d, f, seed):
    E, R = len(sizes), sum(sizes)
    q = dict(zip(("x", "xs"), _operand(moe, (R, d), seed, 1.0)))
    q.update(zip(("w13", "w13s"), _operand(moe, (E, 2 * f, d), seed + 1, d ** -0.5)))
    q.update(zip(("w2", "w2s"), _operand(moe, (E, d, f), seed + 2, f ** -0.5)))
    off = [0]
    for s in sizes:
        off.append(off[-1] + s)
    q["off"] = torch.tensor(off, dtype=torch.int32, device=DEV)
    q["ws"] = torch.full((moe.moe_gemm_workspace_bytes(moe.MOE_MXFP4, E, R, d, f),), 0xFF, dtype=torch.uint8, device=DEV)
    q["d"], q["f"], q["R"] = d, f, R
    return q


def _forward(moe, q, gu=True, h=True):
    bf = dict(dtype=torch.bfloat16, device=DEV)
    g = torch.full((q["R"], 2 * q["f"]), 9.0, **bf) if gu else None
    hh = torch.full((q["R"], q["f"]), 9.0, **bf) if h else None
    y = torch.full((q["R"], q["d"]), 9.0, **bf)
    moe.moe_grouped_gemm_fwd(moe.MOE_MXFP4, q["x"], q["w13"], q["w2"], q["off"], 0, g, hh, y, x_perm_scales=q["xs"],
                             w13_scales=q["w13s"], w2_scales=q["w2s"], ws=q["ws"])
    return g, hh, y


@pytest.mark.parametrize("sizes,d,f", [
    ([3, 1, 2], 256, 128),                                   # few rows
    ([200, 511, 0, 64], 1152, 640), ([70, 0, 260, 90], 256, 384),   # 64- and 128-row tiles
    ([257, 0, 512, 700, 255, 1000], 640, 1536),              # 256-row tiles
])
def test_one_saved_activation_without_the_other(moe, sizes, d, f):
    _say("saved", sizes, d, f)
    q = _case(moe, sizes, d, f, 3)
    gu, h, y = _forward(moe, q)
    g1, _, y1 = _forward(moe, q, h=False)
    _, h2, y2 = _forward(moe, q, gu=False)
    torch.cuda.synchronize()
    assert torch.equal(g1, gu) and torch.equal(h2, h)
    assert torch.equal(y1, y) and torch.equal(y2, y)


def test_no_tokens_into_a_padded_layout(moe):
    _say("no tokens")
    codes = torch.full((12, 32), 0xAA, dtype=torch.uint8, device=DEV)
    scales = torch.full((12, 2), 0xAA, dtype=torch.uint8, device=DEV)
    none = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    dst = torch.empty(0, dtype=torch.int32, device=DEV)
    src = torch.full((12,), -1, dtype=torch.int32, device=DEV)
    src[5] = 0                                               # a row that some slot owns stays as it is
    moe.moe_permute(moe.MOE_MXFP4, none, 2, dst, codes, src_slot=src, x_perm_scales=scales)
    torch.cuda.synchronize()
    keep = torch.zeros(12, dtype=torch.bool, device=DEV)
    keep[5] = True
    assert not bool(codes[~keep].any()) and not bool(scales[~keep].any())
    assert bool((codes[keep] == 0xAA).all()) and bool((scales[keep] == 0xAA).all())


@pytest.mark.parametrize("sizes,d,f", [([3, 2], 256, 128), ([300, 200], 256, 1536)])
def test_a_weight_block_that_is_nan(moe, sizes, d, f):
    """A NaN scale in one row of one expert's W13 (W2) makes that column of its rows NaN and no other."""
    _say("nan weights", sizes)
    q = _case(moe, sizes, d, f, 7)
    gu0, _, y0 = _forward(moe, q)
    clean = q["w13s"].clone()
    q["w13s"][1, 70, 3] = 255                                # gate row 70 of expert 1
    gu, h, y = _forward(moe, q)
    torch.cuda.synchronize()
    n = sizes[0]
    assert bool(gu[n:, 70].isnan().all()) and bool(h[n:, 70].isnan().all()) and bool(y[n:].isnan().all())
    others = torch.arange(2 * f, device=DEV) != 70
    assert torch.equal(gu[:, others], gu0[:, others]) and torch.equal(gu[:n], gu0[:n]) and torch.equal(y[:n], y0[:n])
    q["w13s"] = clean
    q["w2s"][0, 33, f // 32 - 1] = 255
    _, _, y = _forward(moe, q)
    torch.cuda.synchronize()
    others = torch.arange(d, device=DEV) != 33
    assert bool(y[:n, 33].isnan().all()) and torch.equal(y[:, others], y0[:, others]) and torch.equal(y[n:], y0[n:])


def test_two_streams_at_once(moe):
    _say("streams")
    cases = [_case(moe, [300, 17, 600, 129], 512, 384, 11), _case(moe, [5, 0, 1, 9], 512, 384, 12),
             _case(moe, [257, 700, 255, 1000, 900, 100], 640, 1536, 13)]
    refs = [_forward(moe, q) for q in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for rep in range(4):
        for q, s in zip(cases, streams):
            with torch.cuda.stream(s):
                outs.append(_forward(moe, q))
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        for a, b in zip(got, refs[i % 3]):
            assert torch.equal(a, b), i
