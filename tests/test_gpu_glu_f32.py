"""fp32 gated blocks in launches large enough for tiles of 64 x 64, and at either side of the number of tiles where they
take over from those of 32 x 32: each stage against its formula in 64 bits, and the same bits from either tile."""
import pytest
import torch

from tests.test_gpu_glu import BF, F32, Block, _say, moe  # noqa: F401  (moe: the fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _tiles(rows, E, cols):
    """Tiles of 64 x 64 as the host bounds them; from 512 on they are the ones that run."""
    return (rows // 64 + E) * -(-cols // 64)


@pytest.mark.parametrize("limit,p", [(0.0, 0.0), (1.5, 0.2)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("d,f", [(1348, 1412), (260, 1412), (1412, 260)])
def test_large_launches(moe, d, f, act, limit, p):  # noqa: F811
    """Groups that end at, before and behind a tile's rows, columns and K that end inside a tile, an empty group."""
    _say("f32 large", d, f, act, limit, p)
    counts = [300, 64, 129, 513, 0, 40, 1, 63]
    R = sum(counts) + 5
    # gate and up; down and its gradient; the gradient of h: at the first sizes all of them, then where they are long
    assert all(_tiles(R, len(counts), cols) >= 512 for cols in (2 * f, d, f) if cols > 1300)
    b = Block(moe, counts, d, f, F32, act, limit, p, seed=len(act))
    b.forward()
    b.backward()
    b.check()


def test_large_launches_of_a_padded_layout(moe):  # noqa: F811
    assert all(_tiles(1400, 7, cols) >= 512 for cols in (2 * 1156, 1156))
    b = Block(moe, [0] * 7, 1156, 1156, F32, "gelu", 1.5, 0.2, capacity=200)
    b.forward()
    b.backward()
    b.check()


def test_large_launches_of_one_row_a_group(moe):  # noqa: F811
    """More than a hundred groups, most tiles with one row."""
    b = Block(moe, [1, 0, 2] * 40, 260, 516, F32, "relu", 1.0, 0.3, seed=9)
    assert _tiles(b.R, 120, 516) >= 512
    b.forward()
    b.backward()
    b.check()


@pytest.mark.parametrize("plain", [False, True])
@pytest.mark.parametrize("d,f", [(516, 1028), (1028, 260), (132, 68)])
def test_either_tile_has_the_same_bits(moe, d, f, plain):  # noqa: F811
    """A group by itself takes tiles of 32 x 32, many of it those of 64 x 64: the sums are the same chain of additions."""
    m, n = moe, 333
    E = 4
    while _tiles(n * E, E, min(d, f)) < 512:
        E *= 2
    assert _tiles(n, 1, max(d, 2 * f)) < 512
    _say("f32 alone", d, f, plain, E)
    g = torch.Generator(DEV).manual_seed(3)

    def make(*shape, s=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * s
    one = dict(x_perm=make(n, d), dy_perm=make(n, d), w13=make(1, 2 * f, d, s=d ** -0.5), w2=make(1, d, f, s=f ** -0.5))
    gate = m.glu() if plain else m.glu(m.MOE_ACT_GELU, 1.0)      # (a mask is the row's, and these are other rows)
    outs = []
    for reps in (1, E):
        t = {k: v.repeat(reps, *[1] * (v.dim() - 1)).contiguous() for k, v in one.items()}
        R = n * reps
        t.update({k: torch.full((R, w), 7.0, device=DEV)
                  for k, w in (("gu", 2 * f), ("h", f), ("y_perm", d), ("dgu", 2 * f), ("dx_perm", d))})
        t.update(dw13=torch.full_like(t["w13"], 7.0), dw2=torch.full_like(t["w2"], 7.0))
        off = torch.arange(0, R + 1, n, dtype=torch.int32, device=DEV)
        args = m.gemm_tensors(**t)
        for op in range(5):
            if plain:
                m.moe_grouped_gemm_op(op, m.MOE_F32, args, off, 0, reps, R, d, f)
            else:
                m.moe_grouped_glu_op(op, m.MOE_F32, gate, args, off, 0, reps, R, d, f)
        outs.append(t)
    torch.cuda.synchronize()
    for k in ("gu", "h", "y_perm", "dgu", "dx_perm", "dw13", "dw2"):
        a = outs[0][k]
        b = outs[1][k].view(E, *(a.shape if a.dim() == 2 else a.shape[1:]))
        assert bool((a.view(b.shape[1:]) == b).all()), k
