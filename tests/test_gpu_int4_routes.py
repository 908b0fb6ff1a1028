"""4-bit integer experts under routes with dropped slots, destinations and experts out of range, and rows that belong to no
slot, in each of the call's forms: single tokens, few and many rows an expert."""
import pytest
import torch

from tests.test_gpu_int4 import Ffn, _say, moe  # noqa: F401  (moe: the fixture)

pytestmark = pytest.mark.gpu
E, K = 8, 2
# tokens of 2 slots of 8 experts: up to 12 slots go slot by slot, up to 255 take tiles of 16 rows, more those of 64
FORMS = [5, 30, 100, 128, 200, 333]


def _case(moe, T, group=64, zeros=True):  # noqa: F811
    _say("routes", T, group, zeros)
    return Ffn(moe, T, E, 192 if group < 128 else 256, 128, K, group, zeros, act="gelu", limit=2.0, seed=T)


def _live(T):
    return torch.ones(T, K, dtype=torch.bool)


@pytest.mark.parametrize("T", FORMS)
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
def test_dropped_slots(moe, T, group, zeros):  # noqa: F811
    """They add nothing and are no fault; a token with none left gets zeros."""
    c, live = _case(moe, T, group, zeros), _live(T)
    live[::3, 0] = False
    live[T // 2] = False
    c.route["dst_row"].view(T, K)[~live] = -1
    out = c.run()
    c.check(out, live)
    assert int(c.err) == 0 and not bool(out[T // 2].any())


@pytest.mark.parametrize("T", FORMS)
@pytest.mark.parametrize("past", [0, 5, 2 ** 31 - 1])
def test_rows_out_of_range(moe, T, past):  # noqa: F811
    """A destination behind the rows: flagged, and the slot adds nothing."""
    c, live = _case(moe, T), _live(T)
    for t, j in ((0, 1), (T - 1, 0), (T // 2, 1)):
        live[t, j] = False
        c.route["dst_row"][t * K + j] = min(T * K + past, 2 ** 31 - 1)
    c.check(c.run(), live)
    assert int(c.err) == moe.MOE_ERR_ROW_RANGE


@pytest.mark.parametrize("T", FORMS)
@pytest.mark.parametrize("bad", [E, -1, 2 ** 30, -2 ** 31])
def test_experts_out_of_range(moe, T, bad):  # noqa: F811
    c, live = _case(moe, T), _live(T)
    keep = c.route["topk_idx"].clone()
    for t, j in ((0, 0), (T - 1, 1), (T // 2, 0)):
        live[t, j] = False
        c.route["topk_idx"][t, j] = bad
    out = c.run()
    c.route["topk_idx"] = keep
    c.check(out, live)
    assert int(c.err) == moe.MOE_ERR_ROW_RANGE


@pytest.mark.parametrize("T", [T for T in FORMS if T > 6])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("past", [0, 3, 2 ** 30, None])
def test_rows_of_no_slot(moe, T, group, past):  # noqa: F811
    """Rows whose src_slot is negative (None: those alone) are of no token, and so are those whose src_slot is past the
    slots, which are flagged: what would read them adds nothing.  (The form for single tokens reads no src_slot.)"""
    c, live = _case(moe, T, group), _live(T)
    src, owner = c.route["src_slot"], c.route["src_slot"].clone().long()
    rows = [0, 1, 17, T * K // 2, T * K - 1]
    for i, r in enumerate(rows):
        src[r] = (-1, -2 ** 31)[i // 2 % 2] if past is None or i % 2 == 0 else T * K + past
        live.view(-1)[owner[r]] = False
    c.check(c.run(), live)
    assert int(c.err) == (0 if past is None else moe.MOE_ERR_ROW_RANGE)


def test_an_expert_of_rows_of_no_slot_alone(moe):  # noqa: F811
    """Every row of two experts, among them whole tiles of 64."""
    for T in (60, 400):
        c, live = _case(moe, T), _live(T)
        off = c.route["group_off"].tolist()
        for e, v in ((1, -1), (6, T * K)):
            rows = slice(off[e], off[e + 1])
            live.view(-1)[c.route["src_slot"][rows].long()] = False
            c.route["src_slot"][rows] = v
        c.check(c.run(), live)
        assert int(c.err) == moe.MOE_ERR_ROW_RANGE
