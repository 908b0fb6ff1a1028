"""GPU parity of the router's balance loss against the plain 64-bit one.

Tolerances count roundings.  With R the largest distance of a counted logit
from its row's maximum, p = exp(x - max) / sum is off by a relative
(R + 8) 2^-22: the difference and its product with log2 e (2^-24 R each, and
the hardware exponential's and the reciprocal's last places), the sum of E
positive terms, which the butterfly adds in a few steps; a term that underflows
is off by 2^-126.  A mean over n tokens adds n 2^-24.
"""
import sys

import numpy as np
import pytest
import torch

import moe_synth
from tests import _plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _say(*a):
    print("[gpu-balance]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


def _run(moe, x, idx, cb, cz, seg=None, mask=None, dl=None, add=None, alias=False, lse=True):
    T, E = x.shape
    S = 1 if seg is None else len(seg) - 1
    dev = lambda a, t: None if a is None else torch.as_tensor(np.asarray(a)).to(t).to(DEV)
    xg, ig = x.to(DEV), idx.to(torch.int32).to(DEV)
    o = dict(losses=torch.full((2,), 9.0, device=DEV), counts=torch.full((S, E), -7, dtype=torch.int32, device=DEV),
             probs=torch.full((S, E), 9.0, device=DEV), lse=torch.full((T,), 9.0, device=DEV) if lse else None,
             tokens=torch.full((S + 1,), -7, dtype=torch.int32, device=DEV),
             err=torch.zeros(1, dtype=torch.int32, device=DEV))
    ws = torch.full((moe.moe_balance_workspace_bytes(T, E, S),), 0xFF, dtype=torch.uint8, device=DEV)
    sg, mg, dg, ag = dev(seg, torch.int32), dev(mask, torch.uint8), dev(dl, torch.float32), dev(add, torch.float32)
    moe.moe_balance_loss(xg, ig, cb, cz, o["losses"], o["counts"], o["probs"], o["lse"], o["tokens"], ws, seg_off=sg,
                         mask=mg, dev_err=o["err"])
    o["grad"] = ag.clone() if alias else torch.full((T, E), 9.0, device=DEV)
    moe.moe_balance_loss_bwd(xg, o["counts"], o["tokens"], cb, cz, o["grad"], dlosses=dg,
                             add=o["grad"] if alias else ag, seg_off=sg, mask=mg)
    torch.cuda.synchronize()
    return {n: None if v is None else v.cpu().numpy() for n, v in o.items()}


def _check(o, x, idx, cb, cz, seg=None, mask=None, dl=(1.0, 1.0), add=None):
    x = x.numpy().astype(np.float64)
    T, E = x.shape
    r = _plain.balance(x, idx.numpy(), cb, cz, seg, mask, dl)
    np.testing.assert_array_equal(o["counts"], r["counts"])
    np.testing.assert_array_equal(o["tokens"], r["tokens"])
    fin = np.isfinite(x)
    span = np.where(fin, x, -np.inf).max(1) - np.where(fin, x, np.inf).min(1)
    R = float(np.clip(span, 0.0, 104.0).max()) if T else 0.0
    rel = (R + 8) * 2.0 ** -22
    tiny = 2.0 ** -120
    n = np.maximum(r["tokens"][:-1], 1)[:, None]
    assert np.all(np.abs(o["probs"] - r["probs"]) <= r["probs"] * (rel + n * 2.0 ** -24) + tiny)
    big = np.abs(np.nan_to_num(np.where(np.isfinite(x), x, 0))).max(1) if T and E else np.zeros(T)
    ltol = (np.abs(r["lse"]) + big) * 2.0 ** -23 + rel
    if o["lse"] is not None:
        assert np.all(np.abs(o["lse"] - r["lse"]) <= np.where(r["lse"] != 0, ltol, 0) + (r["lse"] == 0) * rel)
    N = max(int(r["tokens"][-1]), 1)
    assert abs(o["losses"][0] - r["losses"][0]) <= abs(r["losses"][0]) * (rel + N * 2.0 ** -24 + 2.0 ** -22) + tiny
    zt = cz / N * (2 * np.abs(r["lse"]) * ltol + ltol ** 2).sum()
    assert abs(o["losses"][1] - r["losses"][1]) <= abs(r["losses"][1]) * (N * 2.0 ** -24 + 2.0 ** -22) + zt
    # the gradient: relative to the sizes of its two terms before they cancel
    kb, kz = abs(dl[0] * cb) * E / N, abs(dl[1] * cz) * 2 / N
    mag = r["p"] * (kb * (r["f"] + r["dot"]) + kz * np.abs(r["lse"])[:, None])
    want = r["grad"] + (0 if add is None else add)
    gtol = mag * 2 * (rel + 2.0 ** -20) + r["p"] * kz * ltol[:, None] + 2.0 ** -23 * np.abs(want) + tiny
    assert np.all(np.abs(o["grad"] - want) <= gtol)
    return r


def _inputs(T, E, k, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g) * spread
    return x, torch.topk(x, k, dim=1).indices if T else torch.zeros(0, k, dtype=torch.int64)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 4, 1), (63, 3, 2), (64, 5, 3), (65, 8, 2), (100, 13, 4), (130, 30, 1),
                                   (257, 64, 8), (300, 100, 2), (1000, 128, 4), (200, 130, 2), (129, 256, 8),
                                   (70, 500, 3), (90, 1024, 8), (66000, 16, 2)])
def test_one_sequence(moe, T, E, k):
    _say("one", T, E, k)
    x, idx = _inputs(T, E, k, T + E)
    o = _run(moe, x, idx, 0.01, 0.001)
    _check(o, x, idx, 0.01, 0.001)
    assert o["err"][0] == 0


@pytest.mark.parametrize("T,E,k,seg,masked", [
    (200, 128, 4, [0, 0, 64, 64, 100, 200, 200], False),       # empty sequences, ends on and inside runs
    (200, 128, 4, [10, 20, 190], True),                        # tokens before the first and behind the last
    (130, 12, 2, list(range(131)), True),                      # one token each
    (500, 40, 2, [0, 499, 500], False), (64, 8, 2, [64, 64], False), (70, 8, 2, [0, 0, 0], True),
    (70000, 8, 1, [5, 128, 64000, 69999], True),               # longer runs
])
def test_sequences_and_masks(moe, T, E, k, seg, masked):
    _say("seq", T, E, k, len(seg) - 1, masked)
    x, idx = _inputs(T, E, k, T * 3 + E)
    mask = (np.random.default_rng(T).random(T) > 0.3).astype(np.uint8) * 5 if masked else None
    add = np.random.default_rng(1).standard_normal((T, E)).astype(np.float32) * 1e-3
    dl = (2.0, -0.25)
    o = _run(moe, x, idx, 0.5, 0.1, seg, mask, dl, add)
    _check(o, x, idx, 0.5, 0.1, seg, mask, dl, add)
    # added in place, and without lse: the same bits
    o2 = _run(moe, x, idx, 0.5, 0.1, seg, mask, dl, add, alias=True, lse=False)
    for n in ("losses", "counts", "probs", "tokens", "grad"):
        np.testing.assert_array_equal(o2[n], o[n])


@pytest.mark.parametrize("T,E,k,seg,masked", [
    # one workgroup with everything (up to 32768 logits, 2048 tokens, two sequences), and the next size
    (2048, 16, 2, None, True), (2049, 15, 2, None, True), (256, 128, 8, None, False), (257, 128, 8, None, False),
    (32, 1024, 4, None, True), (33, 1024, 4, None, True), (31, 1021, 4, None, False),
    (255, 128, 4, [0, 255], True), (255, 128, 4, [3, 100, 250], True), (255, 128, 4, [3, 100, 250, 255], True),
    (300, 9, 3, [0, 0, 300], False), (300, 9, 3, [0, 300, 300], False), (300, 9, 3, [300, 300], False),
    (1, 2, 2, [0, 1, 1], False), (2, 1, 1, [0, 1, 2], True),
])
def test_few_tokens(moe, T, E, k, seg, masked):
    _say("few", T, E, k, seg, masked)
    x, idx = _inputs(T, E, k, T * 5 + E)
    x[T // 2, 0] = float("nan")
    mask = (np.random.default_rng(T).random(T) > 0.3).astype(np.uint8) if masked else None
    o = _run(moe, x, idx, 0.5, 0.1, seg, mask)
    _check(o, x, idx, 0.5, 0.1, seg, mask)
    counted = (mask is None or bool(mask[T // 2])) and (seg is None or seg[0] <= T // 2 < seg[-1])
    assert o["err"][0] == (moe.MOE_ERR_NONFINITE_LOGIT if counted else 0)


@pytest.mark.parametrize("T,E,k,S", [(300, 16, 2, 40), (1000, 100, 4, 64), (5000, 130, 2, 300), (40000, 32, 2, 5000),
                                     (700, 7, 3, 699), (64, 8, 2, 4100), (9000, 30, 1, 65)])
def test_many_sequences(moe, T, E, k, S):
    """Ragged sequences, some empty, tokens outside all of them; more of them than one search step and one ticket hold."""
    _say("many", T, E, k, S)
    g = np.random.default_rng(T + S)
    seg = np.sort(g.integers(T // 50, T + 1 - T // 60, S + 1)).astype(np.int32)
    x, idx = _inputs(T, E, k, T + S)
    mask = (g.random(T) > 0.2).astype(np.uint8)
    add = g.standard_normal((T, E)).astype(np.float32) * 1e-3
    dl = (1.5, -0.5)
    o = _run(moe, x, idx, 0.5, 0.1, list(seg), mask, dl, add)
    _check(o, x, idx, 0.5, 0.1, list(seg), mask, dl, add)
    o2 = _run(moe, x, idx, 0.5, 0.1, list(seg), mask, dl, add)
    for n in ("losses", "counts", "probs", "lse", "tokens", "grad"):
        np.testing.assert_array_equal(o2[n], o[n])


def test_nothing_counted(moe):
    _say("nothing")
    x, idx = _inputs(100, 8, 2, 1)
    add = np.ones((100, 8), np.float32)
    o = _run(moe, x, idx, 1.0, 1.0, mask=np.zeros(100), add=add)
    assert not o["losses"].any() and not o["counts"].any() and not o["probs"].any() and not o["tokens"].any()
    assert not o["lse"].any()
    np.testing.assert_array_equal(o["grad"], add)


def test_no_tokens(moe):
    _say("no tokens")
    x, idx = _inputs(0, 8, 2, 1)
    for seg in (None, [0, 0, 0]):
        o = _run(moe, x, idx, 1.0, 1.0, seg=seg)
        assert not o["losses"].any() and not o["counts"].any() and not o["probs"].any() and not o["tokens"].any()


@pytest.mark.parametrize("E", [8, 13, 128])
def test_values_that_are_not_finite(moe, E):
    _say("nonfinite", E)
    x, idx = _inputs(90, E, 2, E)
    x[3, 1] = float("-inf")
    x[5, 2] = float("nan")
    x[7, 0] = float("inf")
    x[9] = float("-inf")                                       # a row that leaves nothing
    x[11] = float("nan")
    x[13] = torch.finfo(torch.float32).min                     # a row of the type's lowest value
    x[15, 0] = torch.finfo(torch.float32).min
    o = _run(moe, x, idx, 0.3, 0.0)
    r = _check(o, x, idx, 0.3, 0.0)
    assert np.isfinite(o["grad"]).all() and o["err"][0] == moe.MOE_ERR_NONFINITE_LOGIT
    assert not r["p"][9].any() and not o["grad"][9].any() and o["lse"][9] == 0
    # the same values in rows that are masked: nothing is flagged
    mask = np.ones(90)
    mask[[3, 5, 7, 9, 11]] = 0
    o = _run(moe, x, idx, 0.3, 0.0, mask=mask)
    _check(o, x, idx, 0.3, 0.0, mask=mask)
    assert o["err"][0] == 0


def test_large_logits(moe):
    """p comes from differences to the maximum: its accuracy does not depend on the logits' size."""
    _say("large")
    x, idx = _inputs(200, 64, 2, 5)
    x = (x * 4).round() / 4 + 65536.0                          # exact in fp32
    o = _run(moe, x, idx, 0.1, 0.0)
    _check(o, x, idx, 0.1, 0.0)
    small = _run(moe, x - 65536.0, idx, 0.1, 0.0)
    np.testing.assert_array_equal(o["probs"], small["probs"])
    np.testing.assert_array_equal(o["grad"], small["grad"])


def test_indices_outside_count_for_no_expert(moe):
    _say("indices")
    x, idx = _inputs(150, 16, 3, 6)
    idx[4, 1], idx[70, 0], idx[149, 2] = -1, 16, 1 << 30
    o = _run(moe, x, idx, 0.1, 0.1)
    _check(o, x, idx, 0.1, 0.1)
    assert o["counts"].sum() == 150 * 3 - 3


def test_unaligned_logits(moe):
    _say("unaligned")
    T, E = 100, 128
    x, idx = _inputs(T, E, 2, 7)
    buf = torch.zeros(T * E + 1, device=DEV)
    buf[1:] = x.reshape(-1).to(DEV)
    xg = buf[1:].view(T, E)
    assert xg.data_ptr() % 16
    o = {n: torch.empty(s, dtype=t, device=DEV) for n, s, t in (
        ("losses", 2, torch.float32), ("counts", (1, E), torch.int32), ("probs", (1, E), torch.float32),
        ("lse", T, torch.float32), ("tokens", 2, torch.int32), ("grad", (T, E), torch.float32))}
    ws = torch.empty(moe.moe_balance_workspace_bytes(T, E), dtype=torch.uint8, device=DEV)
    moe.moe_balance_loss(xg, idx.to(torch.int32).to(DEV), 0.1, 0.1, o["losses"], o["counts"], o["probs"], o["lse"],
                         o["tokens"], ws)
    moe.moe_balance_loss_bwd(xg, o["counts"], o["tokens"], 0.1, 0.1, o["grad"])
    torch.cuda.synchronize()
    _check({n: v.cpu().numpy() for n, v in o.items()}, x, idx, 0.1, 0.1)


def test_unsorted_offsets_stay_inside(moe):
    """Offsets that are no partition: the values mean nothing, but every access stays in its tensor."""
    _say("unsorted")
    x, idx = _inputs(300, 16, 2, 8)
    for seg in ([0, 200, 100, 300], [300, 0], [-50, 1 << 30], [7, 3, 3, 250, 2]):
        _run(moe, x, idx, 0.1, 0.1, seg=seg)


def test_gradient_against_differences(moe):
    """The kernel's gradient against central differences of the plain loss, the counts held."""
    _say("differences")
    T, E, k = 40, 12, 2
    x, idx = _inputs(T, E, k, 11)
    seg, dl = [0, 13, 40], (1.0, 2.0)
    o = _run(moe, x, idx, 0.5, 0.2, seg=seg, dl=dl)
    x64 = x.numpy().astype(np.float64)
    eps = 1e-5
    rng = np.random.default_rng(3)
    for _ in range(40):
        t, e = rng.integers(T), rng.integers(E)
        hi, lo = x64.copy(), x64.copy()
        hi[t, e] += eps
        lo[t, e] -= eps
        d = sum(w * (a - b) for w, a, b in zip(dl, _plain.balance(hi, idx.numpy(), 0.5, 0.2, seg, counts=o["counts"])["losses"],
                                               _plain.balance(lo, idx.numpy(), 0.5, 0.2, seg, counts=o["counts"])["losses"])) / (2 * eps)
        # the difference's own error is eps^2 and 2^-53 / eps; the kernel's a few units of 2^-20
        assert abs(d - o["grad"][t, e]) <= 1e-5 * (abs(d) + 0.5 / T)


def test_router_step(moe):
    """Scores, route, losses and both gradients of one layer, as a training step runs them, against the oracle's
    gate gradient plus the plain balance gradient; captured and replayed with eager steps in between."""
    _say("step")
    import oracle
    from routing_grouped_gemm_amd.layer import MoELayer
    from tests._chain import np64
    T, d, E, f, k = 300, 256, 12, 128, 2
    seg = torch.tensor([0, 100, 290], dtype=torch.int32, device=DEV)
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(4)) > 0.2).to(torch.uint8).to(DEV)
    inp = moe_synth.make_inputs(T=T, d=d, E=E, f=f, k=k, seed=5)
    g = {n: inp[n].to(DEV) for n in ("x", "w13", "w2", "dout", "w_router")}
    for dtype in (moe.MOE_BF16, moe.MOE_MXFP4):
        lay = MoELayer(T, d, E, f, k, dtype)
        lay.set_weights(g["w13"], g["w2"])

        def step():
            logits = lay.router_scores(g["x"], g["w_router"])
            lay.forward(logits, g["x"])
            lay.balance_loss(logits, 0.01, 0.001, seg_off=seg, mask=mask)
            lay.gate_grad(g["dout"])
            lay.balance_loss_grad(logits, add_to=lay.dlogits)
        step()
        torch.cuda.synchronize()
        x, idx = lay.logits.cpu(), lay.topk_idx.cpu()
        _, gate = oracle.gate_grad(np64(g["dout"]), np64(lay.y_perm), lay.dst_row.cpu().numpy(), idx.numpy(),
                                   lay.topk_w.cpu().numpy(), E)
        lay.gate_grad(g["dout"])
        own = lay.dlogits.cpu().numpy().astype(np.float64)
        assert np.abs(own - gate).max() <= 1e-4 * np.abs(gate).max()
        lay.balance_loss_grad(lay.logits, add_to=lay.dlogits)
        torch.cuda.synchronize()
        o = dict(losses=lay.balance_losses, counts=lay.balance_counts, probs=lay.balance_probs,
                 tokens=lay.balance_tokens, grad=lay.dlogits)
        o = {n: v.cpu().numpy() for n, v in o.items()}
        o["lse"] = None
        _check(o, x, idx, 0.01, 0.001, seg.cpu().numpy(), mask.cpu().numpy(), add=own)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
        for rep in range(3):
            g["x"].copy_((torch.randn(T, d, generator=torch.Generator().manual_seed(rep)) * 0.02).to(torch.bfloat16))
            step()
            torch.cuda.synchronize()
            names = ("balance_losses", "balance_counts", "balance_probs", "balance_tokens", "dlogits", "out")
            ref = {n: getattr(lay, n).clone() for n in names}
            for n in names:
                getattr(lay, n).fill_(0)
            gr.replay()
            torch.cuda.synchronize()
            for n in names:
                assert torch.equal(getattr(lay, n), ref[n]), (rep, n)


def test_two_graphs_share_a_workspace(moe):
    """Two captured losses (two kernels each, one of them over sequences) with one workspace, replayed in turn."""
    _say("graphs")
    E, k = 24, 3
    ws = torch.empty(moe.moe_balance_workspace_bytes(9000, E, 4), dtype=torch.uint8, device=DEV)
    sets = []
    for T, seg in ((9000, None), (5003, [0, 64, 64, 3000, 5003])):
        S = 1 if seg is None else len(seg) - 1
        s = dict(x=torch.empty(T, E, device=DEV), idx=torch.empty(T, k, dtype=torch.int32, device=DEV),
                 losses=torch.empty(2, device=DEV), counts=torch.empty(S, E, dtype=torch.int32, device=DEV),
                 probs=torch.empty(S, E, device=DEV), lse=torch.empty(T, device=DEV),
                 tokens=torch.empty(S + 1, dtype=torch.int32, device=DEV), grad=torch.empty(T, E, device=DEV),
                 seg=None if seg is None else torch.tensor(seg, dtype=torch.int32, device=DEV))

        def step(s=s):
            moe.moe_balance_loss(s["x"], s["idx"], 0.1, 0.01, s["losses"], s["counts"], s["probs"], s["lse"],
                                 s["tokens"], ws, seg_off=s["seg"])
            moe.moe_balance_loss_bwd(s["x"], s["counts"], s["tokens"], 0.1, 0.01, s["grad"], seg_off=s["seg"])
        s["step"] = step
        x, idx = _inputs(T, E, k, T)
        s["x"].copy_(x), s["idx"].copy_(idx.to(torch.int32))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"]):
            step()
        sets.append(s)
    names = ("losses", "counts", "probs", "lse", "tokens", "grad")
    for rep in range(4):
        refs = []
        for s in sets:
            x, idx = _inputs(s["x"].shape[0], E, k, 100 + rep)
            s["x"].copy_(x), s["idx"].copy_(idx.to(torch.int32))
            s["step"]()
            torch.cuda.synchronize()
            refs.append({n: s[n].clone() for n in names})
            for n in names:
                s[n].zero_()
        ws.fill_(0xFF)
        for s in sets:
            s["graph"].replay()
        torch.cuda.synchronize()
        for s, r in zip(sets, refs):
            for n in names:
                assert torch.equal(s[n], r[n]), (rep, n)


def test_more_logits_than_32_bits_count(moe):
    """A block of tokens over and over: counts are exact multiples, every block's lse and gradient the first's bits,
    and the gradient the block's own over the repetitions (the counts' shares are the same quotients)."""
    _say("long")
    n, reps, E, k = 1000, 2200, 1024, 4
    x, idx = _inputs(n, E, k, 8)
    small = _run(moe, x, idx, 0.5, 0.1)
    xg, ig = x.to(DEV).repeat(reps, 1), idx.to(torch.int32).to(DEV).repeat(reps, 1)
    T = n * reps
    assert T * E > 1 << 31
    losses, counts = torch.empty(2, device=DEV), torch.empty(1, E, dtype=torch.int32, device=DEV)
    probs, lse = torch.empty(1, E, device=DEV), torch.empty(T, device=DEV)
    tokens = torch.empty(2, dtype=torch.int32, device=DEV)
    ws = torch.empty(moe.moe_balance_workspace_bytes(T, E, 1), dtype=torch.uint8, device=DEV)
    moe.moe_balance_loss(xg, ig, 0.5, 0.1, losses, counts, probs, lse, tokens, ws)
    grad = torch.full((T, E), 9.0, device=DEV)
    moe.moe_balance_loss_bwd(xg, counts, tokens, 0.5, 0.1, grad)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(counts.cpu().numpy(), small["counts"] * reps)
    assert tokens.tolist() == [T, T]
    first, last = grad[:n], grad[T - n:]
    assert torch.equal(first, last) and torch.equal(grad[T // 2:T // 2 + n], first)
    assert torch.equal(lse.view(reps, n), lse[:n].expand(reps, n))
    # f is counts / sum of counts, here both `reps` times as large (below 2^24: exact), so it is the same
    # quotient; k_b, k_z and the three products after them are rounded anew: 2^-21 of each term's size
    p = torch.softmax(x.double(), 1)
    f = torch.as_tensor(small["counts"]).double() / (n * k)
    mag = p * (0.5 * E / n * (f + (p * f).sum(1, keepdim=True)) + 0.2 / n * torch.as_tensor(small["lse"]).double().abs()[:, None])
    err = (first.cpu().double() * reps - torch.as_tensor(small["grad"]).double()).abs()
    assert bool((err <= 2.0 ** -21 * mag + 2.0 ** -100).all())
    # the sums: at most T additions of rounded terms in any order
    assert float((probs.cpu() - torch.as_tensor(small["probs"])).abs().max()) <= T * 2.0 ** -24 * float(small["probs"].max())
