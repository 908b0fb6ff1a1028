"""The balance loss's long sums against 64-bit ones, from thousands of tokens to runs of thousands per workgroup and
logits past the last-level cache (where accesses stream).

Tolerances count the additions a term passes through, not the number of terms: a sum of positive terms is off by
at most 2^-24 of itself for each of them.  A workgroup's run of tokens goes round NT / LPT lane groups, each lane
adding its tokens one after another; the groups of a wave and the eight waves follow, then a lane of the reduction
adds every 64th run's sums, and 64 lanes.  A softmax value is off by a relative (R + 8) 2^-22, R the logits' span."""
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _say(*a):
    print("[gpu-balance-sums]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def moe():
    import routing_grouped_gemm_amd as m
    assert torch.cuda.is_available()
    m.load()
    return m


def _additions(T, E, S):
    lanes = 1
    while lanes * (4 if E <= 64 else 8 if E <= 128 else 16) < E:
        lanes *= 2
    run = max(64, (-(-T // 512) + 15) // 16 * 16)          # fewer where sequences are short: more runs, shorter chains
    short = min(run, max((T // S + 7) // 8 * 8, 8))
    return run * lanes // 512 + 1 + 6 + 8 + (T // short + S) // 64 + 1 + 6


def _loss(moe, x, idx, cb, cz, seg, mask, lse=True):
    T, E = x.shape
    S = 1 if seg is None else seg.numel() - 1
    o = dict(losses=torch.empty(2, device=DEV), counts=torch.empty(S, E, dtype=torch.int32, device=DEV),
             probs=torch.empty(S, E, device=DEV), lse=torch.empty(T, device=DEV) if lse else None,
             tokens=torch.empty(S + 1, dtype=torch.int32, device=DEV))
    ws = torch.full((moe.moe_balance_workspace_bytes(T, E, S),), 0xFF, dtype=torch.uint8, device=DEV)
    moe.moe_balance_loss(x, idx, cb, cz, o["losses"], o["counts"], o["probs"], o["lse"], o["tokens"], ws, seg_off=seg,
                         mask=mask)
    return o


CB, CZ = 0.5, 0.1


@pytest.mark.parametrize("T,E,k,S,masked", [
    (66000, 16, 2, 1, False), (70000, 8, 1, 4, True), (16391, 128, 4, 23, True), (40000, 130, 2, 3, False),
    (30000, 1024, 8, 1, True), (200000, 32, 2, 2000, False),
    # streamed: 256 MB of logits and more
    (524288, 128, 4, 1, False), (525291, 128, 8, 5, True), (300000, 256, 2, 700, True), (4200000, 16, 1, 1, False),
    (140000, 500, 3, 2, False),
])
def test_sums(moe, T, E, k, S, masked):
    _say(T, E, k, S, masked)
    g = torch.Generator(device=DEV).manual_seed(T + E)
    x = torch.randn(T, E, generator=g, device=DEV) * 1.5
    idx = torch.topk(x, k, dim=1).indices.to(torch.int32)
    mask = (torch.rand(T, generator=g, device=DEV) > 0.2).to(torch.uint8) if masked else None
    seg = None
    if S > 1:
        cut = torch.sort(torch.randint(T // 50, T - T // 60, (S + 1,), generator=g, device=DEV)).values
        seg = cut.to(torch.int32)
    o = _loss(moe, x, idx, CB, CZ, seg, mask)
    add = torch.randn(T, E, generator=g, device=DEV) * 1e-3
    grad = torch.full((T, E), 9.0, device=DEV)
    dl = torch.tensor([1.5, -0.5], device=DEV)
    moe.moe_balance_loss_bwd(x, o["counts"], o["tokens"], CB, CZ, grad, dlosses=dl, add=add, seg_off=seg, mask=mask)
    torch.cuda.synchronize()

    # 64 bits, in blocks of tokens
    off = torch.tensor([0, T], device=DEV) if seg is None else seg.long()
    s_of = torch.searchsorted(off, torch.arange(T, device=DEV), right=True) - 1
    on = (s_of >= 0) & (s_of < S)
    if mask is not None:
        on &= mask != 0
    s_of = s_of.clamp(0, S - 1)
    n = torch.zeros(S, dtype=torch.int64, device=DEV).index_add_(0, s_of, on.long())
    N = int(n.sum())
    assert o["tokens"].tolist() == n.tolist() + [N]
    counts = torch.zeros(S * E, dtype=torch.int64, device=DEV)
    counts.index_add_(0, (s_of[:, None] * E + idx).reshape(-1), on[:, None].expand(T, k).reshape(-1).long())
    counts = counts.view(S, E)
    assert torch.equal(o["counts"].long(), counts)
    f = counts.double() / counts.sum(1, keepdim=True).clamp(min=1)
    sums = torch.zeros(S, E, dtype=torch.float64, device=DEV)
    z, ztol, worst, step = 0.0, 0.0, [], max(1, (1 << 25) // E)
    span = float((x.amax(1) - x.amin(1)).max())
    rel = (span + 8) * 2.0 ** -22
    kb, kz = float(dl[0]) * CB * E / N, float(dl[1]) * CZ * 2 / N
    for a in range(0, T, step):
        sl = slice(a, min(T, a + step))
        v = x[sl].double()
        top = v.amax(1, keepdim=True)
        e = torch.exp(v - top)
        den = e.sum(1, keepdim=True)
        p, lse = e / den, (top + torch.log(den))[:, 0]
        m = on[sl].double()
        for b in range(int(s_of[sl].min()), int(s_of[sl].max()) + 1) if S <= 30 else ():
            sums[b] += (p * (m * (s_of[sl] == b))[:, None]).sum(0)
        if S > 30:
            sums.index_add_(0, s_of[sl], p * m[:, None])
        ltol = (lse.abs() + v.abs().amax(1)) * 2.0 ** -23 + rel
        assert bool(((o["lse"][sl].double() - lse * m).abs() <= ltol * m).all())
        z += float((lse * lse * m).sum())
        ztol += float(((2 * lse.abs() * ltol + ltol ** 2) * m).sum())
        ft = f[s_of[sl]]
        dot = (ft * p).sum(1, keepdim=True)
        want = add[sl].double() + p * (kb * (ft - dot) + kz * lse[:, None]) * m[:, None]
        mag = p * (abs(kb) * (ft + dot) + abs(kz) * lse.abs()[:, None])
        tol = mag * 2 * (rel + 2.0 ** -20) + p * abs(kz) * ltol[:, None] + 2.0 ** -23 * want.abs() + 2.0 ** -120
        worst.append(bool(((grad[sl].double() - want).abs() <= tol).all()))
    assert all(worst)
    adds = _additions(T, E, S) * 2.0 ** -24
    probs = sums / n.clamp(min=1)[:, None]
    err = (o["probs"].double() - probs).abs()
    assert bool((err <= probs * (rel + adds + 2.0 ** -22) + 2.0 ** -120).all()), float((err / probs.clamp(min=1e-30)).max())
    balance = CB * E / N * float((n[:, None] * f * probs).sum())
    # over the experts' groups and the sequences 40 and S / 64 more additions at most, and five roundings
    more = (45 + S / 64) * 2.0 ** -24
    got = o["losses"].tolist()
    assert abs(got[0] - balance) <= balance * (rel + adds + more)
    assert abs(got[1] - CZ * z / N) <= CZ / N * (z * (adds + more) + ztol)


def test_more_logits_than_32_bits_count_in_the_sums(moe):
    """A block of tokens 2200 times over: mean probabilities and losses are the block's."""
    _say("long")
    n, reps, E, k = 1000, 2200, 1024, 4
    g = torch.Generator().manual_seed(8)
    x = torch.randn(n, E, generator=g) * 1.5
    idx = torch.topk(x, k, dim=1).indices
    T = n * reps
    o = _loss(moe, x.to(DEV).repeat(reps, 1), idx.to(torch.int32).to(DEV).repeat(reps, 1), CB, CZ, None, None, lse=False)
    torch.cuda.synchronize()
    v = x.numpy().astype(np.float64)
    top = v.max(1, keepdims=True)
    e = np.exp(v - top)
    p, lse = e / e.sum(1, keepdims=True), (top + np.log(e.sum(1, keepdims=True)))[:, 0]
    probs = p.mean(0)
    counts = np.bincount(idx.numpy().reshape(-1), minlength=E)
    rel = (float((v.max(1) - v.min(1)).max()) + 8) * 2.0 ** -22
    adds = _additions(T, E, 1) * 2.0 ** -24
    assert adds < 4e-5
    np.testing.assert_array_equal(o["counts"].cpu().numpy()[0], counts * reps)
    assert np.all(np.abs(o["probs"].cpu().numpy()[0] - probs) <= probs * (rel + adds + 2.0 ** -22))
    balance = CB * E * (counts / counts.sum() * probs).sum()
    ltol = (np.abs(lse) + np.abs(v).max(1)) * 2.0 ** -23 + rel
    got = o["losses"].tolist()
    assert abs(got[0] - balance) <= balance * (rel + adds + 45 * 2.0 ** -24)
    assert abs(got[1] - CZ * (lse ** 2).mean()) <= CZ * ((lse ** 2).mean() * (adds + 45 * 2.0 ** -24)
                                                         + (2 * np.abs(lse) * ltol + ltol ** 2).mean())
