"""Cases that time the MXFP4 expert products and the router's balance loss.

Three operators, each with its plain form (elementary torch operations in 32
bits) and its definition in 64 bits (``exact``):

  quantise  MXFP4 and back: bf16 rows -> E2M1 codes, two to a byte, with one
            power-of-two scale (E8M0) per 32 elements -> the bf16 values those
            stand for.
  product   the experts' feed-forward over weights kept in MXFP4: each token
            row is quantised into the rows of its k experts, then per expert
            g | u = x W13^T, h = silu(g) u, y = h W2^T, every operand in MXFP4
            and every sum in fp32.
  balance   the router's balance loss and z loss with the per-expert counts,
            over packed sequences, and their gradient to the router logits.

``own`` selects the framework's kernels instead of the plain form.
"""
import math

import torch

own = False

DEV = "cuda"


def _package():
    import routing_grouped_gemm_amd as m
    return m


def listed():
    return [
        # the rows of one decode batch: a few microseconds, launch latency counts
        dict(name="quantise a decode batch", op="quantise", rows=64, K=4096),
        # ragged activations: an odd row count, a width that is no power of two
        dict(name="quantise ragged rows", op="quantise", rows=5003, K=1152),
        # the gate/up weights of one expert-parallel shard, after an optimizer step or a load
        dict(name="quantise a weight shard", op="quantise", rows=49152, K=4096),
        # one token answered: four experts' weights are read for four rows
        dict(name="product of one token", op="product", T=1, E=128, d=4096, f=1536, k=4, routing="uniform", save=False),
        # a serving batch: every expert has a row or two, all weights are read
        dict(name="product of a decode batch", op="product", T=67, E=128, d=4096, f=1536, k=4, routing="uniform", save=False),
        # a prompt chunk over few experts, ragged groups, sizes that end inside tiles
        dict(name="product of a prompt chunk", op="product", T=1000, E=8, d=2048, f=1152, k=2, routing="zipf", save=False),
        # one expert-parallel shard's rows, skewed over its experts, activations saved
        dict(name="product of a skewed shard", op="product", T=32768, E=16, d=4096, f=1536, k=1, routing="zipf", save=True),
        # a whole training batch of the 128-expert layer, activations saved for the backward
        dict(name="product of a training batch", op="product", T=16384, E=128, d=4096, f=1536, k=4, routing="uniform", save=True),
        # the smallest router: latency only
        dict(name="balance of a small batch", op="balance", T=256, E=8, k=2, S=1, mask=False, grad=True),
        # losses and counts alone, as a run that only watches its router takes them
        dict(name="balance watched", op="balance", T=16384, E=128, k=4, S=1, mask=False, grad=False),
        # a training step's router: packed sequences with padding, gradient added to the gate gradient
        dict(name="balance of packed sequences", op="balance", T=16391, E=128, k=4, S=23, mask=True, grad=True),
        # a very large batch of routers
        dict(name="balance of a large batch", op="balance", T=1 << 20, E=128, k=4, S=1, mask=False, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantise", "product", "product", "balance"))
    if op == "quantise":
        K = 128 * _log(rng, 1, 64)
        return dict(op=op, rows=_log(rng, 1, min(131072, (1 << 27) // K)), K=K)
    if op == "product":
        E = _log(rng, 1, 128)
        d = 128 * _log(rng, 1, 32)
        f = 128 * _log(rng, 1, 12)
        k = rng.randint(1, min(E, 8))
        return dict(op=op, T=_log(rng, 1, 8192), E=E, d=d, f=f, k=k, routing=rng.choice(("uniform", "zipf")),
                    save=rng.random() < 0.5)
    E = _log(rng, 2, 1024)
    T = _log(rng, 1, min(1 << 19, (1 << 26) // E))
    return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 8)), S=_log(rng, 1, min(T, 64)), mask=rng.random() < 0.5,
                grad=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1009 + salt)
    return g


def _logits(T, E, routing, g):
    if routing == "zipf":
        u = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-12, 1.0 - 1e-7)
        p = torch.arange(1, E + 1, device=DEV, dtype=torch.float32).pow(-1.2)
        return torch.log(p / p.sum()) - torch.log(-torch.log(u))
    return torch.randn(T, E, generator=g, device=DEV)


def _codes_of(w):
    """MXFP4 codes [rows, K/2] and scales [rows, K/32] of fp32 w (weights as a program keeps them)."""
    rows, K = w.shape
    b = w.view(rows, K // 32, 32)
    m, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(m > 0, (e - 3 + (m > 0.75)).clamp(-127, 127), torch.full_like(e, -127))
    q = torch.ldexp(b, -e[..., None]).reshape(rows, K)
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code |= (torch.signbit(q).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def prepare(case, seed):
    c = dict(case)
    s = dict(case=c)
    if c["op"] == "quantise":
        g = _gen(seed, 1)
        x = torch.randn(c["rows"], c["K"], generator=g, device=DEV) * 0.02
        x[:, ::97] *= 16.0                                 # outlier channels
        s["x"] = x.to(torch.bfloat16)
        if own:
            s["codes"] = torch.empty(c["rows"], c["K"] // 2, dtype=torch.uint8, device=DEV)
            s["scales"] = torch.empty(c["rows"], c["K"] // 32, dtype=torch.uint8, device=DEV)
            s["back"] = torch.empty_like(s["x"])
        return s
    if c["op"] == "product":
        T, E, d, f, k = c["T"], c["E"], c["d"], c["f"], c["k"]
        g = _gen(seed, 2)
        x = torch.randn(T, d, generator=g, device=DEV)     # the output of a norm: unit variance
        x[:, ::97] *= 8.0
        s["x"] = x.to(torch.bfloat16)
        idx = torch.topk(_logits(T, E, c["routing"], g), k, dim=1).indices.reshape(-1)
        order = torch.argsort(idx, stable=True)
        s["src_slot"] = order.to(torch.int32)
        dst = torch.empty_like(order)
        dst[order] = torch.arange(T * k, device=DEV)
        s["dst_row"] = dst.to(torch.int32)
        counts = torch.bincount(idx, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["sizes"] = counts.tolist()                       # the plain form's loop over the experts
        w13 = torch.empty(E, 2 * f, d // 2, dtype=torch.uint8, device=DEV)
        w13s = torch.empty(E, 2 * f, d // 32, dtype=torch.uint8, device=DEV)
        w2 = torch.empty(E, d, f // 2, dtype=torch.uint8, device=DEV)
        w2s = torch.empty(E, d, f // 32, dtype=torch.uint8, device=DEV)
        for e in range(E):
            w13[e], w13s[e] = _codes_of(torch.randn(2 * f, d, generator=g, device=DEV) * 0.02)
            w2[e], w2s[e] = _codes_of(torch.randn(d, f, generator=g, device=DEV) * 0.02)
        s.update(w13=w13, w13s=w13s, w2=w2, w2s=w2s)
        if own:
            m, R = _package(), T * k
            bf = dict(dtype=torch.bfloat16, device=DEV)
            s["xq"] = torch.empty(R, d // 2, dtype=torch.uint8, device=DEV)
            s["xs"] = torch.empty(R, d // 32, dtype=torch.uint8, device=DEV)
            s["gu"] = torch.empty(R, 2 * f, **bf) if c["save"] else None
            s["h"] = torch.empty(R, f, **bf) if c["save"] else None
            s["y"] = torch.empty(R, d, **bf)
            s["ws"] = torch.empty(m.moe_gemm_workspace_bytes(m.MOE_MXFP4, E, R, d, f), dtype=torch.uint8, device=DEV)
        return s
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    g = _gen(seed, 3)
    s["logits"] = _logits(T, E, "zipf" if E > 8 else "uniform", g) * 1.5
    s["topk_idx"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
    # S packed sequences; what follows the last one belongs to none
    cut = torch.sort(torch.randint(0, T + 1, (max(S - 1, 0),), generator=g, device=DEV)).values
    end = T if S == 1 else T - T // 50
    s["seg_off"] = torch.cat([cut.new_zeros(1), cut.clamp(max=end), cut.new_full((1,), end)]).to(torch.int32)
    s["cuts"] = s["seg_off"].tolist()                      # the plain form's loop over the sequences
    s["mask"] = (torch.rand(T, generator=g, device=DEV) > 0.1).to(torch.uint8) if c["mask"] else None
    s["before"] = torch.randn(T, E, generator=g, device=DEV) * 1e-3 if c["grad"] else None   # the gate gradient
    s["dlosses"] = torch.tensor([1.0, 1.0], device=DEV)
    if own:
        m = _package()
        s["losses"] = torch.empty(2, device=DEV)
        s["counts"] = torch.empty(S, E, dtype=torch.int32, device=DEV)
        s["probs"] = torch.empty(S, E, device=DEV)
        s["lse"] = torch.empty(T, device=DEV)
        s["tokens"] = torch.empty(S + 1, dtype=torch.int32, device=DEV)
        s["dlogits"] = torch.empty(T, E, device=DEV) if c["grad"] else None
        s["ws"] = torch.empty(m.moe_balance_workspace_bytes(T, E, S), dtype=torch.uint8, device=DEV)
    return s


BALANCE, Z = 0.01, 0.001           # loss coefficients


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    m, c = _package(), s["case"]
    if c["op"] == "quantise":
        m.moe_quantize_mxfp4(s["x"], s["codes"], s["scales"])
        m.moe_dequantize_mxfp4(s["codes"], s["scales"], s["back"])
        return s["back"]
    if c["op"] == "product":
        m.moe_permute(m.MOE_MXFP4, s["x"], c["k"], s["dst_row"], s["xq"], x_perm_scales=s["xs"])
        m.moe_grouped_gemm_fwd(m.MOE_MXFP4, s["xq"], s["w13"], s["w2"], s["offsets"], 0, s["gu"], s["h"], s["y"],
                               x_perm_scales=s["xs"], w13_scales=s["w13s"], w2_scales=s["w2s"], ws=s["ws"])
        return (s["gu"], s["h"], s["y"]) if c["save"] else s["y"]
    seg = s["seg_off"] if c["S"] > 1 else None
    m.moe_balance_loss(s["logits"], s["topk_idx"], BALANCE, Z, s["losses"], s["counts"], s["probs"], s["lse"],
                       s["tokens"], s["ws"], seg_off=seg, mask=s["mask"])
    out = [s["losses"], s["counts"], s["probs"], s["lse"], s["tokens"]]
    if c["grad"]:
        m.moe_balance_loss_bwd(s["logits"], s["counts"], s["tokens"], BALANCE, Z, s["dlogits"],
                               dlosses=s["dlosses"], add=s["before"], seg_off=seg, mask=s["mask"])
        out.append(s["dlogits"])
    return out


def _round_mx(v):
    """The MXFP4 values of v [rows, K], in v's type."""
    rows, K = v.shape
    b = v.reshape(rows, K // 32, 32)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.where(m > 0, (e - 3 + (m > 0.75)).clamp(-127, 127), torch.full_like(e, -127))
    q = torch.ldexp(b, -e)
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(v.dtype)
    return torch.ldexp(torch.round(q / step) * step, e).reshape(rows, K)


def _values(codes, scales):
    """The values of MXFP4 codes [rows, K/2] and scales [rows, K/32]."""
    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float32, device=codes.device)
    one = torch.cat([one, -one])
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack([one[byte & 15], one[byte >> 4]], 1)
    v = pair[codes.long()].reshape(codes.shape[0], -1, 32)
    return torch.ldexp(v, (scales.to(torch.int32) - 127)[..., None]).reshape(codes.shape[0], -1)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "quantise":
        return _round_mx(s["x"].float()).to(torch.bfloat16)
    if c["op"] == "product":
        k, f = c["k"], c["f"]
        xp = _round_mx(s["x"].float())[torch.div(s["src_slot"], k, rounding_mode="floor").long()]
        gus, hs, ys, at = [], [], [], 0
        for e, n in enumerate(s["sizes"]):
            if not n:
                continue
            gu = xp[at:at + n] @ _values(s["w13"][e], s["w13s"][e]).t()
            g, u = gu[:, :f], gu[:, f:]
            h = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
            ys.append((_round_mx(h.float()) @ _values(s["w2"][e], s["w2s"][e]).t()).to(torch.bfloat16))
            if c["save"]:
                gus.append(gu.to(torch.bfloat16))
                hs.append(h)
            at += n
        y = torch.cat(ys)
        return (torch.cat(gus), torch.cat(hs), y) if c["save"] else y
    return _balance_plain(s)


def _balance_plain(s):
    c = s["case"]
    T, E, S = c["T"], c["E"], c["S"]
    x = s["logits"]
    off = s["seg_off"].long()
    t = torch.arange(T, device=x.device)
    seg = torch.searchsorted(off, t, right=True) - 1
    ok = (seg >= 0) & (seg < S)
    if s["mask"] is not None:
        ok = ok & (s["mask"] != 0)
    seg = seg.clamp(0, S - 1)
    top = x.amax(1, keepdim=True)
    ex = torch.exp(x - top)
    den = ex.sum(1, keepdim=True)
    p = ex / den
    lse = torch.where(ok, (top + torch.log(den))[:, 0], 0.0)
    # sums over the tokens in 64 bits
    pm = p * ok[:, None]
    parts = list(zip(s["cuts"][:-1], s["cuts"][1:]))
    n = torch.stack([ok[a:b].sum() for a, b in parts])
    total = n.sum()
    probs = (torch.stack([pm[a:b].sum(0, dtype=torch.float64) for a, b in parts]) / n.clamp(min=1)[:, None]).float()
    counts = torch.zeros(S * E, dtype=torch.int32, device=x.device)
    counts.scatter_add_(0, (seg[:, None] * E + s["topk_idx"]).reshape(-1),
                        ok[:, None].expand(T, c["k"]).reshape(-1).to(torch.int32))
    counts = counts.view(S, E)
    share = counts / counts.sum(1, keepdim=True).clamp(min=1)
    N = total.clamp(min=1)
    balance = BALANCE * E * ((n / N)[:, None].double() * share.double() * probs.double()).sum()
    z = Z * lse.double().square().sum() / N
    out = [torch.stack([balance, z]).float(), counts, probs, lse, torch.cat([n, total[None]]).to(torch.int32)]
    if c["grad"]:
        f = share[seg]
        dot = (f * p).sum(1, keepdim=True)
        gr = s["dlosses"][0] * BALANCE * E / N * p * (f - dot) + s["dlosses"][1] * 2 * Z / N * lse[:, None] * p
        out.append(s["before"] + torch.where(ok[:, None], gr, 0.0))
    return out


# ------------------------------------------------------------------ bytes and operations
def work(case):
    c = case
    if c["op"] == "quantise":
        n = c["rows"] * c["K"]
        return dict(bytes=2 * n * (2 + 0.5 + 1 / 32), flops=4 * n)
    if c["op"] == "product":
        T, E, d, f, R = c["T"], c["E"], c["d"], c["f"], c["T"] * c["k"]
        mx = 0.5 + 1 / 32
        hit = E * (1 - (1 - c["k"] / E) ** T)              # experts with a row, for even routing
        b = 2 * T * d + 2 * R * d * mx + hit * 3 * d * f * mx + 2 * R * d + 4 * R + 4 * E
        if c["save"]:
            b += 2 * R * 3 * f
        return dict(bytes=b, flops=6 * R * d * f)
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    b = 4 * T * E + 4 * T * k + 4 * T + 8 * S * E + (T if c["mask"] else 0)
    # the gradient reads the logits again, since the counts are known after all tokens only, and adds to what is there
    return dict(bytes=b + ((12 * T * E + 4 * T) if c["grad"] else 0), flops=(20 if c["grad"] else 10) * T * E)


# ------------------------------------------------------------------ the definition, in 64 bits
def _nearest(v):
    """MXFP4 of v [rows, K] in 64 bits, from the definition: the smallest power of two that holds the block's
    maximum within 6, and the nearest of the representable values, of two equally near the one with an even code."""
    rows, K = v.shape
    b = v.double().view(-1, 32)
    top = b.abs().amax(1, keepdim=True)
    e = torch.ceil(torch.log2(top / 6)).clamp(-127, 127)
    e = torch.where(top > 6 * torch.exp2(e), e + 1, e)
    e = torch.where((top <= 6 * torch.exp2(e - 1)) & (e > -127), e - 1, e)
    scale = torch.exp2(torch.where(top > 0, e, torch.full_like(e, -127.0)))
    q = b / scale
    have = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    mid = (have[1:] + have[:-1]) / 2
    below, above = torch.searchsorted(mid, q.abs()), torch.searchsorted(mid, q.abs(), right=True)
    code = torch.where(below % 2 == 0, below, above)       # they differ only on a midpoint
    return (torch.sign(q) * have[code] * scale).view(rows, K)


def _decoded(codes, scales):
    """MXFP4 codes in 64 bits: sign, two exponent bits, one fraction bit, no fraction's leading one at exponent 0."""
    nib = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1)
    ex, fr = ((nib >> 1) & 3).double(), (nib & 1).double()
    mag = torch.where(ex > 0, (1 + fr / 2) * torch.exp2(ex - 1), fr / 2)
    scale = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
    return torch.where(nib > 7, -mag, mag) * scale


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quantise":
        return _nearest(s["x"])
    if c["op"] == "product":
        k, f = c["k"], c["f"]
        xq = _nearest(s["x"])
        gus, hs, ys, at = [], [], [], 0
        for e, n in enumerate(s["sizes"]):
            x = xq[s["src_slot"][at:at + n].long() // k]
            at += n
            if not n:
                continue
            gu = torch.mm(x, _decoded(s["w13"][e], s["w13s"][e]).t().contiguous())
            h = torch.sigmoid(gu[:, :f]) * gu[:, :f] * gu[:, f:]
            ys.append(torch.mm(_nearest(h.to(torch.bfloat16)),
                               _decoded(s["w2"][e], s["w2s"][e]).t().contiguous()))
            if c["save"]:
                gus.append(gu)
                hs.append(h)
        return (torch.cat(gus), torch.cat(hs), torch.cat(ys)) if c["save"] else torch.cat(ys)
    T, E, S = c["T"], c["E"], c["S"]
    x = s["logits"].double().requires_grad_(c["grad"])
    off = s["cuts"]
    ok = torch.ones(T, dtype=torch.bool, device=x.device) if s["mask"] is None else s["mask"].bool()
    inside = torch.zeros(T, dtype=torch.bool, device=x.device)
    inside[off[0]:off[-1]] = True
    ok = ok & inside
    N = max(int(ok.sum()), 1)
    balance, probs, counts, tokens = x.new_zeros(()), [], [], []
    for a, b in zip(off[:-1], off[1:]):
        mine = ok[a:b]
        n = int(mine.sum())
        p = torch.softmax(x[a:b][mine], 1).sum(0) / max(n, 1)
        hit = torch.bincount(s["topk_idx"][a:b][mine].reshape(-1).long(), minlength=E)
        balance = balance + E * n / N * (hit / max(n * c["k"], 1) * p).sum()
        probs.append(p.detach())
        counts.append(hit.to(torch.int32))
        tokens.append(n)
    lse = torch.where(ok, torch.logsumexp(x, 1), 0.0)
    losses = torch.stack([BALANCE * balance, Z * (lse * lse).sum() / N])
    out = [losses.detach(), torch.stack(counts), torch.stack(probs), lse.detach(),
           torch.tensor(tokens + [sum(tokens)], dtype=torch.int32, device=x.device)]
    if c["grad"]:
        (gr,) = torch.autograd.grad((losses * s["dlosses"]).sum(), x)
        out.append(s["before"].double() + gr)
    return out
