"""Cases that time the gated block with its dropout and the 4-bit integer experts.

Four operators, each with its plain form (elementary torch operations in 32
bits) and its definition in 64 bits (``exact``):

  dropout   dropout from a counter-based generator, its mask made anew wherever
            it is needed: of plain rows with a residual, and of the experts'
            combined outputs together with its backward.
  gated     the experts' gated block over dispatched rows, g | u = x W13^T,
            h = dropout(act(min(g, L)) clamp(u, -L, L)), y = h W2^T, for the gates
            silu, gelu (erf and tanh) and relu; forward, and backward from what
            the forward saved.
  quantise  bf16 rows -> 4-bit integers with a bf16 scale (and a zero point) for
            each group along the row, and the bf16 values those stand for.
  answer    the layer's feed-forward for few tokens, from token rows to combined
            outputs, over experts kept in such 4-bit integers.

``own`` selects the framework's kernels instead of the plain form.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
ACTS = ("silu", "gelu_tanh", "gelu", "relu")


def _package():
    import routing_grouped_gemm_amd as m
    return m


def listed():
    return [
        # the smallest training batch's residual stream: launch latency counts
        dict(name="dropout of a small batch", op="dropout", T=256, d=128, p=0.1, dtype="bf16", residual=True),
        # fp32 rows, an odd number of them, a width that is no power of two
        dict(name="dropout of ragged rows", op="dropout", T=5003, d=1152, p=0.25, dtype="f32", residual=False),
        # a training step of the 128-expert layer: outputs combined, dropped and added to the residual, and
        # the upstream gradient under the same mask
        dict(name="combine with dropout", op="combine", T=16384, d=4096, k=4, p=0.1, dtype="bf16"),
        # the smallest layer, fp32
        dict(name="gated block of a small batch", op="gated", part="forward", R=512, E=8, d=128, f=256, act="gelu",
             limit=0.0, p=0.1, dtype="f32", routing="uniform"),
        # ragged groups of a small training batch, sizes that end inside tiles, clamped gates
        dict(name="gated backward of ragged rows", op="gated", part="backward", R=2003, E=8, d=2048, f=1152,
             act="silu", limit=2.0, p=0.1, dtype="bf16", routing="zipf"),
        # a training batch of the eight-expert layer
        dict(name="gated block of a training batch", op="gated", part="forward", R=32768, E=8, d=2048, f=1024,
             act="relu", limit=0.0, p=0.1, dtype="bf16", routing="uniform"),
        # one expert-parallel shard's backward
        dict(name="gated backward of a shard", op="gated", part="backward", R=32768, E=16, d=4096, f=1536,
             act="gelu_tanh", limit=0.0, p=0.1, dtype="bf16", routing="uniform"),
        # ragged rows in small groups, with zero points
        dict(name="quantise ragged rows to int4", op="quantise", rows=5003, K=1152, group=32, zeros=True),
        # the gate/up weights of one expert-parallel shard, once when a model is loaded
        dict(name="quantise a weight shard to int4", op="quantise", rows=49152, K=4096, group=128, zeros=False),
        # one token answered: four experts' weights are read for four rows
        dict(name="answer one token", op="answer", T=1, E=128, d=4096, f=1536, k=4, group=128, zeros=False,
             act="silu", limit=0.0, routing="uniform"),
        # a serving batch: every expert has a row or two, all weights are read
        dict(name="answer a decode batch", op="answer", T=67, E=128, d=4096, f=1536, k=4, group=128, zeros=True,
             act="silu", limit=0.0, routing="uniform"),
        # a prompt chunk over few experts, ragged groups
        dict(name="answer a prompt chunk", op="answer", T=1000, E=8, d=2048, f=1152, k=2, group=64, zeros=True,
             act="gelu_tanh", limit=0.0, routing="zipf"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("dropout", "combine", "gated", "gated", "quantise", "answer", "answer"))
    p = rng.choice((0.0, 0.05, 0.1, 0.3, 0.5))
    if op in ("dropout", "combine"):
        d = 8 * _log(rng, 1, 512)
        k = rng.randint(1, 8)
        T = _log(rng, 1, min(65536, (1 << 26) // d // (k if op == "combine" else 1)))
        c = dict(op=op, T=T, d=d, p=p, dtype=rng.choice(("bf16", "bf16", "f32")))
        c.update(dict(residual=rng.random() < 0.5) if op == "dropout" else dict(k=k))
        return c
    act, limit = rng.choice(ACTS), rng.choice((0.0, 0.0, 1.5, 7.0))
    routing = rng.choice(("uniform", "zipf"))
    if op == "gated":
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        d, f = 8 * _log(rng, 1, 512), 8 * _log(rng, 1, 192)
        R = _log(rng, 1, 32768)
        if dtype == "f32":
            d, f, R = 8 * _log(rng, 1, 64), 8 * _log(rng, 1, 64), _log(rng, 1, 4096)
        return dict(op=op, part=rng.choice(("forward", "backward")), R=R, E=_log(rng, 1, 16), d=d, f=f, act=act,
                    limit=limit, p=p, dtype=dtype, routing=routing)
    group, zeros = rng.choice((32, 64, 128)), rng.random() < 0.5
    if op == "quantise":
        K = group * _log(rng, 1, 8192 // group)
        return dict(op=op, rows=_log(rng, 1, min(131072, (1 << 27) // K)), K=K, group=group, zeros=zeros)
    E = _log(rng, 1, 128)
    return dict(op=op, T=_log(rng, 1, 1024), E=E, d=group * _log(rng, 1, 4096 // group),
                f=group * _log(rng, 1, 1536 // group), k=rng.randint(1, min(E, 8)), group=group, zeros=zeros, act=act,
                limit=limit, routing=routing)


# ------------------------------------------------------------------ inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1013 + salt)
    return g


def _type(c):
    return torch.float32 if c.get("dtype") == "f32" else torch.bfloat16


def _randn(g, scale, dtype, *shape):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _scores(T, E, routing, g):
    if routing == "zipf":
        u = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-12, 1.0 - 1e-7)
        p = torch.arange(1, E + 1, device=DEV, dtype=torch.float32).pow(-1.2)
        return torch.log(p / p.sum()) - torch.log(-torch.log(u))
    return torch.randn(T, E, generator=g, device=DEV)


def _route(T, E, k, routing, g):
    """The route map of T tokens as moe_route_topk makes it."""
    top = torch.topk(_scores(T, E, routing, g), k, dim=1)
    idx = top.indices.reshape(-1)
    order = torch.argsort(idx, stable=True)
    dst = torch.empty_like(order)
    dst[order] = torch.arange(T * k, device=DEV)
    counts = torch.bincount(idx, minlength=E)
    return dict(topk_idx=top.indices.to(torch.int32), topk_w=torch.softmax(top.values, 1), dst_row=dst.to(torch.int32),
                src_slot=order.to(torch.int32), offsets=torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32),
                sizes=counts.tolist())             # sizes: the plain form's loop over the experts


def _int4_of(w, group, zeros):
    """4-bit codes [rows, K/2], scales and zero points [rows, K/group] of fp32 w (weights as a program keeps them)."""
    rows, K = w.shape
    b = w.view(rows, K // group, group)
    if zeros:
        lo, hi = b.amin(-1).clamp(max=0), b.amax(-1).clamp(min=0)
        s = (hi / 2 - lo / 2) / 7.5
    else:
        s = b.abs().amax(-1) / 7
    s = s.to(torch.bfloat16).float().clamp(min=2.0 ** -126)
    z = torch.round(-lo / s).clamp(0, 15) if zeros else torch.full_like(s, 8)
    q = (torch.round(b / s[..., None]).clamp(-15 if zeros else -8, 15 if zeros else 7) + z[..., None]).clamp(0, 15)
    q = q.to(torch.uint8).view(rows, K)
    return q[:, 0::2] | (q[:, 1::2] << 4), s.to(torch.bfloat16), z.to(torch.uint8) if zeros else None


def prepare(case, seed):
    c = dict(case)
    s = dict(case=c)
    op = c["op"]
    if op in ("dropout", "combine", "gated"):
        s["rng"] = torch.tensor([(int(seed) * 0x9E3779B97F4A7C15 + 12345) & (2 ** 63 - 1), 7 + int(seed)],
                                dtype=torch.int64, device=DEV)   # (seed, step)
    if op == "dropout":
        g, t = _gen(seed, 1), _type(c)
        s["x"] = _randn(g, 1.0, t, c["T"], c["d"])
        s["residual"] = _randn(g, 2.0, t, c["T"], c["d"]) if c["residual"] else None
        s["out"] = torch.empty_like(s["x"]) if own else None
        return s
    if op == "combine":
        g, t = _gen(seed, 2), _type(c)
        T, d, k = c["T"], c["d"], c["k"]
        r = _route(T, max(k, 16), k, "uniform", g)
        s.update(dst_row=r["dst_row"], topk_w=r["topk_w"], y=_randn(g, 1.0, t, T * k, d),
                 residual=_randn(g, 2.0, t, T, d), dout=_randn(g, 1.0, t, T, d))
        if own:
            s["out"], s["dsum"] = torch.empty_like(s["residual"]), torch.empty_like(s["dout"])
        return s
    if op == "gated":
        g, t = _gen(seed, 3), _type(c)
        R, E, d, f = c["R"], c["E"], c["d"], c["f"]
        sizes = _route(R, E, 1, c["routing"], g)["sizes"]
        s["sizes"] = sizes
        s["offsets"] = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32, device=DEV)
        s["x"] = _randn(g, 1.0, t, R, d)                 # the output of a norm: unit variance
        s["w13"] = _randn(g, 1.25 / math.sqrt(d), t, E, 2 * f, d)
        s["w2"] = _randn(g, 1.0 / math.sqrt(f), t, E, d, f)
        if c["part"] == "backward":
            s["dy"] = _randn(g, 1.0, t, R, d)
            s["gu"], s["h"], _ = _gated_plain(s, y=False)   # as the forward saved them
        if own:
            m = _package()
            e = dict(dtype=t, device=DEV)
            if c["part"] == "forward":
                s.update(gu=torch.empty(R, 2 * f, **e), h=torch.empty(R, f, **e), y=torch.empty(R, d, **e))
            else:
                s.update(dgu=torch.empty(R, 2 * f, **e), dx=torch.empty(R, d, **e), dw13=torch.empty(E, 2 * f, d, **e),
                         dw2=torch.empty(E, d, f, **e),
                         ws=torch.empty(m.moe_gemm_workspace_bytes(m.MOE_F32 if c["dtype"] == "f32" else m.MOE_BF16,
                                                                   E, R, d, f), dtype=torch.uint8, device=DEV))
        return s
    if op == "quantise":
        g = _gen(seed, 4)
        rows, K, n = c["rows"], c["K"], c["K"] // c["group"]
        w = torch.randn(rows, K, generator=g, device=DEV) * 0.02
        w[:, ::97] *= 4.0                                # outlier channels
        s["w"] = w.to(torch.bfloat16)
        if own:
            s["codes"] = torch.empty(rows, K // 2, dtype=torch.uint8, device=DEV)
            s["scales"] = torch.empty(rows, n, dtype=torch.bfloat16, device=DEV)
            s["zeros"] = torch.empty(rows, n, dtype=torch.uint8, device=DEV) if c["zeros"] else None
            s["back"] = torch.empty_like(s["w"])
        return s
    g = _gen(seed, 5)
    T, E, d, f, k = c["T"], c["E"], c["d"], c["f"], c["k"]
    s["x"] = _randn(g, 1.0, torch.bfloat16, T, d)
    s.update(_route(T, E, k, c["routing"], g))
    w13 = [_int4_of(torch.randn(2 * f, d, generator=g, device=DEV) * (1.25 / math.sqrt(d)), c["group"], c["zeros"])
           for _ in range(E)]
    w2 = [_int4_of(torch.randn(d, f, generator=g, device=DEV) / math.sqrt(f), c["group"], c["zeros"]) for _ in range(E)]
    s["w13"], s["w2"] = (tuple(torch.stack(p) if p[0] is not None else None for p in zip(*w)) for w in (w13, w2))
    if own:
        m = _package()
        s["out"] = torch.empty_like(s["x"])
        s["ws"] = torch.empty(m.moe_int4_workspace_bytes(T * k, d, f), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    m, c = _package(), s["case"]
    op = c["op"]
    dt = m.MOE_F32 if c.get("dtype") == "f32" else m.MOE_BF16
    if op == "dropout":
        m.moe_dropout(dt, s["x"], c["p"], s["rng"], s["out"], residual=s["residual"])
        return s["out"]
    if op == "combine":
        m.moe_combine_dropout(dt, s["y"], s["dst_row"], s["topk_w"], c["k"], c["p"], s["rng"], s["out"],
                              residual=s["residual"])
        m.moe_dropout(dt, s["dout"], c["p"], s["rng"], s["dsum"])
        return s["out"], s["dsum"]
    if op == "gated":
        gate = m.glu(getattr(m, "MOE_ACT_" + c["act"].upper()), limit=c["limit"], p=c["p"], rng=s["rng"])
        if c["part"] == "forward":
            m.moe_grouped_glu_fwd(dt, gate, s["x"], s["w13"], s["w2"], s["offsets"], 0, s["gu"], s["h"], s["y"])
            return s["gu"], s["h"], s["y"]
        m.moe_grouped_glu_bwd(dt, gate, s["dy"], s["x"], s["gu"], s["h"], s["w13"], s["w2"], s["offsets"], 0, s["dgu"],
                              s["dx"], s["dw13"], s["dw2"], ws=s["ws"])
        return s["dgu"], s["dx"], s["dw13"], s["dw2"]
    if op == "quantise":
        m.moe_quantize_int4(s["w"], c["group"], s["codes"], s["scales"], s["zeros"])
        m.moe_dequantize_int4(s["codes"], s["scales"], s["zeros"], c["group"], s["back"])
        return [t for t in (s["back"], s["scales"], s["zeros"]) if t is not None]
    gate = m.glu(getattr(m, "MOE_ACT_" + c["act"].upper()), limit=c["limit"])
    m.moe_int4_ffn(gate, s["x"], s["topk_idx"], s["topk_w"], s["dst_row"], s["src_slot"], s["offsets"], c["group"],
                   s["w13"], s["w2"], s["out"], s["ws"])
    return s["out"]


def _philox(rng, blocks):
    """The generator's four 32-bit words for counters (block, step) under the key seed: int64 tensors."""
    low = 0xFFFFFFFF
    seed, step = rng[0], rng[1]
    b = torch.arange(blocks, device=rng.device)
    c = [b & low, b >> 32, (step & low).expand(blocks), ((step >> 32) & low).expand(blocks)]
    k0, k1 = seed & low, (seed >> 32) & low

    def mul(a, x):                                       # both halves of the 64-bit product
        lo, hi = a * (x & 0xFFFF), a * (x >> 16)
        return (hi + (lo >> 16)) >> 16, (lo + ((hi & 0xFFFF) << 16)) & low

    for _ in range(10):
        h0, l0 = mul(0xD2511F53, c[0])
        h1, l1 = mul(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c


def _threshold(p):
    return min(int(np.rint(np.float32(p) * 65536)), 65535)


def _kept(rng, rows, cols, p):
    """Truth values [rows, cols] and the factor of what is kept.  Eight elements of the flat tensor share a block."""
    n = rows * cols
    words = torch.stack(_philox(rng, (n + 7) // 8), 1)
    u = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]
    thr = _threshold(p)
    return (u >= thr).view(rows, cols), 65536.0 / (65536 - thr)


def _dropped(v, rng, p):
    keep, scale = _kept(rng, v.shape[0], v.shape[1], p)
    return torch.where(keep, v * scale, 0.0)


def _act(name, g):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    if name == "relu":
        return g.clamp(min=0)
    if name == "gelu":
        return g * 0.5 * torch.special.erfc(g * -math.sqrt(0.5))
    return g * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_slope(name, g):
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    if name == "relu":
        return (g > 0).to(g.dtype)
    if name == "gelu":
        return 0.5 * torch.special.erfc(g * -math.sqrt(0.5)) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _gated_plain(s, y=True):
    c = s["case"]
    f, L, t = c["f"], c["limit"], s["x"].dtype
    gus, at = [], 0
    for e, n in enumerate(s["sizes"]):
        if n:
            gus.append(s["x"][at:at + n].float() @ s["w13"][e].float().t())
        at += n
    gu = torch.cat(gus)
    g, u = gu[:, :f], gu[:, f:]
    if L:
        g, u = g.clamp(max=L), u.clamp(-L, L)
    h = _act(c["act"], g) * u
    if c["p"]:
        h = _dropped(h, s["rng"], c["p"])
    if not y:
        return gu.to(t), h.to(t), None
    ys, at = [], 0
    for e, n in enumerate(s["sizes"]):
        if n:
            ys.append(h[at:at + n] @ s["w2"][e].float().t())
        at += n
    return gu.to(t), h.to(t), torch.cat(ys).to(t)


def _gated_back_plain(s):
    c = s["case"]
    f, L, t = c["f"], c["limit"], s["x"].dtype
    dhs, at = [], 0
    for e, n in enumerate(s["sizes"]):
        if n:
            dhs.append(s["dy"][at:at + n].float() @ s["w2"][e].float())
        at += n
    dh = torch.cat(dhs)
    if c["p"]:
        dh = _dropped(dh, s["rng"], c["p"])
    g, u = s["gu"][:, :f].float(), s["gu"][:, f:].float()
    gc, uc = (g.clamp(max=L), u.clamp(-L, L)) if L else (g, u)
    dg, du = dh * uc * _act_slope(c["act"], gc), dh * _act(c["act"], gc)
    if L:
        dg, du = torch.where(g <= L, dg, 0.0), torch.where(u.abs() <= L, du, 0.0)
    dgu = torch.cat([dg, du], 1)
    dxs, at = [], 0
    dw13, dw2 = torch.empty_like(s["w13"]), torch.empty_like(s["w2"])
    for e, n in enumerate(s["sizes"]):
        own_rows = slice(at, at + n)
        if n:
            dxs.append(dgu[own_rows] @ s["w13"][e].float())
        dw13[e] = (dgu[own_rows].t() @ s["x"][own_rows].float()).to(t)
        dw2[e] = (s["dy"][own_rows].float().t() @ s["h"][own_rows].float()).to(t)
        at += n
    return dgu.to(t), torch.cat(dxs).to(t), dw13, dw2


def _codes(codes):
    return torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1)


def _values(w, group):
    """fp32 values of 4-bit integers: w = codes [rows, K/2], scales [rows, K/group] and zero points or None."""
    codes, scales, zeros = w
    q = _codes(codes).float().view(codes.shape[0], -1, group)
    z = zeros.float()[..., None] if zeros is not None else 8.0
    return ((q - z) * scales.float()[..., None]).view(codes.shape[0], -1)


def _expert(w, e):
    return tuple(p[e] if p is not None else None for p in w)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "dropout":
        v = _dropped(s["x"].float(), s["rng"], c["p"])
        return (v if s["residual"] is None else s["residual"].float() + v).to(s["x"].dtype)
    if op == "combine":
        T, k = c["T"], c["k"]
        dst = s["dst_row"].view(T, k).long()
        v = s["topk_w"][:, :1] * s["y"][dst[:, 0]].float()
        for j in range(1, k):
            v += s["topk_w"][:, j:j + 1] * s["y"][dst[:, j]].float()
        keep, scale = _kept(s["rng"], T, c["d"], c["p"])
        t = s["y"].dtype
        return ((s["residual"].float() + torch.where(keep, v * scale, 0.0)).to(t),
                torch.where(keep, s["dout"].float() * scale, 0.0).to(t))
    if op == "gated":
        return _gated_plain(s) if c["part"] == "forward" else _gated_back_plain(s)
    if op == "quantise":
        codes, scales, zeros = _int4_of(s["w"].float(), c["group"], c["zeros"])
        back = _values((codes, scales, zeros), c["group"]).to(torch.bfloat16)
        return [t for t in (back, scales, zeros) if t is not None]
    T, k, f, L = c["T"], c["k"], c["f"], c["limit"]
    xp = s["x"].float()[torch.div(s["src_slot"], k, rounding_mode="floor").long()]
    ys, at = [], 0
    for e, n in enumerate(s["sizes"]):
        if not n:
            continue
        gu = xp[at:at + n] @ _values(_expert(s["w13"], e), c["group"]).t()
        g, u = gu[:, :f], gu[:, f:]
        if L:
            g, u = g.clamp(max=L), u.clamp(-L, L)
        ys.append((_act(c["act"], g) * u) @ _values(_expert(s["w2"], e), c["group"]).t())
        at += n
    y = torch.cat(ys)[s["dst_row"].long()].view(T, k, -1)
    return (y * s["topk_w"][..., None]).sum(1).to(torch.bfloat16)


# ------------------------------------------------------------------ bytes and operations
def work(case):
    c = case
    e = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "dropout":
        n = c["T"] * c["d"]
        return dict(bytes=(3 if c["residual"] else 2) * n * e, flops=12 * n)
    if c["op"] == "combine":
        n = c["T"] * c["d"]
        return dict(bytes=(c["k"] + 4) * n * e + 8 * c["T"] * c["k"], flops=(2 * c["k"] + 24) * n)
    if c["op"] == "gated":
        R, E, d, f = c["R"], c["E"], c["d"], c["f"]
        hit = E * (1 - (1 - 1 / E) ** R)                   # experts with a row, for even routing
        if c["part"] == "forward":
            return dict(bytes=(2 * R * d + 3 * R * f + hit * 3 * d * f) * e, flops=6 * R * d * f)
        return dict(bytes=(3 * R * d + 5 * R * f + (hit + E) * 3 * d * f) * e, flops=12 * R * d * f)
    a = 0.5 + (3 if c["zeros"] else 2) / c["group"]        # bytes of a 4-bit element
    if c["op"] == "quantise":
        n = c["rows"] * c["K"]
        return dict(bytes=2 * n * (2 + a), flops=8 * n)
    T, E, d, f, R = c["T"], c["E"], c["d"], c["f"], c["T"] * c["k"]
    hit = E * (1 - (1 - c["k"] / E) ** T)
    return dict(bytes=4 * T * d + hit * 3 * d * f * a + 16 * R + 4 * E, flops=6 * R * d * f)


# ------------------------------------------------------------------ the definition, in 64 bits
def _mask64(rng, n, p):
    """The mask of n elements from the generator's definition (Philox 4x32, ten rounds), in numpy's 64-bit integers."""
    seed, step = (int(v) & (2 ** 64 - 1) for v in rng.tolist())
    u64, low = np.uint64, np.uint64(0xFFFFFFFF)
    out = np.empty((n + 7) // 8 * 8, dtype=bool)
    thr = _threshold(p)
    for b0 in range(0, (n + 7) // 8, 1 << 20):
        b = np.arange(b0, min(b0 + (1 << 20), (n + 7) // 8), dtype=u64)
        x0, x1 = b & low, b >> u64(32)
        x2, x3 = np.full_like(b, step & 0xFFFFFFFF), np.full_like(b, step >> 32)
        for r in range(10):
            a, q = x0 * u64(0xD2511F53), x2 * u64(0xCD9E8D57)
            ka = u64(((seed & 0xFFFFFFFF) + r * 0x9E3779B9) & 0xFFFFFFFF)
            kb = u64(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
            x0, x1, x2, x3 = (q >> u64(32)) ^ x1 ^ ka, q & low, (a >> u64(32)) ^ x3 ^ kb, a & low
        halves = np.stack([x0, x1, x2, x3], 1).astype(np.uint32).view(np.uint16)   # low half first
        out[8 * b0:8 * (b0 + b.size)] = (halves >= thr).reshape(-1)
    return torch.from_numpy(out[:n]).to(DEV)


def _drop64(v, s):
    p = s["case"]["p"]
    return torch.where(_mask64(s["rng"], v.numel(), p).view(v.shape), v / (1 - _threshold(p) / 65536), 0.0)


def _gate64(c, g, u):
    if c["limit"]:
        g, u = g.clamp(max=c["limit"]), u.clamp(-c["limit"], c["limit"])   # slope 1 at the limits themselves
    a = c["act"]
    if a == "silu":
        v = g * torch.sigmoid(g)
    elif a == "relu":
        v = torch.where(g > 0, g, 0.0)
    elif a == "gelu":
        v = g * torch.special.ndtr(g)
    else:
        v = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))   # (1 + tanh z) / 2 = sigmoid(2 z)
    return v * u


def _decoded(w, group):
    codes, scales, zeros = w
    q = _codes(codes).double()
    z = zeros.double().repeat_interleave(group, 1) if zeros is not None else 8.0
    return (q - z) * scales.double().repeat_interleave(group, 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "dropout":
        v = _drop64(s["x"].double(), s)
        return v if s["residual"] is None else v + s["residual"].double()
    if op == "combine":
        T, k, d = c["T"], c["k"], c["d"]
        v = torch.zeros(T, d, dtype=torch.float64, device=DEV)
        for j in range(k):
            v.addcmul_(s["y"].double()[s["dst_row"][j::k].long()], s["topk_w"][:, j].double()[:, None])
        return s["residual"].double() + _drop64(v, s), _drop64(s["dout"].double(), s)
    if op == "gated":
        f, parts, at = c["f"], [], 0
        if c["part"] == "forward":
            gu = torch.cat([s["x"][a:a + n].double() @ s["w13"][e].double().t().contiguous()
                            for e, (a, n) in enumerate(zip(s["offsets"].tolist(), s["sizes"]))])
            h = _drop64(_gate64(c, gu[:, :f], gu[:, f:]), s)
            y = torch.cat([h[a:a + n] @ s["w2"][e].double().t().contiguous()
                           for e, (a, n) in enumerate(zip(s["offsets"].tolist(), s["sizes"]))])
            return gu, h, y
        keep = _mask64(s["rng"], c["R"] * f, c["p"]).view(c["R"], f) / (1 - _threshold(c["p"]) / 65536)
        dw13, dw2 = [], []
        for e, n in enumerate(s["sizes"]):
            r = slice(at, at + n)
            at += n
            dy = s["dy"][r].double()
            gu = s["gu"][r].double().requires_grad_(True)
            dh = (dy @ s["w2"][e].double()) * keep[r]
            (dgu,) = torch.autograd.grad(_gate64(c, gu[:, :f], gu[:, f:]), gu, dh)
            parts.append((dgu, dgu @ s["w13"][e].double()))
            dw13.append(dgu.t().contiguous() @ s["x"][r].double())
            dw2.append(dy.t().contiguous() @ s["h"][r].double())
        return (torch.cat([a for a, _ in parts]), torch.cat([b for _, b in parts]), torch.stack(dw13), torch.stack(dw2))
    if op == "quantise":
        b = s["w"].double().view(c["rows"], -1, c["group"])
        if c["zeros"]:
            top, low = b.amax(-1).clamp(min=0), b.amin(-1).clamp(max=0)
            scale = (top - low) / 15
        else:
            scale = b.abs().amax(-1) / 7
        scale = scale.to(torch.bfloat16).double()          # the scale that is stored
        scale = torch.where(scale < 2.0 ** -126, 2.0 ** -126, scale)
        zero = torch.round(-low / scale).clamp(0, 15) if c["zeros"] else torch.full_like(scale, 8)
        q = torch.round(b / scale[..., None]) + zero[..., None]
        back = (q.clamp(0, 15) - zero[..., None]) * scale[..., None]
        out = [back.view(c["rows"], -1), scale]
        return out + [zero.to(torch.uint8)] if c["zeros"] else out
    T, k, f = c["T"], c["k"], c["f"]
    out = torch.zeros(T, c["d"], dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        t, j = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
        if not t.numel():
            continue
        gu = s["x"][t].double() @ _decoded(_expert(s["w13"], e), c["group"]).t().contiguous()
        y = _gate64(c, gu[:, :f], gu[:, f:]) @ _decoded(_expert(s["w2"], e), c["group"]).t().contiguous()
        out.index_add_(0, t, y * s["topk_w"][t, j].double()[:, None])
    return out
