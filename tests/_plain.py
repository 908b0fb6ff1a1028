"""Plain 64-bit implementations (numpy) of the MXFP4 codec and of the router's
balance loss, for the tests.  They share nothing with the HIP library."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def mxfp4_quantize(v):
    """v [rows, K] float64 -> codes [rows, K/2] uint8, scales [rows, K/32] uint8."""
    v = np.asarray(v, np.float64)
    rows, K = v.shape
    b = v.reshape(rows, K // 32, 32)
    code = np.zeros(b.shape, np.uint8)
    scale = np.zeros(b.shape[:2], np.uint8)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    for r in range(rows):
        for j in range(K // 32):
            x = b[r, j]
            if not np.isfinite(x).all():
                scale[r, j] = 255
                continue
            top = np.abs(x).max()
            e = -127
            while e < 127 and top > 6 * 2.0 ** e:
                e += 1
            scale[r, j] = e + 127
            q = np.abs(x) / 2.0 ** e
            c = np.searchsorted(mid, q, side="left")          # a midpoint goes to the lower value
            tie = (c < 7) & (q == mid[np.minimum(c, 6)]) & (c % 2 == 1)
            c = c + tie                                       # ... unless that one's code is odd
            code[r, j] = c | (np.signbit(x).astype(np.uint8) << 3)
    code = code.reshape(rows, K)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), scale


def mxfp4_decode(codes, scales):
    """The values (float64) of codes [..., K/2] and scales [..., K/32]."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    v = np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def mxfp4_qdq(v):
    return mxfp4_decode(*mxfp4_quantize(v))


def bf16_round(v):
    """Round to nearest even at 8 significant bits (values in bf16's normal range)."""
    m, e = np.frexp(np.asarray(v, np.float64))
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def balance(logits, topk_idx, cb, cz, seg_off=None, mask=None, dlosses=(1.0, 1.0), counts=None):
    """The balance loss, z loss, counts and their gradient, token by token in
    float64.  counts given: used as they are (finite differences keep them)."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    seg_off = [0, T] if seg_off is None else [int(v) for v in seg_off]
    S = len(seg_off) - 1
    seg = np.full(T, -1)
    for s in range(S):
        seg[seg_off[s]:seg_off[s + 1]] = s
    if mask is not None:
        seg[np.asarray(mask) == 0] = -1
    p = np.zeros((T, E))
    lse = np.zeros(T)
    for t in range(T):
        fin = np.isfinite(x[t])
        if seg[t] < 0 or not fin.any():
            continue
        top = x[t][fin].max()
        ex = np.where(fin, np.exp(np.where(fin, x[t], 0) - top, where=fin, out=np.zeros(E)), 0)
        p[t] = ex / ex.sum()
        lse[t] = top + np.log(ex.sum())
    n = np.array([(seg == s).sum() for s in range(S)])
    N = n.sum()
    if counts is None:
        counts = np.zeros((S, E), np.int64)
        for t in range(T):
            for e in topk_idx[t]:
                if seg[t] >= 0 and 0 <= e < E:
                    counts[seg[t], e] += 1
    f = counts / np.maximum(counts.sum(1, keepdims=True), 1)
    probs = np.stack([p[seg == s].sum(0) / max(n[s], 1) for s in range(S)])
    inv = 1 / N if N else 0.0
    losses = np.array([cb * E * inv * (n[:, None] * f * probs).sum(), cz * inv * (lse ** 2).sum()])
    on = seg >= 0
    ft = np.where(on[:, None], f[np.maximum(seg, 0)], 0.0)
    dot = (ft * p).sum(1, keepdims=True)
    g = p * (dlosses[0] * cb * E * inv * (ft - dot) + dlosses[1] * 2 * cz * inv * lse[:, None])
    return dict(losses=losses, counts=counts, probs=probs, lse=lse, tokens=np.append(n, N), p=p, f=ft, dot=dot,
                grad=np.where(on[:, None], g, 0.0))
