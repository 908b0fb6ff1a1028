"""Plain 64-bit implementations of the dropout generator, the gated block and the 4-bit integer codec, for the
tests.  They share nothing with the HIP library."""
import math

import numpy as np
import torch

ACTS = ("silu", "gelu", "gelu_tanh", "relu")     # in the order of MOE_ACT_*


def philox(counter, key):
    """Philox 4x32 with ten rounds: four 32-bit words from a counter of four and a key of two, in Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def philox_blocks(blocks, seed, step):
    """uint32 [n, 4] for an array of block numbers (numpy uint64)."""
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    seed, step = int(seed) & (2 ** 64 - 1), int(step) & (2 ** 64 - 1)
    b = np.asarray(blocks, u)
    c = [b & low, b >> u(32), np.full_like(b, step & 0xFFFFFFFF), np.full_like(b, step >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        x, y = u(0xD2511F53) * c[0], u(0xCD9E8D57) * c[2]
        c = [(y >> u(32)) ^ c[1] ^ u(k[0]), y & low, (x >> u(32)) ^ c[3] ^ u(k[1]), x & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1).astype(np.uint32)


def threshold(p):
    return min(int(np.rint(np.float32(p) * np.float32(65536))), 65535)


def factors(n, p, seed, step, first=0):
    """float64 factors (0 or 65536 / (65536 - thr)) of elements first .. first + n - 1."""
    lo = first // 8
    w = philox_blocks(np.arange(lo, (first + n + 7) // 8, dtype=np.uint64), seed, step)
    halves = np.stack([w & 0xFFFF, w >> 16], -1).reshape(-1)[first - 8 * lo:][:n]
    thr = threshold(p)
    return torch.from_numpy(np.where(halves >= thr, 65536 / (65536 - thr), 0.0))


def act(name, g):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    if name == "relu":
        return torch.where(g < 0, 0.0, g)
    if name == "gelu":
        return g * 0.5 * torch.special.erfc(-g / math.sqrt(2))
    return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))


def slope_terms(name, g):
    """The terms whose sum is the gate's slope."""
    if name == "silu":
        s = torch.sigmoid(g)
        return s, g * s * (1 - s)
    if name == "relu":
        return ((g > 0).double(),)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-g / math.sqrt(2)), g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(c * (g + 0.044715 * g ** 3))
    return s, g * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g)


def limited(g, u, L):
    return (g.clamp(max=L), u.clamp(-L, L)) if L else (g, u)


def int4_quantize(v, group, zeros):
    """v [rows, K] float64 (bf16 values) -> codes [rows, K] 0..15, scales [rows, K/group] float64, zero points."""
    v = np.asarray(v, np.float64)
    b = v.reshape(v.shape[0], -1, group)
    f32 = np.float32

    def bf16(x):
        return torch.from_numpy(x.astype(f32)).to(torch.bfloat16).double().numpy()
    ok = np.isfinite(b).all(-1)
    b = np.where(ok[..., None], b, 0.0)
    if zeros:
        lo, hi = np.minimum(b.min(-1), 0), np.maximum(b.max(-1), 0)
        s = bf16((f32(0.5) * hi.astype(f32) - f32(0.5) * lo.astype(f32)) / f32(7.5))
    else:
        s = bf16(np.abs(b).max(-1).astype(f32) / f32(7))
    s = np.maximum(s, 2.0 ** -126)
    z = np.clip(np.rint(-lo / s), 0, 15) if zeros else np.full(s.shape, 8.0)
    q = np.rint(b / s[..., None])
    q = np.clip(q + z[..., None], 0, 15) if zeros else np.clip(q, -8, 7) + 8
    q, z, s = np.where(ok[..., None], q, 8), np.where(ok, z, 8), np.where(ok, s, np.nan)
    return q.reshape(v.shape).astype(np.uint8), s, z.astype(np.uint8)


def int4_pack(q):
    return (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)


def int4_values(q, s, z, group):
    return (q.astype(np.float64) - np.repeat(z.astype(np.float64), group, 1)) * np.repeat(s, group, 1)
