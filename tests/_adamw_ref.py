"""Plain references of the steps over lists of tensors, in 64 bits (numpy), written from the rules stated in
include/ob_adam.h; an fp32 rounding that a rule states is made with astype(float32).  Test infrastructure."""
from __future__ import annotations

import numpy as np

BLOCK = 256
F32 = np.float32


def r32(x):
    """x rounded to fp32, as fp64."""
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        return np.asarray(x, np.float64).astype(F32).astype(np.float64)


def philox_words(seed, t, count):
    """Words of elements 0..count-1 (uint32): output word i & 3 of Philox4x32-10 at the counter (i >> 2, t)."""
    n = -(-count // 4)
    M = np.uint64(0xFFFFFFFF)
    blk = np.arange(n, dtype=np.uint64)
    c = [blk & M, blk >> np.uint64(32), np.full(n, t & 0xFFFFFFFF, np.uint64), np.full(n, (t >> 32) & 0xFFFFFFFF, np.uint64)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & M, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & M]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).reshape(-1)[:count].astype(np.uint32)


PAR_STREAM = 1 << 63


# ---- the 8-bit format ----

def code_value(k, q, second):
    r = r32(np.asarray(k, np.float64) ** 2 * q)
    return r32(r * r) if second else r


def decode(codes, scales, second):
    """fp64 values (exact fp32 numbers); codes of any length, one scale per 256."""
    c = codes.astype(np.float64)
    q = np.repeat(np.asarray(scales, np.float64), BLOCK)[: len(c)]
    with np.errstate(invalid="ignore"):
        return code_value(c, q, True) if second else np.sign(c) * code_value(np.abs(c), q, False) + 0 * q


def scales_of(x, second):
    """Scales of the blocks of x (fp32 values); short last block allowed."""
    most = 255 if second else 127
    out = []
    for s in range(0, len(x), BLOCK):
        b = np.asarray(x[s:s + BLOCK], np.float64)
        if not np.all(np.isfinite(b)) or (second and np.any(b < 0)):
            out.append(np.nan)
            continue
        top = np.max(np.abs(b))
        out.append(0.0 if top < 2.0 ** -96 else float(r32((r32(np.sqrt(top)) if second else top) * r32(1 / most ** 2))))
    return np.array(out, F32)


def encode(x, second, words=None):
    """(codes, scales); words: the elements' random words, or None for rounding to nearest.  Codes by bisection over
    the borders, which are fp32 numbers by the rules."""
    most = 255 if second else 127
    scales = scales_of(x, second)
    q = np.repeat(scales.astype(np.float64), BLOCK)[: len(x)]
    a = np.abs(np.asarray(x, np.float64))
    live = q > 0
    q, a = np.where(live, q, 1.0), np.where(live, a, 0.0)
    lo, hi = np.zeros(len(a)), np.full(len(a), float(most))
    half = 0.5 if words is None else 0.0
    while np.any(lo < hi):
        mid = np.ceil((lo + hi) / 2)
        up = a >= code_value(mid - half, q, second)
        lo, hi = np.where(up, mid, lo), np.where(up, hi, mid - 1)
    k = lo
    if words is not None:
        u = ((words >> 16) if second else (words & 0xFFFF)).astype(np.float64)
        low = code_value(k, q, second)
        gap = r32(code_value(k + 1, q, second) - low)
        k = np.minimum(k + (r32(u * gap) < r32(r32(a - low) * 65536)), most)
    if second:
        k = np.where(a > 0, np.maximum(k, 1), k)
    k = np.where(live, k, 0)
    if second:
        return k.astype(np.uint8), scales
    return (np.sign(np.where(live, x, 0.0)) * k).astype(np.int8), scales


# ---- the steps ----

def grad_norm(grads, g_mult, max_norm):
    """(norm, factor) in fp64 of fp64 gradients; both arguments are fp32 numbers to the call."""
    g_mult, max_norm = float(F32(g_mult)), float(F32(max_norm))
    s = sum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads if g is not None)
    norm = abs(g_mult) * np.sqrt(s)
    f = min(1.0, max_norm / (norm + 1e-6)) if 0 < max_norm < np.inf else 1.0
    return norm, g_mult * f


def adamw(g, m, v, p, *, lr, beta1, beta2, eps, wd, bc1=1.0, bc2=1.0, scale=1.0):
    """fp32 states: unrounded (m, v) and p from the rounded moments, all fp64.  The rates are fp64."""
    b1, b2 = float(F32(beta1)), float(F32(beta2))
    g = r32(np.asarray(g, np.float64) * float(F32(scale)))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    u = (r32(m) / bc1) / (np.sqrt(r32(v) / bc2) + float(F32(eps)))
    return m, v, p - lr * (u + wd * p), u


def adamw8_moments(g, m, v, *, beta1, beta2, scale=1.0):
    """8-bit states: the fp32 moments of the step from decoded ones (fp64 arrays of fp32 numbers).  A product of fp32
    numbers is exact in fp64, and a sum of such a product and an fp32 number, rounded to fp64 and then to fp32, is the
    fused operation's value but where the fp64 sum falls on an fp32 midpoint by its own rounding (2^-29 of cases)."""
    b1, b2 = float(F32(beta1)), float(F32(beta2))
    c1, c2 = float(r32(1 - b1)), float(r32(1 - b2))
    g = r32(np.asarray(g, np.float64) * float(F32(scale)))
    return r32(b1 * m + r32(c1 * g)), r32(b2 * v + r32(c2 * r32(g * g)))


def bc(beta, t):
    return 1 - float(F32(beta)) ** t
