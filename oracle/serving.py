"""Plain 64-bit forms of the serving operators: window attention, rotary
positions, the 4-bit cache's rows and pages, and the cache plan."""

from __future__ import annotations

import decimal
import math
from decimal import Decimal as D

import numpy as np

TWO_PI = D("6.28318530717958647692528676655900576839433879875021164194989")


def visible(n_q, n_k, window, sinks):
    """[n_q, n_k] truth values: which keys the rows at n_k - n_q + i see."""
    p = n_k - n_q + np.arange(n_q)[:, None]
    j = np.arange(n_k)[None]
    see = j <= p
    return see & ((p - j < window) | (j < sinks)) if window else see


def attention(q, k, v, window, sinks, scale=0.0, extra=None):
    """One head: q [n_q, d], k, v [n_k, d].  Returns out, lse, and two sums for
    error bounds: sum_j w_j |v_j| and the largest scale sum_c |q_c| (|k_c| + extra_c)
    of a visible key.  Keys that no row sees are left out."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n_q, d = q.shape
    scale = scale or 1 / math.sqrt(d)
    see = visible(n_q, k.shape[0], window, sinks)
    used = see.any(0)
    k, v, see = k[used], v[used], see[:, used]
    big = np.abs(k) + (0 if extra is None else extra[used])
    out, absv = np.zeros((n_q, d)), np.zeros((n_q, d))
    lse, size = np.full(n_q, -np.inf), np.zeros(n_q)
    if used.any():
        s = np.where(see, q @ k.T * scale, -np.inf)
        size = np.where(see, np.abs(q) @ big.T * scale, 0).max(1)
        m = s.max(1)
        some = m > -np.inf
        e = np.exp(s - np.where(some, m, 0)[:, None])
        total = e.sum(1)
        w = e / np.where(some, total, 1)[:, None]
        out, absv = w @ v, w @ np.abs(v)
        with np.errstate(divide="ignore"):
            lse = np.where(some, m + np.log(total), -np.inf)
    return out, lse, absv, size


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """Radians per position of each pair, and the factor on the result."""
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    w = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return w / factor, 1.0
    if scaling != "yarn":
        return w, 1.0

    def pair(turns):
        return rot * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(0, math.floor(pair(beta_fast))), min(rot - 1, math.ceil(pair(beta_slow)))
    r = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
    return w * (1 - r) + w / factor * r, 0.1 * math.log(factor) + 1


def rope_turns(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """The frequencies in turns per position, as decimal fractions of 60 digits."""
    with decimal.localcontext(decimal.Context(prec=60)):
        base, factor = D(base), D(factor)
        if scaling == "ntk" and rot > 2:
            base *= (factor.ln() * rot / (rot - 2)).exp()
        w = [(base.ln() * -2 * i / rot).exp() for i in range(rot // 2)]
        if scaling == "linear":
            w = [x / factor for x in w]
        if scaling == "yarn":
            def pair(turns):
                return rot * (D(original_len) / (D(turns) * TWO_PI)).ln() / (2 * base.ln())
            lo, hi = max(0, math.floor(pair(beta_fast))), min(rot - 1, math.ceil(pair(beta_slow)))
            r = [min(D(1), max(D(0), D(i - lo) / (D(hi - lo) if hi > lo else D("0.001")))) for i in range(rot // 2)]
            w = [x * (1 - y) + x / factor * y for x, y in zip(w, r)]
        return [x / TWO_PI for x in w]


def far_angles(pos, turns):
    """[T, pairs]: the angles of positions (of any size and sign) as radians within half a turn."""
    with decimal.localcontext(decimal.Context(prec=60)):
        rest = [[(int(p) * t) % 1 for t in turns] for p in pos]
        return np.array([[float((r - round(r)) * TWO_PI) for r in row] for row in rest])


def rope(x, pos, w, mag, layout, inverse=False):
    """x [..., T, H, d], pos [..., T].  Also |x1| + |x2| of every output's pair."""
    x = np.asarray(x, np.float64)
    a = np.asarray(pos, np.float64)[..., None, None] * w * (-1 if inverse else 1)
    c, s = np.cos(a) * mag, np.sin(a) * mag
    n = w.size
    one, two = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    x1, x2 = x[..., one], x[..., two]
    y, size = x.copy(), np.zeros_like(x)
    y[..., one], y[..., two] = x1 * c - x2 * s, x2 * c + x1 * s
    size[..., one] = size[..., two] = (np.abs(x1) + np.abs(x2)) * mag
    return y, size


# ---------------------------------------------------------------------------
# The 4-bit cache
# ---------------------------------------------------------------------------

def round_bf16(x):
    """float64 to the nearest bf16 (ties to even), as float64; subnormals included."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    unit = np.ldexp(1.0, np.maximum(e - 8, -133))
    return np.rint(x / unit) * unit


def quantise(x):
    """bf16 values [..., d] to codes [..., d] in [-7, 7] and scales [..., d / 32]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = np.abs(g).max(-1)
    s = np.where(np.isfinite(top), round_bf16(np.where(np.isfinite(top), top, 0) / 7), np.nan)
    ok = (s > 0)[..., None]
    c = np.where(ok, np.clip(np.rint(np.where(ok, g, 0) / np.where(ok, s[..., None], 1)), -7, 7), 0)
    return c.reshape(x.shape).astype(np.int64), s


def values(codes, scales):
    c = codes.reshape(*codes.shape[:-1], codes.shape[-1] // 32, 32)
    return (c * scales[..., None]).reshape(codes.shape)


def bf16_bits(x):
    bits = (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), bits)


def store(pages, slot, h, kc, ks, vc, vs):
    """One token's codes [d] and scales [d / 32] into pages uint8 [n, Hkv, page / 16, 18 d], byte by byte."""
    per = pages.shape[2] * 16
    page, place = divmod(int(slot), per)
    sub, t = pages[page, h, place // 16], place % 16
    d = kc.size
    G = d // 32
    p, t4, hi = t // 8, t % 8 // 2, t % 2
    for c in range(0, d, 2):
        g, r = divmod(c, 32)
        sub[t * 16 * G + r // 8 * 4 * G + g * 4 + r % 8 // 2] = (kc[c] + 8) | (kc[c + 1] + 8) << 4
        at = 256 * G + p * 128 * G + (r // 4 * 4 + t4) * 4 * G + g * 4 + hi * 2 + r % 4 // 2
        sub[at] = (vc[c] + 8) | (vc[c + 1] + 8) << 4
    kb, vb = bf16_bits(ks).view(np.uint8), bf16_bits(vs).view(np.uint8)
    for g in range(G):
        a, b = 512 * G + t * 2 * G + 2 * g, 544 * G + p * 16 * G + t4 * 4 * G + 4 * g + 2 * hi
        sub[a:a + 2], sub[b:b + 2] = kb[2 * g:2 * g + 2], vb[2 * g:2 * g + 2]


# ---------------------------------------------------------------------------
# The cache plan
# ---------------------------------------------------------------------------

def plan(kv_len, q_len, table, free, page, max_tokens):
    """One step: the same results as lists, with free the stack's entries (top
    last).  Raises MemoryError where the pages, blocks or token places run out."""
    table = [list(r) for r in table]
    free, num = list(free), 0
    for b, (old, add) in enumerate(zip(kv_len, q_len)):
        if add < 0:
            free += table[b][:-(-old // page)]
    peak = list(free)
    slots, positions, cu, new_len = [], [], [0], []
    for b, (old, add) in enumerate(zip(kv_len, q_len)):
        if add < 0:
            new_len.append(0)
            cu.append(cu[-1])
            continue
        for blk in range(-(-old // page), -(-(old + add) // page)):
            if not free or blk >= len(table[b]):
                raise MemoryError
            table[b][blk] = free.pop()
        for pos in range(old, old + add):
            slots.append(table[b][pos // page] * page + pos % page)
            positions.append(pos)
        cu.append(cu[-1] + add)
        new_len.append(old + add)
    num = max_tokens - len(slots)
    if num < 0:
        raise MemoryError
    return dict(table=table, free=free, peak=peak, new_len=new_len, cu_q=cu, slots=slots + [-1] * num,
                positions=positions + [0] * num)
