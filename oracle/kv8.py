"""The paged 8-bit cache in fp64: codes, the append's quantisation, attention over the cached values.

A code is one byte, e4m3 (sign, 4 exponent bits with bias 7, 3 mantissa bits; 0x7F and 0xFF are NaN, no
infinity) or int8 (-127 .. 127).  A block is 16 consecutive tokens of one head; its codes share a scale.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16
QMAX = {"e4m3": 448.0, "int8": 127.0}


def _e4m3_value(byte):
    sign, exp, man = byte >> 7, (byte >> 3) & 15, byte & 7
    if exp == 15 and man == 7:
        return math.nan
    v = man * 2.0 ** -9 if exp == 0 else (8 + man) * 2.0 ** (exp - 10)
    return -v if sign else v


E4M3 = np.array([_e4m3_value(b) for b in range(256)])
_POS = E4M3[:127]  # 0 .. 448, ascending


def decode(codes, kind):
    """Values of codes (uint8 array)."""
    return E4M3[codes] if kind == "e4m3" else codes.astype(np.uint8).view(np.int8).astype(np.float64)


def encode(y, kind):
    """Nearest codes of values (ties to the even code), saturating; uint8 array."""
    y = np.asarray(y, dtype=np.float64)
    if kind == "int8":
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)  # first value >= a
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - a, a - _POS[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    c = np.where(_POS[hi] == a, hi, c)
    return (c | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def block_scale(top, kind):
    """Smallest power of two s >= 2^-126 with top <= qmax s."""
    e = -126
    if top > 0:
        e = max(-126, math.frexp(top)[1] - math.frexp(QMAX[kind])[1] - 1)
        while top > QMAX[kind] * 2.0 ** e:
            e += 1
    return 2.0 ** e


def append(x, pages, scales, table, seqlens, new_lens, page_size, kind):
    """One pool (K or V) after the append of x [B, Nt, Hkv, D] (fp64): new (pages, scales, saw a non-finite)."""
    pages, scales, odd = pages.copy(), scales.astype(np.float64), False
    B, _, Hkv, _ = x.shape
    for b in range(B):
        end, n = int(seqlens[b]), int(new_lens[b])
        first = end - n
        for blk in range(first // BLOCK, -(-end // BLOCK) if n else 0):
            lo, hi = max(first, blk * BLOCK), min(end, (blk + 1) * BLOCK)
            page, r = int(table[b, blk * BLOCK // page_size]), blk * BLOCK % page_size
            for h in range(Hkv):
                v = x[b, lo - first:hi - first, h]
                fin = np.isfinite(v)
                odd |= not fin.all()
                s = block_scale(float(np.abs(v[fin]).max(initial=0.0)), kind)
                old = lo - blk * BLOCK
                if old:
                    was = float(scales[page, h, r // BLOCK])
                    s = max(s, was)
                    if s != was:
                        c = pages[page, h, r:r + old]
                        pages[page, h, r:r + old] = encode(decode(c, kind) * (was / s), kind)
                scales[page, h, r // BLOCK] = s
                q = np.where(np.isnan(v), 0.0, v) / s
                pages[page, h, r + old:r + old + hi - lo] = encode(np.clip(q, -QMAX[kind], QMAX[kind]), kind)
    return pages, scales, odd


def rows(pages, scales, table_row, n, page_size, h, kind):
    """The first n cached values of head h of a sequence, [n, D]."""
    out = []
    for i in range(-(-n // page_size)):
        p = int(table_row[i])
        out.append(decode(pages[p, h], kind) * np.repeat(scales[p, h].astype(np.float64), BLOCK)[:, None])
    return np.concatenate(out)[:n] if out else np.zeros((0, pages.shape[-1]))


def attend(q, k_pages, v_pages, k_scales, v_scales, table, seqlens, page_size, scale, kind):
    """O [B, Nq, Hq, D], LSE [B, Hq, Nq] and, per element of O, sum_j p_j |V_j|; per row, the largest
    scale * sum_d |q_d K_jd| and the largest p_j * vs(j) of a visible key (what error bounds need)."""
    B, Nq, Hq, D = q.shape
    Hkv = k_pages.shape[1]
    G = Hq // Hkv
    o, spread = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((B, Hq, Nq), -np.inf)
    mass, top = np.zeros((B, Hq, Nq)), np.zeros((B, Hq, Nq))
    for b in range(B):
        n = int(seqlens[b])
        vs_of = np.concatenate([v_scales[int(p)] for p in table[b, : -(-n // page_size)]], axis=-1) if n else None
        for h in range(Hkv):
            K, V = rows(k_pages, k_scales, table[b], n, page_size, h, kind), rows(v_pages, v_scales, table[b], n, page_size, h, kind)
            for i in range(Nq):
                vis = min(n, n - Nq + i + 1)
                if vis <= 0:
                    continue
                Q = q[b, i, h * G:(h + 1) * G]
                s = scale * (Q @ K[:vis].T)
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(1, keepdims=True)
                sl = slice(h * G, (h + 1) * G)
                o[b, i, sl] = (p / l) @ V[:vis]
                lse[b, sl, i] = (m + np.log(l))[:, 0]
                spread[b, i, sl] = (p / l) @ np.abs(V[:vis])
                mass[b, sl, i] = (scale * (np.abs(Q) @ np.abs(K[:vis]).T)).max(1)
                top[b, sl, i] = (p / l * np.repeat(vs_of[h], BLOCK)[:vis]).max(1)
    return o, lse, spread, mass, top
