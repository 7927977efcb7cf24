"""Caches and inputs for the tests of the paged 8-bit cache, and the error bounds of its attention."""
from __future__ import annotations

import numpy as np

import oracle

NAN_CODE = {"e4m3": 0x7F, "int8": 0x80}  # what an unused row is filled with (int8 has no NaN: -128, which no append writes)


def make_cache(rng, lens, Hkv, D, page, kind, spare=3, scales="powers", cols=1):
    """Random codes for each sequence's keys on shuffled pages: (k_pages, v_pages, k_scales, v_scales, table).

    Every byte that no sequence uses is NaN_CODE, every scale of an unused block NaN, every unused table entry -1.
    scales: "powers" (of two, 2^-9 .. 2^-4), "any" (arbitrary fp32), "wild" (V scales from 2^-60 to 2^60 and zeros).
    """
    need = [-(-int(n) // page) for n in lens]
    P = sum(need) + spare
    perm = rng.permutation(P)
    table = np.full((len(lens), max(need + [1]) + cols), -1, dtype=np.int32)
    pools, scs = [], []
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    for which in range(2):
        codes = np.full((P, Hkv, page, D), NAN_CODE[kind], dtype=np.uint8)
        sc = np.full((P, Hkv, page // 16), np.nan, dtype=np.float32)
        for b, n in enumerate(lens):
            for i in range(need[b]):
                r = min(page, int(n) - i * page)
                p = table[b, i]
                y = rng.standard_normal((Hkv, r, D)) * (100 if kind == "e4m3" else 40)
                codes[p, :, :r] = oracle.kv8.encode(y, kind)
                blocks = -(-r // 16)
                if scales == "powers":
                    s = 2.0 ** rng.integers(-9, -4, (Hkv, blocks))
                else:
                    s = np.exp(rng.uniform(-6, -3, (Hkv, blocks)))
                if scales == "wild" and which == 1:
                    s = 2.0 ** rng.integers(-60, 60, (Hkv, blocks))
                    s[rng.random((Hkv, blocks)) < 0.1] = 0.0
                sc[p, :, :blocks] = s
        pools.append(codes)
        scs.append(sc)
    return pools[0], pools[1], scs[0], scs[1], table


def bounds(o, spread, mass, top, keys, D, kind, out):
    """Largest errors of O [B, Nq, Hq, D] and LSE [B, Hq, Nq] that the kernel's roundings explain.

    Scores: products of fp16-exact operands added in fp32, then three multiplications and the subtraction of
    the maximum, each at most 2^-24 of mass = max_j scale sum_d |q_d K_jd|: ds <= (D + 8) 2^-24 mass (the tensor
    core truncates: twice that), and 2^x adds 2^-22.  p has a relative error of at most 2 ds + 2^-21 (weight and
    sum).  Weights are rounded to fp16: 2^-11 of each, or 2^-25 of the unit (the largest contribution `top`, in
    values) where they are subnormal; sums of `keys` terms in fp32 add keys 2^-24 / 16 (16 lanes of partial
    sums).  Then one rounding to the output type.
    """
    ds = 2 * (D + 8) * 2.0 ** -24 * mass
    rel = 2 * ds + 2.0 ** -20 + keys * 2.0 ** -24
    step = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[out]
    r = np.swapaxes(rel, 1, 2)[..., None]
    t = np.swapaxes(top, 1, 2)[..., None]
    tol = spread * (2.0 ** -11 + r) + keys * 2.0 ** -25 * oracle.kv8.QMAX[kind] * t
    tol = tol + (np.abs(o) + tol) * step + (2.0 ** -25 if out == "fp16" else 2.0 ** -126)
    return tol, ds + 2.0 ** -20 + keys * 2.0 ** -24
