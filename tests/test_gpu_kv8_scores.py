"""Attention over the 8-bit cache where scores are large, far apart, or not numbers.

All caches here are one sequence and one KV head on pages in order, so that the right answer can be written down: both
kernels, with units that lie in one share (up to 1024 keys of table for the first, 512 for the second) and cut ones.
"""
import math

import numpy as np
import pytest

import oracle
from test_gpu_kv8 import CODE, codes_to

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D, PAGE = 64, 16
# keys, tokens, heads of a group: first kernel whole, cut, cut into many pieces; tcgen05 kernel whole, cut
CASES = [(600, 1, 4), (5000, 3, 12), (40000, 1, 3), (400, 100, 2), (3000, 150, 2)]
IDS = [f"n{n}q{q}g{g}" for n, q, g in CASES]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_47_b200 import build
    build.build()
    import exact_tiled_attention_47_b200 as fa
    fa.fa_device_status(clear=True)
    yield
    assert fa.fa_device_status(clear=True) == 0


def attend(q, k, v, ks, vs, kind, scale=None):
    """O [Nq, G, D], LSE [G, Nq] in fp64 from values k, v [n, D] that codes hold exactly, one scale per 16 of them."""
    import exact_tiled_attention_47_b200 as fa
    n = len(k)
    pages = -(-n // PAGE)

    def pool(x):
        full = np.zeros((pages * PAGE, D))
        full[:n] = x
        codes = oracle.kv8.encode(full, kind)
        assert np.array_equal(oracle.kv8.decode(codes, kind)[:n], x)
        return codes_to(codes.reshape(pages, 1, PAGE, D), kind)

    def scales(x):
        return torch.from_numpy(np.broadcast_to(x, pages).astype(np.float32).reshape(pages, 1, 1)).cuda()

    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    o, lse = fa.attend_kv8(q.cuda()[None], pool(k), pool(v), scales(ks), scales(vs), table, lens, scale=scale, out_dtype=torch.float32)
    return o[0].double().cpu().numpy(), lse[0].double().cpu().numpy()


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("kind", list(CODE))
@pytest.mark.parametrize("score", [1e3, 1e5, 1e6, 5e7])
def test_one_key_far_ahead_at_large_scores(case, kind, score):
    # Key 5 has the score given, every other one half of it: the softmax is 1 at key 5 and 0 elsewhere, so O is that key's
    # value.  Its weight is off by 2^-11 (rounded to fp16) and by the exponentials and the merges (2^-22 each, a handful,
    # below 2^-18 in all), O once more by its rounding to fp32; nothing of it grows with the score.  The LSE is the score:
    # six roundings or constants of 2^-24 relative, 2^-21 with room.
    n, Nq, G = case
    rng = np.random.default_rng(n)
    k = np.zeros((n, D))
    k[:, 0], k[5, 0] = 60.0, 120.0
    v = rng.integers(1, 8, (n, D)).astype(np.float64)
    q = torch.zeros((Nq, G, D), dtype=torch.float16)
    q[..., 0] = 1.0
    scale = float(np.float32(score / 120.0 * 1.0314159))
    o, lse = attend(q, k, v, 1.0, 0.37, kind, scale)
    want = v[5] * float(np.float32(0.37))
    assert np.all(np.abs(o - want) <= want * (2.0 ** -11 + 2.0 ** -18)), np.abs(o / want - 1).max()
    assert np.all(np.abs(lse - 120.0 * scale) <= 2.0 ** -21 * 120.0 * scale)


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("kind", list(CODE))
@pytest.mark.parametrize("gap", [18.0, 20.0])
def test_small_keys_beside_large_ones_of_no_value(case, kind, gap):
    # Keys 3, 19, 35 and 51 (one in each of the first four blocks, so every warp that starts there meets one) are `gap` ahead
    # and have V = 0: all of O is what the others add, each with exp(-gap) of the weight (2^-26 and 2^-28.9).
    # Off by: 2^-11 where a weight is a normal fp16 number; else at most 2^-32 of the largest contribution (in values: qmax
    # times the scale times that key's share) for each key; 2^-20 + keys 2^-24 for exponentials and fp32 sums, 2 ds for
    # scores off by ds = 2 (D + 8) 2^-24 gap; then the rounding to fp32.
    n, Nq, G = case
    rng = np.random.default_rng(n + 1)
    qmax = oracle.kv8.QMAX[kind]
    k = np.zeros((n, D))
    v = rng.integers(14, 29, (n, D)) * 16.0 if kind == "e4m3" else rng.integers(64, 128, (n, D)) * 1.0
    v = oracle.kv8.decode(oracle.kv8.encode(v, kind), kind)
    big = [3, 19, 35, 51]
    k[big, 0], v[big] = gap, 0.0
    q = torch.zeros((Nq, G, D), dtype=torch.float16)
    q[..., 0] = 8.0
    o, lse = attend(q, k, v, 1.0, 1.0, kind, 0.125)
    for i in range(Nq):
        s = k[: n - Nq + i + 1, 0]
        p = np.exp(s - s.max())
        total = p.sum()
        want = (p / total) @ v[: len(p)]
        rel = 2.0 ** -11 + 2.0 ** -20 + n * 2.0 ** -24 + 4 * (D + 8) * 2.0 ** -24 * gap
        tol = want * (rel + 2.0 ** -24) + n * 2.0 ** -32 * qmax / total
        assert np.all(np.abs(o[i] - want) <= tol), (i, np.abs(o[i] / want - 1).max())
        assert np.all(np.abs(lse[:, i] - (gap + math.log(total))) <= 2 * (D + 8) * 2.0 ** -24 * gap + 2.0 ** -20 + n * 2.0 ** -24)


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_nan_in_a_query_stays_in_its_row(case, dtype):
    n, Nq, G = case
    rng = np.random.default_rng(n + 2)
    k, v = (rng.integers(-7, 8, (n, D)).astype(np.float64) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((Nq, G, D)) * 0.2).to(dtype)
    clean_o, clean_lse = attend(q, k, v, 1.0, 1.0, "int8")
    rows = [(0, 0), (Nq - 1, G - 1)]
    for i, g in rows:
        q[i, g, 5 + i % 50] = math.nan
    o, lse = attend(q, k, v, 1.0, 1.0, "int8")
    for i, g in rows:
        assert np.isnan(o[i, g]).all() and np.isnan(lse[g, i]), (i, g, lse[g, i])
        o[i, g], lse[g, i] = clean_o[i, g], clean_lse[g, i]
    assert np.array_equal(o, clean_o) and np.array_equal(lse, clean_lse)


@pytest.mark.parametrize("n,Nq,G", [(3, 5, 4), (40, 200, 2)])
def test_a_nan_in_a_query_that_sees_no_key(n, Nq, G):
    q = torch.full((Nq, G, D), math.nan, dtype=torch.bfloat16)
    o, lse = attend(q, np.ones((n, D)), np.ones((n, D)), 1.0, 1.0, "e4m3")
    dead = Nq - n
    assert not o[:dead].any() and np.isneginf(lse[:, :dead]).all()
    assert np.isnan(o[dead:]).all() and np.isnan(lse[:, dead:]).all()


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_v_scales_of_zero_stand_for_zeros(case):
    # codes under a scale of zero: 0 exactly where there is nothing else, and as if the codes were zeros beside other blocks
    n, Nq, G = case
    rng = np.random.default_rng(n + 3)
    k, v = (rng.integers(-7, 8, (n, D)).astype(np.float64) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((Nq, G, D)) * 0.2).to(torch.bfloat16)
    o, lse = attend(q, k, v, 1.0, 0.0, "int8")
    same_o, same_lse = attend(q, k, np.zeros((n, D)), 1.0, 1.0, "int8")
    assert not o.any() and not same_o.any()
    assert np.all(np.abs(lse - same_lse) <= 2.0 ** -20 + n * 2.0 ** -24)  # (the sums may be added up in another way)
    some = np.arange(-(-n // 16)) % 3 > 0
    o, lse = attend(q, k, v, 1.0, np.where(some, 1.0, 0.0), "int8")
    want, want_lse = attend(q, k, v * np.repeat(some, 16)[:n, None], 1.0, 1.0, "int8")
    # two roundings of each weight to fp16 (2^-11 of the values added up, or 2^-32 of the largest) apart
    p = 2.0 ** -10 * np.abs(v).max() + n * 2.0 ** -31 * 7
    assert np.all(np.abs(o - want) <= p) and np.all(np.abs(lse - want_lse) <= 2.0 ** -20 + n * 2.0 ** -24)


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("score", [1e5, 1e6, 5e7])
def test_one_key_far_ahead_beside_blocks_of_small_values(case, score):
    # as test_one_key_far_ahead_at_large_scores, with V scales of 2^-100 in every other block (what an append of zeros leaves)
    n, Nq, G = case
    rng = np.random.default_rng(n)
    k = np.zeros((n, D))
    k[:, 0], k[5, 0] = 60.0, 120.0
    v = rng.integers(1, 8, (n, D)).astype(np.float64)
    q = torch.zeros((Nq, G, D), dtype=torch.float16)
    q[..., 0] = 1.0
    scale = float(np.float32(score / 120.0 * 1.0314159))
    o, lse = attend(q, k, v, 1.0, np.where(np.arange(-(-n // 16)) % 2, 2.0 ** -100, 0.37), "int8", scale)
    want = v[5] * float(np.float32(0.37))
    assert np.all(np.abs(o - want) <= want * (2.0 ** -11 + 2.0 ** -18)), np.abs(o / want - 1).max()
    assert np.all(np.abs(lse - 120.0 * scale) <= 2.0 ** -21 * 120.0 * scale)


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("step", [0.3, 5.0, 5.6, 40.0, -5.0])  # nats from one block to the next; the lazy maxima move from 5.5 on
@pytest.mark.parametrize("values", ["even", "rising", "falling", "mixed"])
def test_scores_and_scales_that_climb(case, step, values):
    # K has the same codes everywhere and a scale that grows from block to block, so scores climb by `step`; V scales stay, climb
    # or fall by 2^3 a block (for 40 blocks, then again), or jump about: both maxima are raised late, early and apart.
    n, Nq, G = case
    rng = np.random.default_rng(n + 4)
    blocks = -(-n // 16)
    at = np.arange(blocks)
    ks = np.abs(step) / 8 * (at % 50 + 1 if step > 0 else 50 - at % 50)
    vs = {"even": np.ones(blocks), "rising": 2.0 ** (3 * (at % 40) - 60), "falling": 2.0 ** (60 - 3 * (at % 40)),
          "mixed": 2.0 ** rng.integers(-40, 40, blocks)}[values]
    ks = ks.astype(np.float32).astype(np.float64)
    k = np.zeros((n, D))
    k[:, 0] = 8.0 + rng.integers(0, 2, n)
    v = rng.integers(-7, 8, (n, D)).astype(np.float64)
    q = torch.zeros((Nq, G, D), dtype=torch.bfloat16)
    q[..., 0] = torch.arange(1, G + 1) / 4
    scale = 4.0 / G
    o, lse = attend(q, k, v, ks, vs, "int8", scale)
    per_key_k, per_key_v = np.repeat(ks, 16)[:n], np.repeat(vs, 16)[:n]
    for i in sorted({0, Nq // 2, Nq - 1}):
        vis = n - Nq + i + 1
        for g in range(G):
            s = np.float64(np.float32(scale)) * (g + 1) / 4 * (k[:vis, 0] * per_key_k[:vis])
            p = np.exp(s - s.max())
            total = p.sum()
            p /= total
            V = v[:vis] * per_key_v[:vis, None]
            want, spread = p @ V, p @ np.abs(V)
            ds = 16 * 2.0 ** -24 * s.max()  # one product and a handful of roundings at the size of the score
            rel = 2.0 ** -11 + 2 * ds + 2.0 ** -18 + n * 2.0 ** -24
            tol = spread * rel + n * 2.0 ** -32 * 7 * (p * per_key_v[:vis]).max() + np.abs(want) * 2.0 ** -23
            assert np.all(np.abs(o[i, g] - want) <= tol), (i, g, (np.abs(o[i, g] - want) / tol).max())
            assert abs(lse[g, i] - (s.max() + math.log(total))) <= ds + 2.0 ** -18 + n * 2.0 ** -24
