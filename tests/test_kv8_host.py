"""The paged 8-bit cache and the page operations without a GPU: refusals at the C boundary (before any
device is touched), refusals of the helpers, and pins of their oracle."""
import ctypes
import math

import numpy as np
import pytest

import exact_tiled_attention_47_b200 as fa
import oracle
from exact_tiled_attention_47_b200 import build as fabuild

torch = pytest.importorskip("torch")

A = 0x100000  # a 16-byte aligned fake address (never dereferenced: every case fails validation)


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa._lib.load()


def _append(lib, k=A, kp=A, ks=A, table=A, sl=A, new=None, B=2, Nt=4, Hkv=2, pages=8, page=16, pps=4, D=64, dt=0, kv=3):
    return lib.fa_kv8_append(k, A, kp, A, ks, A, table, sl, new, B, Nt, Hkv, pages, page, pps, D, None, dt, kv)


def test_append_refusals(lib):
    for name in ("k", "kp", "ks", "table", "sl"):
        assert _append(lib, **{name: None}) == fa.FA_ERR_NULL, name
    assert _append(lib, dt=2) == fa.FA_ERR_DTYPE
    assert _append(lib, dt=3) == fa.FA_ERR_DTYPE
    for kv in (0, 1, 2, 5, -1):
        assert _append(lib, kv=kv) == fa.FA_ERR_DTYPE
    assert _append(lib, D=96) == fa.FA_ERR_HEADDIM
    for bad in (dict(B=0), dict(B=65536), dict(Nt=0), dict(Hkv=0), dict(pages=0), dict(page=8), dict(page=48), dict(page=1 << 17),
                dict(pps=0), dict(pps=(1 << 26) + 1), dict(B=65535, pps=1 << 16), dict(pages=1 << 30, page=1 << 12)):
        assert _append(lib, **bad) == fa.FA_ERR_SHAPE, bad
    for name, off in (("k", 8), ("kp", 8), ("ks", 2), ("table", 2), ("sl", 2), ("new", 2)):
        assert _append(lib, **{name: A + off}) == fa.FA_ERR_ALIGN, name


def _attend(lib, q=A, kp=A, vs=A, table=A, o=A, lse=A, B=2, Nq=1, Hq=8, Hkv=2, pages=8, page=16, pps=4, D=128, scale=0.1, sl=A, ws=A,
            wsb=1 << 24, dt=0, kv=3, od=0):
    return lib.fa_kv8_attend(q, kp, A, A, vs, table, o, lse, B, Nq, Hq, Hkv, pages, page, pps, D, scale, sl, ws, wsb, None, dt, kv, od)


def test_attend_refusals(lib):
    for name in ("q", "kp", "vs", "table", "o", "lse"):
        assert _attend(lib, **{name: None}) == fa.FA_ERR_NULL, name
    assert _attend(lib, dt=2, od=2) == fa.FA_ERR_DTYPE
    assert _attend(lib, od=1) == fa.FA_ERR_DTYPE
    assert _attend(lib, kv=0) == fa.FA_ERR_DTYPE
    assert _attend(lib, D=80) == fa.FA_ERR_HEADDIM
    for bad in (dict(Nq=0), dict(Nq=(1 << 24) + 1), dict(Hkv=3), dict(Hq=2, Hkv=4), dict(Hq=0), dict(B=0), dict(page=24), dict(scale=0.0),
                dict(scale=math.inf), dict(B=60000, Nq=1 << 20), dict(pps=(1 << 26) + 1)):
        assert _attend(lib, **bad) == fa.FA_ERR_SHAPE, bad
    for name, off in (("q", 8), ("kp", 8), ("vs", 2), ("table", 2), ("o", 8), ("lse", 2), ("sl", 2), ("ws", 8)):
        assert _attend(lib, **{name: A + off}) == fa.FA_ERR_ALIGN, name
    need = fa.fa_kv8_attend_workspace_bytes(2, 1, 8, 2, 128)
    assert need > 0 and _attend(lib, wsb=need - 1) == fa.FA_ERR_WORKSPACE
    assert _attend(lib, ws=None) == fa.FA_ERR_WORKSPACE
    for bad in ((0, 1, 8, 2, 128), (2, 0, 8, 2, 128), (2, 1, 8, 3, 128), (2, 1, 8, 0, 128), (2, 1, 8, 2, 96)):
        assert fa.fa_kv8_attend_workspace_bytes(*bad) == 0


def _state(table=A, lens=A, refs=A):
    return table, lens, refs


def test_pages_refusals(lib):
    need = fa.fa_pages_workspace_bytes(4, 8, 32)
    assert need > 0
    for bad in ((0, 8, 32), (4, 0, 32), (4, 8, 0), ((1 << 20) + 1, 8, 32)):
        assert fa.fa_pages_workspace_bytes(*bad) == 0
    pools, sizes = (ctypes.c_void_p * 2)(A, A), (ctypes.c_size_t * 2)(64, 64)

    def extend(table=A, lens=A, refs=A, slots=A, add=A, n=4, S=8, pps=4, pages=32, page=16, ws=A, wsb=need):
        return lib.fa_pages_extend(table, lens, refs, slots, add, n, S, pps, pages, page, ws, wsb, None)

    def fork(src=A, dst=A, pools=pools, sizes=sizes, n_pools=2, wsb=need, n=4, table=A):
        return lib.fa_pages_fork(table, A, A, src, dst, n, 8, 4, 32, 16, pools, sizes, n_pools, A, wsb, None)

    def free(slots=A, n=4, page=16):
        return lib.fa_pages_free(A, A, A, slots, n, 8, 4, 32, page, None)

    def compact(out=A, remap=A, n_live=A, pools=pools, sizes=sizes, n_pools=2, wsb=1 << 20, ws=A):
        return lib.fa_pages_compact(A, A, A, out, A, remap, n_live, 8, 4, 32, 16, pools, sizes, n_pools, ws, wsb, None)

    def copy(a=pools, b=pools, sizes=sizes, n_pools=2, src=A, n=4, pages=32, wsb=1 << 20):
        return lib.fa_pages_copy(a, b, sizes, n_pools, src, A, n, pages, 32, A, wsb, None)

    for name in ("table", "lens", "refs", "add"):
        assert extend(**{name: None}) == fa.FA_ERR_NULL
    assert extend(slots=None, n=9) == fa.FA_ERR_SHAPE
    for bad in (dict(n=0), dict(S=0), dict(pps=0), dict(pages=0), dict(page=20), dict(S=1 << 20, pps=1 << 12)):
        assert extend(**bad) == fa.FA_ERR_SHAPE, bad
    assert extend(add=A + 2) == fa.FA_ERR_ALIGN
    assert extend(ws=A + 8) == fa.FA_ERR_ALIGN
    assert extend(wsb=need - 1) == fa.FA_ERR_WORKSPACE
    assert extend(ws=None) == fa.FA_ERR_WORKSPACE
    assert fork(src=None) == fa.FA_ERR_NULL
    assert fork(pools=None) == fa.FA_ERR_NULL
    assert fork(pools=(ctypes.c_void_p * 2)(A, None)) == fa.FA_ERR_NULL
    assert fork(pools=(ctypes.c_void_p * 2)(A, A + 2)) == fa.FA_ERR_ALIGN
    assert fork(sizes=(ctypes.c_size_t * 2)(64, 66)) == fa.FA_ERR_ALIGN
    assert fork(sizes=(ctypes.c_size_t * 2)(64, 0)) == fa.FA_ERR_SHAPE
    assert fork(n_pools=-1) == fa.FA_ERR_SHAPE
    assert fork(wsb=16) == fa.FA_ERR_WORKSPACE
    assert free(slots=None) == fa.FA_ERR_NULL
    assert free(n=0) == fa.FA_ERR_SHAPE
    assert free(page=4) == fa.FA_ERR_SHAPE
    assert compact(remap=None) == fa.FA_ERR_NULL
    assert compact(n_live=None) == fa.FA_ERR_NULL
    assert compact(out=A + 1) == fa.FA_ERR_ALIGN
    assert compact(ws=None) == fa.FA_ERR_WORKSPACE
    assert copy(src=None) == fa.FA_ERR_NULL
    assert copy(n_pools=0) == fa.FA_ERR_SHAPE
    assert copy(pages=0) == fa.FA_ERR_SHAPE
    assert copy(wsb=16) == fa.FA_ERR_WORKSPACE


def test_helpers_refuse_what_is_not_on_a_gpu_or_not_alike():
    kp = torch.zeros((4, 2, 16, 64), dtype=torch.int8)
    ks = torch.zeros((4, 2, 1))
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros((1, 1, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.attend_kv8(q, kp, kp, ks, ks, table, lens)
    with pytest.raises(ValueError, match="k_pages"):
        fa.attend_kv8(q, kp.to(torch.uint8), kp, ks, ks, table, lens)
    with pytest.raises(ValueError, match="v_pages"):
        fa.attend_kv8(q, kp, kp.view(torch.float8_e4m3fn), ks, ks, table, lens)
    with pytest.raises(ValueError, match="k_scales"):
        fa.attend_kv8(q, kp, kp, ks.double(), ks, table, lens)
    with pytest.raises(ValueError, match="block_table"):
        fa.attend_kv8(q, kp, kp, ks, ks, table.long(), lens)
    with pytest.raises(ValueError, match="block_table"):
        fa.attend_kv8(q, kp, kp, ks, ks, torch.zeros((1, 4), dtype=torch.int32)[:, ::2], lens)
    with pytest.raises(ValueError, match="seqlens_k"):
        fa.attend_kv8(q, kp, kp, ks, ks, table, torch.ones(2, dtype=torch.int32))
    k = torch.zeros((1, 3, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="alike"):
        fa.append_kv8(k, k.bfloat16(), kp, kp, ks, ks, table, lens)
    with pytest.raises(ValueError, match="heads"):
        fa.append_kv8(k[:, :, :1], k[:, :, :1], kp, kp, ks, ks, table, lens)
    with pytest.raises(ValueError, match="seqlens_k"):
        fa.append_kv8(k, k, kp, kp, ks, ks, table, None)
    with pytest.raises(ValueError, match="new_lens"):
        fa.append_kv8(k, k, kp, kp, ks, ks, table, lens, new_lens=lens.long())
    refs = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="add"):
        fa.extend_pages(table, lens, refs, 16, lens.long())
    with pytest.raises(ValueError, match="dst"):
        fa.fork_pages(table, lens, refs, 16, lens, torch.zeros(2, dtype=torch.int32), [kp])
    with pytest.raises(ValueError, match="pools"):
        fa.fork_pages(table, lens, refs, 16, lens, lens, [kp[:3]])
    with pytest.raises(ValueError, match="CUDA"):
        fa.free_pages(table, lens, refs, 16, lens)
    with pytest.raises(ValueError, match="unlike"):
        fa.copy_pages([kp], [kp[:, :1].contiguous()], lens, lens)


# ---- pins of the oracle ------------------------------------------------------------------------


def test_codes_agree_with_torch():
    bits = torch.arange(256, dtype=torch.uint8)
    mine, ref = oracle.kv8.E4M3, bits.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(mine), np.isnan(ref)) and np.array_equal(mine[~np.isnan(ref)], ref[~np.isnan(ref)])
    y = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * np.exp2(np.random.default_rng(1).integers(-12, 8, 20000)).astype(np.float32)
    y = np.clip(np.concatenate([y, mine[:127].astype(np.float32), (mine[1:127] + mine[:126]).astype(np.float32) / 2]), -448, 448)
    assert np.array_equal(oracle.kv8.encode(y, "e4m3"), torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_block_scale_is_the_smallest_power(kind):
    rng = np.random.default_rng(2)
    q = oracle.kv8.QMAX[kind]
    for top in [0.0, 1e-45, 2.0 ** -133, q, q * 2.0 ** -5, np.nextafter(q, 1e9), 3.4e38, *np.exp(rng.uniform(-80, 80, 200))]:
        s = oracle.kv8.block_scale(float(top), kind)
        assert math.frexp(s)[0] == 0.5 and s >= 2.0 ** -126 and top <= q * s
        assert s == 2.0 ** -126 or top > q * s / 2


def test_attend_is_attention_over_the_values():
    from kv8_cases import make_cache
    rng = np.random.default_rng(3)
    lens = [40, 3, 0]
    kp, vp, ks, vs, table = make_cache(rng, lens, 2, 64, 16, "e4m3")
    q = rng.standard_normal((3, 4, 4, 64))
    o, lse, *_ = oracle.kv8.attend(q, kp, vp, ks, vs, table, lens, 16, 0.2, "e4m3")
    for b, n in enumerate(lens):
        for h in range(4):
            K = oracle.kv8.rows(kp, ks, table[b], n, 16, h // 2, "e4m3")
            V = oracle.kv8.rows(vp, vs, table[b], n, 16, h // 2, "e4m3")
            if n == 0:
                assert not o[b, :, h].any() and np.all(lse[b, h] == -np.inf)
                continue
            ro, rl = oracle.attention_head(q[b, :, h], K, V, 0.2, causal=True)
            assert np.allclose(o[b, :, h], ro, rtol=1e-12, atol=1e-14) and np.array_equal(np.isinf(lse[b, h]), np.isinf(rl))
            assert np.allclose(lse[b, h][~np.isinf(rl)], rl[~np.isinf(rl)], rtol=1e-12)


def test_append_row_by_row_keeps_the_values_near():
    # sixteen single appends with growing magnitudes: every row stays within half a step of the block's final
    # scale for each time the scale grew (e4m3: requantisation by powers of two is exact above the subnormals)
    rng = np.random.default_rng(4)
    x = rng.standard_normal((1, 16, 1, 64)) * np.exp2(np.arange(16) / 3)[None, :, None, None]
    for kind in ("e4m3", "int8"):
        pages, scales = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1, 1))
        for n in range(1, 17):
            pages, scales, odd = oracle.kv8.append(x[:, n - 1:n], pages, scales, np.zeros((1, 1), np.int32), [n], [1], 16, kind)
            assert not odd
        got = oracle.kv8.decode(pages[0, 0], kind) * scales[0, 0, 0]
        err = np.abs(got - x[0, :, 0])
        if kind == "e4m3":
            assert np.all(err <= np.abs(x[0, :, 0]) * 2.0 ** -4 + scales[0, 0, 0] * 2.0 ** -9)
        else:
            assert np.all(err <= scales[0, 0, 0] * 1.0)  # half a step of the last scale, a quarter of the one before, ...


def test_page_oracle_keeps_counts():
    rng = np.random.default_rng(5)
    S, pps, P, page = 6, 5, 20, 16
    table, lens, refs = np.full((S, pps), -1, np.int32), np.zeros(S, np.int32), np.zeros(P, np.int32)
    pool = rng.integers(0, 99, (P, 3))

    def counted():
        want = np.zeros(P, int)
        for s in range(S):
            for c in range(-(-lens[s] // page)):
                want[table[s, c]] += 1
        return np.array_equal(want, refs)

    assert oracle.pages.extend(table, lens, refs, page, [3, 0], [33, 16]) and counted()
    assert list(table[3, :3]) == [0, 1, 2] and table[0, 0] == 3
    assert oracle.pages.fork(table, lens, refs, page, [3, 3], [1, 5], [pool]) and counted()
    assert refs[0] == 3 and refs[2] == 1 and np.array_equal(pool[table[5, 2]], pool[2])
    assert not oracle.pages.fork(table, lens, refs, page, [3], [1], [pool])
    assert not oracle.pages.extend(table, lens, refs, page, [0, 0], [1, 1])
    oracle.pages.free(table, lens, refs, page, [3, 0])
    assert counted()
    before = {s: [pool[p].copy() for p in table[s, : -(-lens[s] // page)]] for s in range(S)}
    table, refs, remap, n = oracle.pages.compact(table, lens, refs, page, [pool])
    assert counted() and n == 4 and not refs[n:].any() and (refs[:n] > 0).all()
    assert all(np.array_equal(pool[p], x) for s in range(S) for p, x in zip(table[s], before[s]))
