"""The paged 8-bit cache on the GPU: append bit for bit against the oracle, attention against fp64 within the
bounds its roundings explain (kv8_cases.bounds), and both together as a serving loop uses them."""
import math

import numpy as np
import pytest

import oracle
from kv8_cases import bounds, make_cache

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FLOAT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


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


def codes_to(x, kind):
    return torch.from_numpy(x).cuda().view(CODE[kind])


def to_gpu(cache, kind):
    kp, vp, ks, vs, table = cache
    return [codes_to(kp, kind), codes_to(vp, kind), *(torch.from_numpy(x).cuda() for x in (ks, vs, table))]


def rounded(rng, shape, dtype, scale=1.0):
    """Random values that the type holds exactly: (the tensor on the device, the values in fp64)."""
    t = torch.from_numpy(rng.standard_normal(shape) * scale).to(FLOAT[dtype])
    return t.cuda(), t.double().numpy()


def check_attend(seed, lens, Nq, Hkv, G, D, page, kind, dtype, out, scales="powers", q_scale=1.0):
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(seed)
    cache = make_cache(rng, lens, Hkv, D, page, kind, scales=scales)
    q, qv = rounded(rng, (len(lens), Nq, Hkv * G, D), dtype, q_scale)
    kp, vp, ks, vs, table = to_gpu(cache, kind)
    o, lse = fa.attend_kv8(q, kp, vp, ks, vs, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out_dtype=FLOAT[out])
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == 0
    ro, rl, spread, mass, top = oracle.kv8.attend(qv, *cache[:4], cache[4], lens, page, 1 / math.sqrt(D), kind)
    tol, ltol = bounds(ro, spread, mass, top, max(lens), D, kind, out)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all()
    dead = np.isinf(rl)
    assert np.array_equal(np.isneginf(lse), dead)
    assert not o[np.swapaxes(dead, 1, 2)].any()
    assert np.all(np.abs(lse[~dead] - rl[~dead]) <= ltol[~dead] + 2.0 ** -23 * np.abs(rl[~dead])), np.abs(lse[~dead] - rl[~dead]).max()
    assert np.all(np.abs(o - ro) <= tol), (np.abs(o - ro) / tol).max()
    return o, lse


ATTEND = [
    # lens, Nq, Hkv, G, D, page, codes, dtype, out
    ([37, 0, 1], 1, 2, 4, 64, 16, "e4m3", "bf16", "bf16"),
    ([1, 1000], 1, 1, 1, 128, 16, "int8", "fp16", "fp16"),
    ([16, 15, 17, 64], 1, 3, 5, 64, 32, "int8", "bf16", "fp32"),
    ([2049, 3, 300], 5, 4, 7, 128, 32, "int8", "fp16", "fp16"),      # a length below Nq: rows without keys
    ([777], 1, 2, 16, 128, 64, "e4m3", "fp16", "fp32"),
    ([515, 4, 129], 3, 1, 24, 64, 256, "e4m3", "bf16", "fp32"),       # 72 rows, group above one tile
    ([130, 200], 2, 2, 9, 128, 128, "e4m3", "bf16", "bf16"),
    ([300, 17, 0], 130, 1, 8, 128, 16, "e4m3", "bf16", "fp32"),       # chunk longer than a sequence
    ([260, 1100], 70, 2, 3, 64, 64, "int8", "fp16", "fp32"),
    ([513], 513, 2, 2, 128, 32, "e4m3", "fp16", "fp16"),              # a whole prompt, causal from the first key
    ([400, 300], 129, 1, 1, 64, 16, "int8", "bf16", "bf16"),          # one head: rows end one behind a tile
    ([9000, 20], 1, 1, 8, 128, 16, "e4m3", "bf16", "fp32"),
]


@pytest.mark.parametrize("case", ATTEND, ids=[f"n{max(c[0])}q{c[1]}h{c[2]}x{c[3]}d{c[4]}p{c[5]}{c[6]}{c[7]}" for c in ATTEND])
@pytest.mark.parametrize("scales", ["powers", "any"])
def test_attend(case, scales):
    check_attend(100 + len(case[0]) + case[1], *case, scales=scales)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("Nq", [1, 6, 150])
def test_attend_scales_far_apart(kind, Nq):
    # V scales from 2^-60 to 2^60 (and zeros) from block to block: the weights keep their precision
    check_attend(300 + Nq, [700, 33], Nq, 2, 4, 128, 32, kind, "bf16", "fp32", scales="wild")


@pytest.mark.parametrize("q_scale", [1e-30, 1e3, 1e20])
def test_attend_queries_outside_the_range_of_fp16(q_scale):
    # bf16 queries are scaled by powers of two on their way to fp16; scores of 1e3 and more are near one-hot
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(7)
    lens = [200]
    cache = make_cache(rng, lens, 1, 64, 16, "e4m3")
    q, qv = rounded(rng, (1, 2, 4, 64), "bf16", q_scale)
    kp, vp, ks, vs, table = to_gpu(cache, "e4m3")
    scale = 1 / (8 * q_scale)
    o, lse = fa.attend_kv8(q, kp, vp, ks, vs, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=scale, out_dtype=torch.float32)
    ro, rl, spread, mass, top = oracle.kv8.attend(qv, *cache, lens, 16, np.float64(np.float32(scale)), "e4m3")
    tol, ltol = bounds(ro, spread, mass, top, 200, 64, "e4m3", "fp32")
    assert np.all(np.abs(o.double().cpu().numpy() - ro) <= tol)
    assert np.all(np.abs(lse.double().cpu().numpy() - rl) <= ltol + 2.0 ** -23 * np.abs(rl))


def test_attend_without_lengths_uses_the_whole_table():
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(8)
    lens = [96, 96]
    cache = make_cache(rng, lens, 2, 128, 32, "int8", cols=0)
    q, _ = rounded(rng, (2, 1, 8, 128), "bf16")
    g = to_gpu(cache, "int8")
    a = fa.attend_kv8(q, *g, None)
    b = fa.attend_kv8(q, *g, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attend_is_the_same_each_time_and_with_a_dirty_workspace():
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(9)
    lens = [3000, 1, 0, 555]
    cache = make_cache(rng, lens, 2, 128, 16, "e4m3")
    q, _ = rounded(rng, (4, 1, 16, 128), "bf16")
    g, sl = to_gpu(cache, "e4m3"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    n = fa.fa_kv8_attend_workspace_bytes(4, 1, 16, 2, 128)
    ws = [torch.full((n,), x, dtype=torch.uint8, device="cuda") for x in (0, 255, 0x7F)]
    outs = [fa.attend_kv8(q, *g, sl, workspace=w) for w in ws]
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_attend_shared_pages():
    # two sequences whose tables name the same pages see the same keys
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(10)
    cache = make_cache(rng, [200, 0], 2, 64, 16, "e4m3")
    g = to_gpu(cache, "e4m3")
    g[4][1] = g[4][0]
    q, _ = rounded(rng, (1, 1, 4, 64), "fp16")
    o, lse = fa.attend_kv8(q.expand(2, -1, -1, -1), *g, torch.tensor([200, 200], dtype=torch.int32, device="cuda"))
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])


def test_attend_reports_bad_lengths_and_tables():
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(11)
    lens = [100, 100, 100]
    cache = make_cache(rng, lens, 1, 64, 16, "int8")
    g = to_gpu(cache, "int8")
    q, _ = rounded(rng, (3, 1, 2, 64), "bf16")
    good, _ = fa.attend_kv8(q, *g, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    cap = cache[4].shape[1] * 16
    o, lse = fa.attend_kv8(q, *g, torch.tensor([100, cap + 1, -1], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_CU_SEQLENS
    assert torch.equal(o[0], good[0]) and not o[1:].any() and torch.isneginf(lse[1:]).all()
    bad = g[4].clone()
    bad[1, 2], bad[2, 0] = cache[0].shape[0], -3
    o, _ = fa.attend_kv8(q, *g[:4], bad, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_PAGE_TABLE
    assert torch.equal(o[0], good[0])


@pytest.mark.parametrize("Nq", [1, 100])
def test_attend_on_two_streams_and_in_a_graph(Nq):
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(12)
    lens = [1500, 640]
    cache = make_cache(rng, lens, 2, 128, 16, "e4m3")
    g, sl = to_gpu(cache, "e4m3"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = [rounded(rng, (2, Nq, 8, 128), "bf16")[0] for _ in range(2)]
    want = [fa.attend_kv8(q, *g, sl) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [fa.attend_kv8(q, *g, sl, stream=s) for _ in range(4) for q, s in zip(qs, streams)]
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
    graph = torch.cuda.CUDAGraph()
    q = qs[0].clone()
    with torch.cuda.graph(graph):
        o, lse = fa.attend_kv8(q, *g, sl)
    for i in (1, 0):
        q.copy_(qs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


# ---- append ------------------------------------------------------------------------------------


def check_append(seed, before, new, Nt, Hkv, D, page, kind, dtype, values=None, scales="powers"):
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(seed)
    B = len(before)
    ends = [a + n for a, n in zip(before, new)]
    kp, vp, ks, vs, table = make_cache(rng, ends, Hkv, D, page, kind, scales=scales)
    k, kv = rounded(rng, (B, Nt, Hkv, D), dtype)
    v, vv = rounded(rng, (B, Nt, Hkv, D), dtype)
    if values is not None:
        for t, x in ((k, kv), (v, vv)):
            values(t, x)
    g = to_gpu((kp, vp, ks, vs, table), kind)
    fa.append_kv8(k, v, *g, torch.tensor(ends, dtype=torch.int32, device="cuda"), torch.tensor(new, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    odd = False
    for i, (x, codes, sc) in enumerate(((kv, kp, ks), (vv, vp, vs))):
        want, wscale, o = oracle.kv8.append(x, codes, sc, table, ends, new, page, kind)
        odd |= o
        got = g[i].view(torch.uint8).cpu().numpy()
        # -0 and 0 are the same e4m3 value
        same = (got == want) | ((kind == "e4m3") & ((got & 0x7F) == 0) & ((want & 0x7F) == 0))
        assert same.all(), (np.argwhere(~same)[:4], got[~same][:4], want[~same][:4])
        assert np.array_equal(g[2 + i].cpu().numpy(), wscale.astype(np.float32), equal_nan=True)
    assert fa.fa_device_status(clear=True) == (fa.FA_ERR_NONFINITE if odd else 0)


APPEND = [
    # before, new, Nt, Hkv, D, page, codes, dtype
    ([0], [1], 1, 1, 64, 16, "e4m3", "bf16"),
    ([31, 16, 15, 0], [1, 1, 1, 1], 1, 8, 128, 16, "e4m3", "bf16"),
    ([100, 7, 48], [5, 0, 7], 7, 5, 64, 32, "int8", "fp16"),
    ([0, 3], [200, 133], 200, 2, 128, 64, "e4m3", "fp16"),
    ([17], [17], 17, 3, 128, 256, "int8", "bf16"),
    ([9, 250], [33, 32], 33, 1, 64, 128, "int8", "fp16"),
]


@pytest.mark.parametrize("case", APPEND, ids=[f"n{max(c[1])}h{c[3]}d{c[4]}p{c[5]}{c[6]}{c[7]}" for c in APPEND])
def test_append(case):
    check_append(500 + case[2], *case)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_into_blocks_with_scales_of_any_kind(kind):
    check_append(600, [5, 40, 15], [3, 9, 1], 9, 2, 64, 16, kind, "bf16", scales="any")


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_edge_values(kind, dtype):
    top = {"bf16": 3.0e38, "fp16": 65504.0}[dtype]
    small = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24}[dtype]

    def values(t, x):
        x[0, 0], x[0, 1], x[0, 2] = 0.0, small, top  # a block of its own each: zeros, subnormals, the largest
        x[0, 3] = oracle.kv8.QMAX[kind]              # exactly on the border of a power of two
        x[0, 3, :, 0] = -oracle.kv8.QMAX[kind] / 3
        t.copy_(torch.from_numpy(x))
        x[...] = t.double().cpu().numpy()

    for start in range(4):  # row `start` alone in its block
        def one(t, x, start=start):
            values(t, x)
            x[0, 0] = x[0, start]
            t.copy_(torch.from_numpy(x))
        check_append(610 + start, [16], [1], 4, 2, 64, 16, kind, dtype, values=one)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_infinities_and_nan_are_reported(kind):
    def values(t, x):
        x[0, 0, 0, 3], x[0, 1, 0, 5], x[0, 2, 0, 7] = np.nan, np.inf, -np.inf
        t.copy_(torch.from_numpy(x))
    check_append(620, [4], [3], 3, 2, 64, 16, kind, "bf16", values=values)


def test_append_of_strided_rows_and_without_new_lens():
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(630)
    cache = make_cache(rng, [20, 36], 2, 64, 16, "e4m3")
    qkv, _ = rounded(rng, (2, 4, 8, 64), "bf16")
    sl = torch.tensor([20, 36], dtype=torch.int32, device="cuda")
    a, b = to_gpu(cache, "e4m3"), to_gpu(cache, "e4m3")
    fa.append_kv8(qkv[:, :, 4:6], qkv[:, :, 6:8], *a, sl)
    fa.append_kv8(qkv[:, :, 4:6].contiguous(), qkv[:, :, 6:8].contiguous(), *b, sl, torch.full((2,), 4, dtype=torch.int32, device="cuda"))
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.int8 if x.element_size() == 1 else torch.int32), y.view(torch.int8 if y.element_size() == 1 else torch.int32))


def test_append_reports_bad_lengths_and_tables():
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(640)
    cache = make_cache(rng, [40, 40, 40, 40], 1, 64, 16, "int8")
    g = to_gpu(cache, "int8")
    before = [t.clone() for t in g]
    x, _ = rounded(rng, (4, 3, 1, 64), "fp16")
    cap = cache[4].shape[1] * 16
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for lens, new in ((i32(2, cap + 1, -5, 40), i32(3, 1, 0, 4)), (i32(40, 40, 40, 40), i32(-1, 4, 5, -2))):
        fa.append_kv8(x, x, *g, lens, new)
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_CU_SEQLENS
        for a, b in zip(g[:2], before[:2]):
            assert torch.equal(a.view(torch.int8), b.view(torch.int8))
    g[4][0, 2], g[4][1, 2] = cache[0].shape[0], -1
    fa.append_kv8(x, x, *g, i32(40, 40, 40, 40), i32(3, 3, 0, 0))
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_PAGE_TABLE
    for a, b in zip(g[:2], before[:2]):
        assert torch.equal(a.view(torch.int8), b.view(torch.int8))


# ---- together ----------------------------------------------------------------------------------


@pytest.mark.parametrize("kind,dtype", [("e4m3", "bf16"), ("int8", "fp16")])
def test_serving_loop(kind, dtype):
    """Prompts, single tokens, a fork, a drafted window, a freed sequence and a compaction, all on the device:
    after every append the attention equals fp64 attention over what the oracle says the cache holds."""
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(700)
    S, page, Hkv, G, D, pages, pps = 4, 16, 2, 3, 64, 40, 8
    kp, vp, ks, vs = fa.new_kv8_cache(pages, page, Hkv, D, dtype=CODE[kind])
    table = torch.full((S, pps), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    h = dict(kp=np.zeros((pages, Hkv, page, D), np.uint8), ks=np.zeros((pages, Hkv, 1)), table=table.cpu().numpy(), lens=np.zeros(S, np.int32),
             refs=np.zeros(pages, np.int32))
    h["vp"], h["vs"] = h["kp"].copy(), h["ks"].copy()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def step(add, Nq):
        nonlocal table
        k, kv = rounded(rng, (S, max(add), Hkv, D), dtype)
        v, vv = rounded(rng, (S, max(add), Hkv, D), dtype, 0.3)
        fa.extend_pages(table, lens, refs, page, i32(add))
        assert oracle.pages.extend(h["table"], h["lens"], h["refs"], page, range(S), add)
        fa.append_kv8(k, v, kp, vp, ks, vs, table, lens, i32(add))
        for x, p, s in ((kv, "kp", "ks"), (vv, "vp", "vs")):
            h[p], h[s], _ = oracle.kv8.append(x, h[p], h[s], h["table"], h["lens"], add, page, kind)
        q, qv = rounded(rng, (S, Nq, Hkv * G, D), dtype)
        o, lse = fa.attend_kv8(q, kp, vp, ks, vs, table, lens, out_dtype=torch.float32)
        ro, rl, spread, mass, top = oracle.kv8.attend(qv, h["kp"], h["vp"], h["ks"], h["vs"], h["table"], h["lens"], page, D ** -0.5, kind)
        tol, ltol = bounds(ro, spread, mass, top, int(h["lens"].max()), D, kind, "fp32")
        assert np.all(np.abs(o.double().cpu().numpy() - ro) <= tol)
        dead = np.isinf(rl)
        lse = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(lse), dead) and np.all(np.abs(lse[~dead] - rl[~dead]) <= ltol[~dead] + 2.0 ** -23 * np.abs(rl[~dead]))
        assert np.array_equal(table.cpu().numpy(), h["table"]) and np.array_equal(refs.cpu().numpy(), h["refs"])

    step([40, 0, 23, 0], 40)          # two prompts
    step([1, 0, 1, 0], 1)
    pools = [kp, vp, ks, vs]
    fa.fork_pages(table, lens, refs, page, i32([0, 0]), i32([1, 3]), pools)
    assert oracle.pages.fork(h["table"], h["lens"], h["refs"], page, [0, 0], [1, 3], [h["kp"], h["vp"], h["ks"], h["vs"]])
    for _ in range(9):
        step([1, 1, 1, 1], 1)         # the forks go on on their own
    step([4, 5, 0, 1], 5)             # drafts of unlike lengths
    fa.free_pages(table, lens, refs, page, i32([0, 2]))
    oracle.pages.free(h["table"], h["lens"], h["refs"], page, [0, 2])
    table, refs, remap, n_live = fa.compact_pages(table, lens, refs, page, pools)
    h["table"], h["refs"], want, n = oracle.pages.compact(h["table"], h["lens"], h["refs"], page, [h["kp"], h["vp"], h["ks"], h["vs"]])
    assert int(n_live) == n and np.array_equal(remap.cpu().numpy(), want)
    step([17, 1, 30, 2], 2)
    assert fa.fa_device_status(clear=True) == 0
