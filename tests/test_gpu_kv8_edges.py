"""The paged 8-bit cache at its edges on the GPU: how ragged work is cut over the CTAs, offsets above 32 bits,
guard bands around every output, and the index-checking debug build."""
import math

import numpy as np
import pytest

import oracle
from kv8_cases import bounds, make_cache
from parity import Guarded
from test_gpu_kv8 import CODE, FLOAT, rounded, to_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_tiled_attention_47_b200 import build
    build.build()
    build.build(debug=True)
    import exact_tiled_attention_47_b200 as fa
    fa.fa_device_status(clear=True)
    yield
    assert fa.fa_device_status(clear=True) == 0


def plain(q, cache, lens, kind):
    """O and LSE of every row in fp64 on the GPU, from values gathered in table order."""
    kp, vp, ks, vs, table = cache
    B, Nq, Hq, D = q.shape
    Hkv, page = kp.shape[1], kp.shape[2]
    G = Hq // Hkv
    o = torch.zeros((B, Nq, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")
    spread = torch.zeros_like(o)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = table[b, : -(-n // page)].long()
        val = lambda c, s: (c.view(torch.int8)[ids].view(CODE[kind]).double() * s[ids].double().repeat_interleave(16, -1).unsqueeze(-1)).transpose(0, 1).flatten(1, 2)[:, :n]  # noqa: E731
        K, V = val(kp, ks), val(vp, vs)
        x = torch.einsum("thgd,hkd->hgtk", q[b].double().view(Nq, Hkv, G, D), K) * D ** -0.5
        see = torch.arange(n, device="cuda") <= n - Nq + torch.arange(Nq, device="cuda")[:, None]
        x = x.masked_fill(~see, -math.inf)
        t = torch.logsumexp(x, -1)
        w = torch.exp(x - torch.where(torch.isinf(t), 0.0, t)[..., None])
        o[b] = torch.einsum("hgtk,hkd->thgd", w, V).reshape(Nq, Hq, D)
        spread[b] = torch.einsum("hgtk,hkd->thgd", w, V.abs()).reshape(Nq, Hq, D)
        lse[b] = t.reshape(Hq, Nq)
    return o, lse, spread


# Weights are rounded to fp16: 2^-11 of sum_j p_j |V_j|.  With these inputs sum_d |q_d k_d| / sqrt(D) stays below 2^5, so
# scores are off by at most ds = 2 (D + 8) 2^-24 2^5 < 2^-10.9 (kv8_cases.bounds): the LSE by as much, O by 2 ds of the
# spread beside the 2^-11.  A piece that is lost or merged twice is off by far more.
def close(o, lse, ref, what):
    ro, rl, spread = ref
    dead = torch.isinf(rl)
    assert torch.equal(torch.isneginf(lse), dead), what
    assert torch.all((o.double() - ro).abs() <= spread * 2.0 ** -9 + 2.0 ** -24), what
    assert torch.all((lse.double() - rl)[~dead].abs() <= 2.0 ** -10), what


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("Nq,G", [(1, 4), (1, 16), (2, 11), (3, 9), (9, 15)])
def test_shares_of_ragged_batches(seed, Nq, G):
    # lengths of all orders, zeros and lengths below Nq among them: the borders of the shares fall on every place
    # of a unit, and units come in one piece, two, or dozens
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(seed * 100 + Nq * G)
    B = int(rng.choice([1, 2, 7, 40, 300]))
    top = int(rng.choice([1100, 5000, 40000 // B + 1030]))
    lens = [int(np.exp(rng.uniform(0, np.log(top)))) if rng.random() < 0.9 else 0 for _ in range(B)]
    lens[0] = top
    kind = "e4m3" if seed % 2 else "int8"
    cache = make_cache(rng, lens, 1, 64, 32, kind)
    q, _ = rounded(rng, (B, Nq, G, 64), "bf16", 0.3)
    g = to_gpu(cache, kind)
    o, lse = fa.attend_kv8(q, *g, torch.tensor(lens, dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == 0
    close(o, lse, plain(q, g, lens, kind), (B, top))


@pytest.mark.parametrize("Nq,G,D,kind", [(1, 1, 128, "e4m3"), (3, 5, 128, "int8"), (1, 16, 64, "e4m3"), (4, 9, 128, "e4m3")])
def test_units_of_many_pieces(Nq, G, D, kind):
    # few heads and long contexts: a unit is cut into a hundred pieces, beside one of a single key and an empty one
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(900 + G)
    lens = [60000, 1, 20011, 0]
    cache = make_cache(rng, lens, 1, D, 64, kind)
    q, _ = rounded(rng, (4, Nq, G, D), "bf16", 0.3)
    g = to_gpu(cache, kind)
    o, lse = fa.attend_kv8(q, *g, torch.tensor(lens, dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == 0
    close(o, lse, plain(q, g, lens, kind), lens)
    again, _ = fa.attend_kv8(q, *g, torch.tensor(lens, dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    assert torch.equal(o, again)


@pytest.mark.parametrize("Nq,G", [(1, 2), (40, 3)])
def test_more_items_than_threads(Nq, G):
    # the scan over the lengths takes several steps
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(5)
    B = 1500
    lens = [int(x) for x in rng.integers(0, 60, B)]
    lens[700], lens[1499] = 1200, 1300
    cache = make_cache(rng, lens, 1, 64, 16, "e4m3")
    q, _ = rounded(rng, (B, Nq, G, 64), "fp16", 0.3)
    g = to_gpu(cache, "e4m3")
    o, lse = fa.attend_kv8(q, *g, torch.tensor(lens, dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    close(o, lse, plain(q, g, lens, "e4m3"), B)


@pytest.mark.parametrize("Nq", [1, 80])
def test_offsets_above_32_bits(Nq):
    # pools of 5 GB each: the pages in use lie at their end
    import exact_tiled_attention_47_b200 as fa
    page, Hkv, D, P = 64, 8, 128, 80000
    rng = np.random.default_rng(6)
    small = make_cache(rng, [200, 131], Hkv, D, page, "int8", spare=0)
    n = small[0].shape[0]
    kp, vp = (torch.empty((P, Hkv, page, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((P, Hkv, page // 16), device="cuda") for _ in range(2))
    g = to_gpu(small, "int8")
    for big, part in zip((kp, vp, ks, vs), g):
        big[P - n:] = part
    table = torch.where(g[4] >= 0, g[4] + (P - n), g[4])
    q, _ = rounded(rng, (2, Nq, Hkv, D), "bf16")
    sl = torch.tensor([200, 131], dtype=torch.int32, device="cuda")
    want, got = fa.attend_kv8(q, *g[:4], g[4], sl), fa.attend_kv8(q, kp, vp, ks, vs, table, sl)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    k, _ = rounded(rng, (2, 5, Hkv, D), "bf16")
    fa.append_kv8(k, k, *g[:4], g[4], sl)
    fa.append_kv8(k, k, kp, vp, ks, vs, table, sl)
    for big, part in zip((kp, vp), g):
        assert torch.equal(big[P - n:], part)
    # the same places copied down by the page operations
    before = kp[P - 1].clone()
    fa.copy_pages([kp, vp], [kp, vp], torch.tensor([P - 1], dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda"))
    assert torch.equal(kp[3], before)
    assert fa.fa_device_status(clear=True) == 0


def test_guard_bands():
    # nothing outside O, LSE, the workspace, the pools' used rows and the state is written
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(7)
    for Nq, G, lens in ((1, 3, [1500, 0, 77]), (50, 3, [700, 20, 0])):
        cache = make_cache(rng, lens, 2, 128, 16, "e4m3")
        g = to_gpu(cache, "e4m3")
        q, _ = rounded(rng, (3, Nq, 2 * G, 128), "fp16")
        o, lse = Guarded((3, Nq, 2 * G, 128), torch.float16), Guarded((3, 2 * G, Nq), torch.float32)
        n = fa.fa_kv8_attend_workspace_bytes(3, Nq, 2 * G, 2, 128)
        ws = Guarded((n,), torch.uint8)
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st = fa.fa_kv8_attend(q, *g, o.t, lse.t, 3, Nq, 2 * G, 2, g[0].shape[0], 16, g[4].shape[1], 128, 128 ** -0.5, sl, ws.t)
        assert st == fa.FA_OK
        want = fa.attend_kv8(q, *g, sl)
        torch.cuda.synchronize()
        assert o.intact() and lse.intact() and ws.intact()
        assert torch.equal(o.t, want[0]) and torch.equal(lse.t, want[1])
    ends, new = [37, 16, 5], [9, 16, 0]
    cache = make_cache(rng, ends, 2, 64, 16, "int8", spare=1)
    gk, gv = (Guarded(cache[0].shape, torch.int8) for _ in range(2))
    sk, sv = (Guarded(cache[2].shape, torch.float32) for _ in range(2))
    src = to_gpu(cache, "int8")
    for a, b in zip((gk, gv, sk, sv), src):
        a.t.copy_(b)
    k, _ = rounded(rng, (3, 16, 2, 64), "bf16")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    fa.append_kv8(k, k, gk.t, gv.t, sk.t, sv.t, src[4], i32(ends), i32(new))
    fa.append_kv8(k, k, *src, i32(ends), i32(new))
    torch.cuda.synchronize()
    assert all(x.intact() for x in (gk, gv, sk, sv)) and torch.equal(gk.t, src[0]) and torch.equal(gv.t, src[1])


@pytest.fixture
def use_debug(monkeypatch):
    import exact_tiled_attention_47_b200 as fa
    monkeypatch.setattr(fa._lib, "_lib", fa._lib.load(fa.DEBUG_LIB_PATH))
    fa.fa_device_status(clear=True)
    yield fa
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == 0, "an index check of the debug build fired"


@pytest.mark.parametrize("Nq,G,D,kind", [(1, 4, 128, "e4m3"), (5, 3, 64, "int8"), (4, 7, 128, "int8"), (90, 2, 128, "e4m3"), (300, 1, 64, "int8")])
def test_debug_build_agrees_and_finds_no_stray_index(use_debug, Nq, G, D, kind):
    fa = use_debug
    rng = np.random.default_rng(Nq)
    lens = [1700, 33, 0, 260]
    cache = make_cache(rng, lens, 2, D, 32, kind)
    g = to_gpu(cache, kind)
    q, _ = rounded(rng, (4, Nq, 2 * G, D), "bf16", 0.3)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.attend_kv8(q, *g, sl, out_dtype=torch.float32)
    close(o, lse, plain(q, g, lens, kind), "debug")
    assert fa.fa_build_flags() == fa.FA_BUILD_DEBUG
    k, _ = rounded(rng, (4, 20, 2, D), "bf16")
    new = torch.tensor([20, 7, 0, 1], dtype=torch.int32, device="cuda")
    fa.append_kv8(k, k, *g, sl, new)


def test_debug_build_page_operations(use_debug):
    from test_gpu_pages import Both
    t = Both(11, 8, 6, 40, 16)
    assert t.extend([0, 3], [50, 16])
    assert t.fork([0, 3], [5, 1])
    t.free([0])
    t.compact(False)
    t.compact(True)
