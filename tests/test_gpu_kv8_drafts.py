"""Drafted tokens that are not accepted: what a caller does with the lengths, so that no page and no key is lost."""
import numpy as np
import pytest

import oracle
from kv8_cases import bounds
from test_gpu_kv8 import CODE, rounded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


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


def i32(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("own_lengths", [True, False])
@pytest.mark.parametrize("kind,dtype", [("e4m3", "bf16"), ("int8", "fp16")])
def test_rejected_drafts(kind, dtype, own_lengths):
    """Windows of up to 6 drafted tokens, 0 to all of them accepted.  own_lengths: the slots keep what they hold and the valid
    lengths are an array of their own; else the slots' lengths are lowered, drafts being kept short enough for the page."""
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(800 + own_lengths)
    S, page, Hkv, G, D, pages, pps = 3, 16, 2, 2, 64, 40, 12
    cache = fa.new_kv8_cache(pages, page, Hkv, D, dtype=CODE[kind])
    table = torch.full((S, pps), -1, dtype=torch.int32, device="cuda")
    held, refs = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    h = [np.zeros((pages, Hkv, page, D), np.uint8) for _ in range(2)] + [np.zeros((pages, Hkv, 1)) for _ in range(2)]
    h_table, h_held, h_refs = np.full((S, pps), -1, np.int32), np.zeros(S, np.int32), np.zeros(pages, np.int32)
    valid = np.zeros(S, np.int64)

    def step(new):
        add = [max(0, int(n + d - x)) for n, d, x in zip(valid, new, h_held)]
        fa.extend_pages(table, held, refs, page, i32(add))
        assert oracle.pages.extend(h_table, h_held, h_refs, page, range(S), add)
        ends = valid + new
        assert np.all(ends <= h_held)
        lens = i32(ends) if own_lengths else held
        Nt = max(int(max(new)), 1)
        k, kv = rounded(rng, (S, Nt, Hkv, D), dtype, float(2.0 ** rng.integers(-3, 4)))  # scales that rejected rows raise
        v, vv = rounded(rng, (S, Nt, Hkv, D), dtype)
        q, qv = rounded(rng, (S, Nt, Hkv * G, D), dtype, 0.3)
        fa.append_kv8(k, v, *cache, table, lens, i32(new))
        o, lse = fa.attend_kv8(q, *cache, table, lens, out_dtype=torch.float32)
        for i, x in enumerate((kv, vv)):
            h[i], h[2 + i], _ = oracle.kv8.append(x, h[i], h[2 + i], h_table, ends, new, page, kind)
        ro, rl, spread, mass, top = oracle.kv8.attend(qv, *h, h_table, ends, page, D ** -0.5, kind)
        tol, ltol = bounds(ro, spread, mass, top, int(ends.max()), D, kind, "fp32")
        assert np.all(np.abs(o.double().cpu().numpy() - ro) <= tol)
        lse, dead = lse.double().cpu().numpy(), np.isinf(rl)
        assert np.array_equal(np.isneginf(lse), dead) and np.all(np.abs(lse[~dead] - rl[~dead]) <= ltol[~dead] + 2.0 ** -23 * np.abs(rl[~dead]))
        assert np.array_equal(table.cpu().numpy(), h_table) and np.array_equal(refs.cpu().numpy(), h_refs)
        return ends

    valid = step(np.array([20, 5, 33]))
    for _ in range(20):
        drafts = rng.integers(0, 7, S)
        if not own_lengths:  # rejected keys must lie in the page of the last accepted one
            drafts = np.minimum(drafts, (-valid) % page)
            drafts[valid % page == 0] = 0
        ends = step(drafts)
        valid = ends - [int(rng.integers(0, d + 1)) for d in drafts]
        if not own_lengths:
            assert np.all(-(-valid // page) == -(-ends // page))
            held.copy_(i32(valid))
            h_held[:] = valid
            valid = step(np.ones(S, np.int64))  # the token that the model itself gives
    fa.free_pages(table, held, refs, page, i32(range(S)))
    assert not refs.any() and not held.any()  # no page is lost
    assert fa.fa_device_status(clear=True) == 0
