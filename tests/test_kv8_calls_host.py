"""Helpers and the functions named like the C entry points pass on the same arguments (CPU, a stand-in for the library)."""
import ctypes

import pytest

import exact_tiled_attention_47_b200 as fa
from exact_tiled_attention_47_b200 import _lib, kv8, pages

torch = pytest.importorskip("torch")

STREAM = 77


class Library:
    """Keeps what each entry point is called with: numbers as they are, host arrays by what they hold."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_workspace_bytes"):
                return 4096
            assert len(args) == len(_lib.SIGNATURES[name][1])
            self.calls.append((name, [list(a) if isinstance(a, ctypes.Array) else a for a in args]))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(_lib, "_lib", lib)
    for module in (fa, kv8, pages):
        monkeypatch.setattr(module, "load", lambda: lib)
    for module in (kv8, pages):
        monkeypatch.setattr(module, "place_of", lambda device, stream: (None, STREAM))
    kv8._workspace_bytes.cache_clear()
    pages._workspace_bytes.cache_clear()
    yield lib
    kv8._workspace_bytes.cache_clear()
    pages._workspace_bytes.cache_clear()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def same(lib):
    """The two calls since the last look were alike."""
    first, second = lib.calls
    assert first == second
    lib.calls.clear()


@pytest.mark.parametrize("code", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("new_lens", [None, i32(3)])
def test_append(lib, code, new_lens):
    cache = fa.new_kv8_cache(5, 32, 2, 64, dtype=code, device="cpu")
    k, v = torch.zeros((2, 3, 7, 2, 64), dtype=torch.bfloat16)
    table, lens = i32(3, 4), i32(3)
    fa.append_kv8(k, v, *cache, table, lens, new_lens)
    assert fa.fa_kv8_append(k, v, *cache, table, lens, new_lens, 3, 7, 2, 5, 32, 4, 64, STREAM) == 0
    same(lib)


@pytest.mark.parametrize("out", [None, torch.float32])
@pytest.mark.parametrize("lens", [None, i32(3)])
def test_attend(lib, out, lens):
    cache = fa.new_kv8_cache(5, 16, 2, 128, device="cpu")
    q, table, ws = torch.zeros((3, 4, 6, 128), dtype=torch.float16), i32(3, 9), torch.zeros(4096, dtype=torch.uint8)
    o, lse = fa.attend_kv8(q, *cache, table, lens, scale=0.3, out_dtype=out, workspace=ws)
    assert o.shape == q.shape and o.dtype == (out or q.dtype) and lse.shape == (3, 6, 4)
    assert fa.fa_kv8_attend(q, *cache, table, o, lse, 3, 4, 6, 2, 5, 16, 9, 128, 0.3, lens, ws, stream=STREAM) == 0
    same(lib)


def test_pages(lib):
    table, lens, refs, n2, ws = i32(4, 6), i32(4), i32(9), i32(2), torch.zeros(4096, dtype=torch.uint8)
    pools, sizes = [torch.zeros((9, 20), dtype=torch.uint8), torch.zeros((9, 3, 2))], [20, 24]
    state = (table, lens, refs)
    for slots in (None, n2):
        fa.extend_pages(*state, 16, n2, slots, workspace=ws)
        assert fa.fa_pages_extend(*state, slots, n2, 2, 4, 6, 9, 16, ws, stream=STREAM) == 0
        same(lib)
    fa.fork_pages(*state, 16, n2, n2, pools, workspace=ws)
    assert fa.fa_pages_fork(*state, n2, n2, 2, 4, 6, 9, 16, pools, sizes, ws, stream=STREAM) == 0
    same(lib)
    fa.free_pages(*state, 16, n2)
    assert fa.fa_pages_free(*state, n2, 2, 4, 6, 9, 16, STREAM) == 0
    same(lib)
    for in_place in (False, True):
        out = fa.compact_pages(*state, 16, pools, in_place=in_place, workspace=ws)
        assert fa.fa_pages_compact(*state, *out, 4, 6, 9, 16, pools, sizes, ws, stream=STREAM) == 0
        same(lib)
    other = [torch.zeros((12, 20), dtype=torch.uint8), torch.zeros((12, 6))]
    fa.copy_pages(pools, other, n2, n2, workspace=ws)
    assert fa.fa_pages_copy(pools, other, sizes, n2, n2, 2, 9, 12, ws, stream=STREAM) == 0
    same(lib)
