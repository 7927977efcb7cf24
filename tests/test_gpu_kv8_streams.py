"""The helpers of the 8-bit cache with a stream of the caller's: they run there, and leave what was current as it was."""
import numpy as np
import pytest

from kv8_cases import make_cache
from test_gpu_kv8 import rounded, to_gpu
from test_gpu_pages import Both, i32

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


@pytest.fixture(params=["stream", "handle", "default"])
def stream(request):
    """A stream as a caller names it; what was current must be current behind the test's calls."""
    s = torch.cuda.Stream()
    was = torch.cuda.current_stream(), torch.cuda.current_device()
    yield {"stream": s, "handle": s.cuda_stream, "default": 0}[request.param]
    assert (torch.cuda.current_stream(), torch.cuda.current_device()) == was
    torch.cuda.synchronize()


def test_empty_lists(stream):
    import exact_tiled_attention_47_b200 as fa
    t, e, was = Both(1, 4, 4, 24, 16), i32([]), torch.cuda.current_stream()
    torch.cuda.synchronize()
    for call in (lambda: fa.extend_pages(t.gt, t.gl, t.gr, 16, e, e, stream=stream), lambda: fa.fork_pages(t.gt, t.gl, t.gr, 16, e, e, t.gp, stream=stream),
                 lambda: fa.free_pages(t.gt, t.gl, t.gr, 16, e, stream=stream), lambda: fa.copy_pages(t.gp, t.gp, e, e, stream=stream)):
        call()
        assert torch.cuda.current_stream() == was
    t.same()


def test_append_attend_and_pages(stream):
    import exact_tiled_attention_47_b200 as fa
    rng = np.random.default_rng(2)
    cache = make_cache(rng, [40, 21], 2, 64, 16, "e4m3")
    a, b = to_gpu(cache, "e4m3"), to_gpu(cache, "e4m3")
    k, _ = rounded(rng, (2, 3, 2, 64), "bf16")
    q, _ = rounded(rng, (2, 1, 4, 64), "bf16")
    sl, add = i32([40, 21]), i32([17, 30])
    t = Both(3, 4, 4, 24, 16)
    fa.append_kv8(k, k, *b, sl)
    want = fa.attend_kv8(q, *b, sl)
    torch.cuda.synchronize()
    fa.append_kv8(k, k, *a, sl, stream=stream)
    o, lse = fa.attend_kv8(q, *a, sl, stream=stream)
    fa.extend_pages(t.gt, t.gl, t.gr, 16, add, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert t.gl.tolist() == [17, 30, 0, 0] and t.gr.tolist() == [1] * 4 + [0] * 20
