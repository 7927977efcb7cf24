"""Page operations on a state that does not fit together: what is reported, and that nothing else is touched."""
import pytest

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


def status():
    import exact_tiled_attention_47_b200 as fa
    torch.cuda.synchronize()
    return fa.fa_device_status(clear=True)


@pytest.mark.parametrize("bad", [8, 3, 15])  # free pages: the lowest one, which would be handed out, and others
def test_fork_of_a_partial_page_that_nobody_holds(bad):
    import exact_tiled_attention_47_b200 as fa
    t = Both(1, 8, 4, 16, 16)
    assert t.extend([0, 1], [64, 50])  # pages 0 to 3 and 4 to 7
    if bad == 3:  # free again by hand
        t.refs[3] = 0
        t.lens[0] = 48
    t.table[1, 3] = bad
    t.dev()
    fa.fork_pages(t.gt, t.gl, t.gr, 16, i32([0, 1]), i32([2, 3]), t.gp)
    assert status() == fa.FA_ERR_PAGE_TABLE
    t.same()
    assert (t.gt[2:4] == -1).all()


@pytest.mark.parametrize("bad", [8, 9, 15, 16, -1])  # handed out to another fork of the call; free; outside the pool
@pytest.mark.parametrize("forks", [1, 3])
def test_fork_of_a_full_page_that_nobody_holds(bad, forks):
    import exact_tiled_attention_47_b200 as fa
    t = Both(2, 12, 4, 16, 16)
    assert t.extend([0, 1], [64, 50])
    t.table[0, 2] = bad
    t.dev()
    dst = list(range(2, 2 + forks))
    fa.fork_pages(t.gt, t.gl, t.gr, 16, i32([0] * forks + [1]), i32(dst + [10]), t.gp)
    assert status() == fa.FA_ERR_PAGE_TABLE
    for d in dst:
        assert t.gt[d].tolist() == [0, 1, -1, 3]
    assert t.gt[10].tolist() == [4, 5, 6, 8]  # the other fork is met: its partial page is copied to page 8
    assert all(torch.equal(x[8], x[7]) for x in t.gp)
    assert t.gr.tolist() == [1 + forks, 1 + forks, 1, 1 + forks, 2, 2, 2, 1, 1] + [0] * 7
    assert t.gl.tolist() == [64, 50] + [64] * forks + [0] * (8 - forks) + [50, 0]


@pytest.mark.parametrize("length", [-1, 65, 2 ** 31 - 1, -2 ** 31])
def test_free_of_a_slot_whose_length_is_out_of_range(length):
    import exact_tiled_attention_47_b200 as fa
    t = Both(3, 4, 4, 16, 16)
    assert t.extend([0, 1, 2], [40, 33, 64])
    t.lens[1] = length
    t.dev()
    fa.free_pages(t.gt, t.gl, t.gr, 16, i32([0, 1, 1, 2]))
    assert status() == fa.FA_ERR_CU_SEQLENS
    # slots 0 and 2 are free, slot 1 is as it was: put right, it can be freed as well
    assert t.gl.tolist() == [0, length, 0, 0] and t.gr.tolist() == [0, 0, 0, 1, 1, 1] + [0] * 10
    assert t.gt[1].tolist() == t.table[1].tolist() and (t.gt[[0, 2]] == -1).all()
    t.gl[1] = 33
    fa.free_pages(t.gt, t.gl, t.gr, 16, i32([1, 1]))
    assert status() == 0 and not t.gl.any() and not t.gr.any()
