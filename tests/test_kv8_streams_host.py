"""Which stream and device the helpers of the 8-bit cache make current, and that they put back what was: on the CPU,
with stand-ins for torch.cuda's contexts, streams and devices."""
import contextlib
import types

import pytest

from exact_tiled_attention_47_b200 import kv8, pages

torch = pytest.importorskip("torch")

HERE, THERE = torch.device("cuda", 0), torch.device("cuda", 1)


def stream_of(device, raw):
    return types.SimpleNamespace(device=device, cuda_stream=raw)


@pytest.fixture
def cuda(monkeypatch):
    """The contexts that are open, and all that were ever entered."""
    log = types.SimpleNamespace(open=[], entered=[])

    @contextlib.contextmanager
    def context(x):
        log.open.append(x)
        log.entered.append(x)
        try:
            yield
        finally:
            assert log.open.pop() is x

    kv8._torch()
    monkeypatch.setattr(torch.cuda, "device", context)
    monkeypatch.setattr(torch.cuda, "stream", context)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: stream_of(device, 70 + device.index))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: stream_of(device, 0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device: stream_of(device, raw))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 70 + index, raising=False)
    yield log
    assert not log.open


@pytest.mark.parametrize("device,stream,raw,entered", [
    (HERE, None, 70, 0),
    (THERE, None, 71, 1),
    (HERE, stream_of(HERE, 5), 5, 2),
    (THERE, stream_of(THERE, 6), 6, 2),
    (HERE, 0, 0, 2),
    (THERE, 8, 8, 2),
])
def test_the_place_of_a_call(cuda, device, stream, raw, entered):
    context, got = kv8.place_of(device, stream)
    assert got == raw and (context is None) == (entered == 0)
    assert not cuda.entered  # not before the helper runs
    assert kv8.in_context(context, lambda: list(cuda.open)) == cuda.entered and len(cuda.entered) == entered
    assert not entered or cuda.entered[0] == device
    assert entered < 2 or cuda.entered[1].cuda_stream == raw


def test_refusals_enter_nothing(cuda):
    with pytest.raises(ValueError, match="another device"):
        kv8.place_of(THERE, stream_of(HERE, 5))
    with pytest.raises(ValueError, match="CUDA"):
        kv8.place_of(torch.device("cpu"), stream_of(HERE, 5))
    assert not cuda.entered


def test_errors_leave_what_was_entered(cuda):
    context, _ = kv8.place_of(THERE, stream_of(THERE, 5))
    with pytest.raises(RuntimeError):
        kv8.in_context(context, lambda: (_ for _ in ()).throw(RuntimeError()))
    assert len(cuda.entered) == 2 and not cuda.open


@pytest.mark.parametrize("device", [HERE, THERE])
@pytest.mark.parametrize("stream", [None, 9])
@pytest.mark.parametrize("name", ["extend", "fork", "free", "copy"])
def test_an_empty_list_leaves_stream_and_device_as_they_were(cuda, monkeypatch, name, stream, device):
    monkeypatch.setattr(pages, "_check_state", lambda *a: (4, 4, 16, device))
    monkeypatch.setattr(pages, "_check_list", lambda *a: 0)
    monkeypatch.setattr(pages, "_page_bytes", lambda *a: [64])
    pool = [types.SimpleNamespace(device=device, shape=(16, 64))]
    call = {
        "extend": lambda: pages.extend_pages(None, None, None, 16, None, stream=stream),
        "fork": lambda: pages.fork_pages(None, None, None, 16, None, None, pool, stream=stream),
        "free": lambda: pages.free_pages(None, None, None, 16, None, stream=stream),
        "copy": lambda: pages.copy_pages(pool, pool, None, None, stream=stream),
    }[name]
    call()
    assert not cuda.open
