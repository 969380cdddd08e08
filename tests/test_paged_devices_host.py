"""On which device and stream the paged cache's Python calls run, with a library and devices that are fakes
(no GPU)."""
import contextlib
from types import SimpleNamespace

import pytest

from quantized_attention_kvq_b200 import native


@pytest.fixture
def two_devices(monkeypatch):
    """Device 0 is current; returns what the library was called with and the device it was called on."""
    calls, on = [], [0]

    @contextlib.contextmanager
    def device(d):
        on.append(d)
        yield
        on.pop()

    monkeypatch.setattr(native.torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    monkeypatch.setattr(native.torch.cuda, "current_device", lambda: on[-1])
    monkeypatch.setattr(native.torch.cuda, "current_stream", lambda d=None: SimpleNamespace(cuda_stream=1000 + (on[-1] if d is None else d)))
    monkeypatch.setattr(native.torch.cuda, "device", device)

    def status(ref, batch, q_heads, ws, nbytes, stream):
        calls.append((on[-1], stream, ws))
        return native.KVQ_ERR_TIMEOUT

    monkeypatch.setattr(native, "lib", lambda: SimpleNamespace(kvq_paged_decode_status=status))
    return calls


def tensor(dev, ptr):
    return SimpleNamespace(get_device=lambda: dev, is_cuda=True, is_contiguous=lambda: True, data_ptr=lambda: ptr, nbytes=64,
                           device=f"cuda:{dev}")


def test_decode_status_asks_the_workspaces_device_and_its_current_stream(two_devices):
    # the decode ran on the current stream of the workspace's device: read anywhere else, the
    # status words could be copied before the decode wrote them
    cache = native.PagedKVQCache.__new__(native.PagedKVQCache)
    cache._ref, cache.pages = None, tensor(1, 7)
    assert cache.decode_status(2, 8, tensor(1, 5)) == native.KVQ_ERR_TIMEOUT
    assert cache.decode_status(2, 8, tensor(1, 5), stream=SimpleNamespace(cuda_stream=77)) == native.KVQ_ERR_TIMEOUT
    assert two_devices == [(1, 1001, 5), (1, 77, 5)]
    with pytest.raises(ValueError):
        cache.decode_status(2, 8, tensor(0, 5))
