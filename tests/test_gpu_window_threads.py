"""Decodes with bf16 windows of different sizes from several host threads at once."""
import ctypes
import threading

import pytest
import torch

from quantized_attention_kvq_b200 import native

pytestmark = pytest.mark.gpu


def test_windows_of_different_size_decode_at_the_same_time():
    # each size asks the window kernel for its own amount of shared memory (over 48 KB); neither
    # call may narrow the other's
    H, G, T = 1, 16, 2048
    failed = []

    def work(window, stream):
        try:
            torch.cuda.set_device(0)
            gen = torch.Generator(device="cuda").manual_seed(window)
            cache = native.KVQCache(1, H, T, 4, 4, sink=4, recent=window - 4)
            k, v = (torch.randn(1, H, T, 128, device="cuda", generator=gen, dtype=torch.bfloat16) for _ in range(2))
            cache.append(k, v, 0)
            q = torch.randn(1, H * G, 128, device="cuda", generator=gen, dtype=torch.bfloat16)
            lens = torch.full((1,), T, dtype=torch.int32, device="cuda")
            ref = cache.decode(q, lens, T)
            out = torch.empty_like(ref)
            ws = torch.empty(cache.workspace_bytes(H * G, T), dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
            call = native.lib().kvq_decode_attention
            args = (ctypes.byref(cache.desc), q.data_ptr(), native.KVQ_BF16, H * G, lens.data_ptr(), T, None, 128 ** -0.5,
                    out.data_ptr(), ws.data_ptr(), ws.numel(), stream.cuda_stream)
            for i in range(3000):
                assert call(*args) == native.KVQ_OK, i
            stream.synchronize()
            assert torch.equal(out, ref)
        except Exception as e:  # noqa: BLE001
            failed.append((window, e))

    threads = [threading.Thread(target=work, args=(w, torch.cuda.Stream())) for w in (2048, 700, 1000, 1500)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
