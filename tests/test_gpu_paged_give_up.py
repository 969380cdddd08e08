"""The paged decode's bounded waits, and the paged kernels in the bounds-checked build.

A test hook leaves one tile of the decode's first warp unfilled (no fault, no trap:
a barrier that nothing completes).  The decode must then return, the heads of that
warp's tiles must be NaN, the others as before, the status must say so, and the
next decode on the same workspace must be right again.
"""
import json
import os
import subprocess
import sys

import pytest
import torch

from quantized_attention_kvq_b200 import native

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("B,T,masked", [
    (2, 9000, True),      # many partials a row
    (2, 300, True),       # a warp of the joining pass has one partial, the lost one
    (300, 64 * 3, False),  # few partials a row
])
def test_a_wait_that_runs_out_is_reported(B, T, masked):
    H, G, P = 2, 4, 64
    pages = (T + P - 1) // P
    cache = native.PagedKVQCache(B * pages, H, 4, 4, page_tokens=P)
    gen = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(B * T, H, 128, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    pos = torch.arange(T, device="cuda")
    cache.append(k, v, (table[:, pos // P] * P + pos % P).int().flatten())
    q = torch.randn(B, H * G, 128, generator=gen, device="cuda", dtype=torch.bfloat16)
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    mask = cache.select(q, 20) if masked else None
    ws = torch.empty(cache.workspace_bytes(B, H * G), dtype=torch.uint8, device="cuda")
    ref = cache.decode(q, table, lens, T, mask, workspace=ws).clone()
    assert torch.isfinite(ref.float()).all() and cache.decode_status(B, H * G, ws) == native.KVQ_OK
    native.lib().kvq_test_withhold_tile(0)
    out = cache.decode(q, table, lens, T, mask, workspace=ws)
    assert cache.decode_status(B, H * G, ws) == native.KVQ_ERR_TIMEOUT
    lost = out[0, :G].float()  # the first warp's range starts with request 0, head 0
    assert lost.isnan().all()
    assert torch.equal(out.view(-1, 128)[G:], ref.view(-1, 128)[G:])
    again = cache.decode(q, table, lens, T, mask, workspace=ws)
    assert cache.decode_status(B, H * G, ws) == native.KVQ_OK
    assert torch.equal(again, ref)


def test_checked_build_gives_the_same_bits_and_counts_nothing():
    got = {}
    for which in ("", "checked"):
        env = dict(os.environ, KVQ_LIBRARY=which)
        r = subprocess.run([sys.executable, os.path.join(HERE, "paged_bounds_worker.py")], env=env, capture_output=True,
                           text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        got[which] = json.loads(r.stdout.strip().splitlines()[-1])
    assert got["checked"]["violations"] == 0
    assert got["checked"]["digest"] == got[""]["digest"]
