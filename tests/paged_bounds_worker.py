"""Runs small paged plans, appends, read-backs and decodes through whichever library
KVQ_LIBRARY selects and prints a digest of the pool's bytes and the outputs and
the library's bounds-violation count as JSON.  Used by
tests/test_gpu_paged_give_up.py in a child process."""
import hashlib
import json
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from quantized_attention_kvq_b200 import native  # noqa: E402


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def main():
    L = native.lib()
    L.kvq_bounds_violations(1)
    h = hashlib.sha256()
    gen = torch.Generator().manual_seed(77)
    for kb, vb, P, H, G, dtype, ch0, keep in [(4, 4, 64, 2, 1, torch.bfloat16, 0, None), (4, 2, 128, 2, 8, torch.float16, 1, 19),
                                              (2, 4, 64, 1, 16, torch.float32, 1, 24), (2, 2, 192, 3, 5, torch.bfloat16, 0, 3)]:
        cache = native.PagedKVQCache(24, H, kb, vb, page_tokens=P, keep_ch0=ch0)
        lens = [700, 0, 1, 65, 333]
        B, n = len(lens), sum(lens)
        table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
        plan = cache.planner.plan(i32([0] * B), i32(lens), table, torch.arange(24, dtype=torch.int32, device="cuda"), i32([24]),
                                  n + 5)
        k, v = (torch.randn(n + 5, H, 128, generator=gen).to("cuda", dtype) for _ in range(2))
        cache.append(k, v, plan.slots)
        q = torch.randn(B, H * G, 128, generator=gen).to("cuda", dtype)
        mask = None if keep is None else cache.select(q, keep)
        out = cache.decode(q, table, plan.seq_lens, 12 * P, mask)
        table[0, 2] = 1 << 30  # and a page that is none
        for t in (cache.pages, plan.slots, plan.seq_lens, *cache.gather(plan.slots, dtype), out,
                  cache.decode(q, table, plan.seq_lens, 12 * P, mask)):
            assert t.dtype == torch.uint8 or torch.isfinite(t.float()).all()
            h.update(t.contiguous().view(torch.uint8).cpu().numpy().tobytes())
    print(json.dumps({"digest": h.hexdigest(), "violations": int(L.kvq_bounds_violations(0))}))


if __name__ == "__main__":
    main()
