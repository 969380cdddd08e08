"""The paged cache on the GPU at the ends of its ranges, against values in 64 bits."""
import math

import numpy as np
import pytest
import torch

from paged_testlib import BT, D, Layout, attention, hadamard, output_bound
from quantized_attention_kvq_b200 import native
from test_gpu_paged import TYPES, Pool, decode_case, i32

pytestmark = pytest.mark.gpu


def held(cache, lay, h):
    """Keys and values [num_pages * page_tokens][128] of head h in 64 bits, as the pool's bytes hold them."""
    raw = cache.pages.cpu().numpy().reshape(cache.num_pages, cache.H, cache.page_tokens // BT, lay.bytes)
    kv = [lay.values(b) for b in raw[:, h].reshape(-1, lay.bytes)]
    return np.concatenate([x[0] for x in kv]), np.concatenate([x[1] for x in kv])


# ------------------------------------------------------------- large rotated values
@pytest.mark.parametrize("kb,vb,value", [(4, 4, 12000.0), (4, 4, -12000.0), (2, 2, 12000.0), (4, 2, 24000.0), (2, 4, 32000.0)])
@pytest.mark.parametrize("dtype,G", [("f16", 1), ("f16", 5), ("f16", 16), ("bf16", 4), ("f32", 4)])
def test_decode_of_large_equal_values_taken_back_through_the_rotation(kb, vb, value, dtype, G):
    # A row of equal values is one large channel after the rotation, sqrt(128) times the value: beyond
    # fp16, though its scale, its zero and the output fit.
    n, P = 130, 64
    cache = native.PagedKVQCache(3, 1, kb, vb, page_tokens=P, rotate_v=1)
    g = torch.Generator(device="cuda").manual_seed(kb + vb)
    k = torch.randn(n, 1, D, device="cuda", generator=g).half()
    cache.append(k, torch.full((n, 1, D), value, device="cuda", dtype=torch.float16), i32(np.arange(n)))
    q = torch.randn(1, G, D, device="cuda", generator=g).to(TYPES[dtype])
    out = cache.decode(q, i32([[0, 1, 2]]), i32([n]), n)
    kh, vh = (x[:n] for x in held(cache, Layout(kb, vb, 0), 0))
    for j in range(G):
        qr = hadamard() @ q[0, j].double().cpu().numpy()
        o = attention(qr, kh, vh, 1 / math.sqrt(D))
        bound = output_bound(o, qr, kh, vh, 1 / math.sqrt(D), dtype)
        bound = np.full(D, np.linalg.norm(bound)) + 2.0 ** -21 * np.linalg.norm(o)  # errors add up over the row
        o = hadamard() @ o
        bound = bound + np.abs(o) * torch.finfo(TYPES[dtype]).eps / 2
        err = np.abs(out[0, j].double().cpu().numpy() - o)
        assert (err <= bound).all()  # not-a-number fails


def test_value_scales_at_the_ends_of_fp16_with_fp16_outputs():
    # scales and zeros side by side over the whole type; outputs stay inside it
    pool = Pool(11, 9, 1, 64, 4, 4, 0)
    L = pool.lay
    half = lambda x: np.asarray(x, np.float16).view(np.uint8)  # noqa: E731
    n = pool.raw.shape[0] * 256
    sc = np.random.RandomState(0).choice([0.0, 6e-8, 1e-5, 0.2, 900.0, 4000.0], n)
    pool.raw[..., L.vs:L.vs + 512] = half(sc).reshape(pool.raw[..., L.vs:L.vs + 512].shape)
    pool.cache.pages.copy_(torch.from_numpy(pool.raw.reshape(-1)))
    _, check = decode_case(pool, 4, "f16", [513])
    for j in range(4):
        check(0, j)


# ------------------------------------------------------------- a caller's stream
def new_segments(call):
    """Streams of the memory the allocator takes from the device during a call."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = {x["address"] for x in torch.cuda.memory_snapshot()}
    call()  # what it returned is given back, but stays the allocator's
    return [x["stream"] for x in torch.cuda.memory_snapshot() if x["address"] not in before]


def test_memory_made_for_a_call_on_a_given_stream_belongs_to_that_stream():
    # sizes over the allocator's shared small blocks, so that each call takes memory of its own
    B, H, G, P, num = 512, 8, 4, 64, 64
    cache = native.PagedKVQCache(num, H, 4, 4, page_tokens=P)
    q = torch.randn(B, H * G, D, device="cuda", dtype=torch.bfloat16)
    table, lens = i32(np.arange(2 * B).reshape(B, 2) % num), i32(np.full(B, 100))
    n = 1 << 20
    zeros, ones = i32(np.zeros(B)), i32(np.ones(B))
    free, count, slots = i32(np.arange(num)), i32([num]), i32(np.arange(4096) % (num * P))
    side = torch.cuda.Stream()
    out = torch.empty_like(q)
    calls = [lambda: cache.decode(q, table, lens, 128, stream=side),
             lambda: cache.decode(q, table, lens, 128, out=out, stream=side),  # the workspace alone
             lambda: cache.gather(slots, torch.float32, stream=side),
             lambda: cache.planner.plan(zeros, ones, table, free, count, n, stream=side).slots]
    main = torch.cuda.current_stream()
    for call in calls:
        streams = new_segments(call)
        assert streams and all(s == side.cuda_stream for s in streams)
        assert torch.cuda.current_stream() == main  # as it was
    for call in (lambda: cache.decode(q, table, lens, 128), lambda: cache.gather(slots, torch.float32)):
        streams = new_segments(call)
        assert streams and all(s == main.cuda_stream for s in streams)


def test_decodes_on_a_given_stream_beside_allocations_on_the_current_one():
    pool = Pool(13, 60, 2, 64, 4, 4, 0)
    B, Hq = 6, 8
    table, lens = i32(np.random.RandomState(1).permutation(60).reshape(B, 10)), i32([640, 100, 7, 333, 64, 0])
    q = torch.randn(B, Hq, D, device="cuda", dtype=torch.bfloat16)
    ref = pool.cache.decode(q, table, lens, 640)
    side = torch.cuda.Stream()
    words = pool.cache.workspace_bytes(B, Hq) // 4
    torch.cuda.synchronize()
    outs, fills = [], []
    for i in range(60):
        outs.append(pool.cache.decode(q, table, lens, 640, stream=side))
        fills.append(torch.full((words,), float(i), device="cuda"))
        if i % 7 == 6:
            assert all(bool((f == j + 7 * (i // 7)).all()) for j, f in enumerate(fills))
            fills = []
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_selections_and_contiguous_decodes_on_a_given_stream_use_memory_of_that_stream():
    B, H, G, T = 64, 8, 4, 1024
    cache = native.KVQCache(B, H, T, 4, 4)
    paged = native.PagedKVQCache(4, 4096, 4, 4)
    q = torch.randn(B, H * G, D, device="cuda", dtype=torch.bfloat16)
    wide = torch.randn(128, 4096, D, device="cuda", dtype=torch.bfloat16)
    lens = i32(np.full(B, T))
    mask, out = cache.select(q, 20), torch.empty(B, H * G, D, device="cuda")
    side = torch.cuda.Stream()
    for call in (lambda: cache.decode(q, lens, T, stream=side), lambda: cache.decode(q, lens, T, mask, out=out, stream=side),
                 lambda: cache.decode_select(q, lens, T, 20, stream=side), lambda: cache.select(q, 20, stream=side),
                 lambda: cache.select_at(q, lens, 20, stream=side), lambda: paged.select(wide, 20, stream=side)):
        streams = new_segments(call)
        assert streams and all(s == side.cuda_stream for s in streams)


@pytest.mark.parametrize("stream", ["x", 1.5])
def test_a_stream_that_is_none_is_refused(stream):
    cache = native.PagedKVQCache(2, 1, 4, 4)
    fast = native._binding()
    with pytest.raises((TypeError, ValueError)):
        fast.gather(cache._at, cache.H, cache._dev, i32([0]), native.KVQ_F32, 0, None, None, stream)


# ------------------------------------------------------------- planning
def test_plans_of_two_threads_with_batches_of_different_size():
    # each batch asks for its own amount of shared memory (over 48 KB); neither call may narrow the other's
    import threading
    failed = []

    def work(B, stream):
        try:
            torch.cuda.set_device(0)
            p = native.PagePlanner(4 * B, 64)
            args = [i32(np.zeros(B)), i32(np.ones(B)), i32(np.full((B, 2), -1)), i32(np.arange(4 * B)), i32([4 * B])]
            out = native.PagePlan(*(torch.zeros(m, dtype=torch.int32, device="cuda") for m in (B, B, B + 1, B, 1)))
            torch.cuda.synchronize()
            for _ in range(3000):
                p.plan(*args, B, out=out, stream=stream)
            stream.synchronize()
            assert int(out.free_count) == 3 * B and out.seq_lens.eq(1).all()
        except Exception as e:  # noqa: BLE001
            failed.append((B, e))

    threads = [threading.Thread(target=work, args=(B, torch.cuda.Stream())) for B in (8192, 3100, 5000, 4000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_plan_gives_no_slot_on_a_page_outside_the_pool():
    # a served request whose partly filled page is none: its tokens on that page get slot -1 (their positions
    # stand), wherever page * page_tokens lands in 32 bits; tokens on its other pages are as always
    P, num = 64, 8
    for bad in (-1, -2 ** 31, num, 1 << 26, (1 << 26) + 3, 2 ** 31 - 1):
        table = i32([[bad, -1], [5, -1]])
        p = native.PagePlanner(num, P).plan(i32([10, 10]), i32([60, 2]), table, i32([0, 1, 2, 3, 4, 6, 7, -1]), i32([7]), 70)
        assert p.seq_lens.tolist() == [70, 12] and int(p.free_count) == 6
        assert p.positions.tolist() == list(range(10, 70)) + [10, 11] + [-1] * 8
        assert p.slots.tolist() == [-1] * 54 + [7 * P + i for i in range(6)] + [5 * P + 10, 5 * P + 11] + [-1] * 8, bad


# ------------------------------------------------------------- small values
@pytest.mark.parametrize("vb", [4, 2])
@pytest.mark.parametrize("std", [2e-4, 5e-5, 2e-6, 150.0, 4000.0])
@pytest.mark.parametrize("G,dtype", [(4, "bf16"), (8, "bf16"), (4, "f16"), (16, "f16"), (4, "f32"), (8, "f32")])
def test_decode_accuracy_does_not_depend_on_the_values_magnitude(vb, std, G, dtype):
    # one token holds some 3/4 of the weight, 131071 others share the rest: products of their
    # probabilities and scales span 2^-19 below the largest, wherever the scales lie.  As many
    # requests as the decode has warps, over the same pages: a request is not cut into short pieces
    num, P, n, B = 32, 4096, 131072, 148 * 16
    pool = Pool(3, 1, 1, 64, 4, vb, 0, rot=0)
    L = pool.lay
    r = np.random.RandomState(int(1e7 * std) % 1000 + vb)
    raw = np.zeros((num * P // BT, L.bytes), np.uint8)
    half = lambda x: np.asarray(x).astype(np.float16).view(np.uint8)  # noqa: E731
    raw[:, L.vc:L.vs] = r.randint(0, 256, (len(raw), L.vs - L.vc))
    step = 4 * std / ((1 << vb) - 1)
    raw[:, L.vs:L.vs + 512] = half(step * r.uniform(0.8, 1.2, (len(raw), 256)))
    raw[:, L.vz:L.vz + 512] = half(-2 * std * r.uniform(0.5, 1.5, (len(raw), 256)))
    top = 4097  # the token with the weight: its keys are constants, all others zero
    for grp in range(4):
        at = L.kz + L.tables()["kz"][top % BT, grp]
        raw[top // BT, at:at + 2] = half([13.0 / 128 * math.sqrt(D)])
    raw = raw.reshape(num, 1, P // BT, L.bytes)
    cache = native.PagedKVQCache(num, 1, 4, vb, page_tokens=P, rotate_k=0)
    cache.pages.copy_(torch.from_numpy(raw.reshape(-1)))
    kh, vh = held(cache, L, 0)
    q = torch.ones(B, G, D, device="cuda", dtype=TYPES[dtype])
    out = cache.decode(q, i32(np.tile(np.arange(num), (B, 1))), i32(np.full(B, n)), n)
    o = attention(np.ones(D), kh, vh, 1 / math.sqrt(D))
    bound = output_bound(o, np.ones(D), kh, vh, 1 / math.sqrt(D), dtype)
    if dtype == "f16":
        bound = bound + 2.0 ** -25  # half a step of the type's subnormals
    if dtype == "f32":  # a lane adds its 8 tokens of a tile one after another, n / 8 sums that are each off by up
        # to 2^-24 of what they hold, in the numerator and in the divisor
        bound = bound + 2 * (n / 8) * 2.0 ** -24 * np.abs(vh).max()
    for b in (0, 1, B // 2, B - 1):
        for j in range(G):
            err = np.abs(out[b, j].double().cpu().numpy() - o)
            assert (err <= bound).all(), (b, j, float((err / bound).max()))


@pytest.mark.parametrize("vb", [4, 2])
@pytest.mark.parametrize("G,dtype", [(4, "bf16"), (8, "bf16"), (16, "bf16"), (4, "f16"), (8, "f16"), (4, "f32")])
@pytest.mark.parametrize("large,n", [(3000.0, 4), (60000.0, 4), (60000.0, 300)])
def test_a_token_of_large_values_and_no_weight_takes_no_accuracy_from_the_others(vb, G, dtype, large, n):
    # the token's score is some 60 nats below every other's: its weight is 0 in any of the types, and
    # the outputs are those of the request without it (its own part, below 1e6 * e^-60, is nothing).
    # As many requests as the decode has warps, over the same pages: each has one warp
    P, B = 64, 148 * 16
    L = Layout(4, vb, 0)
    r = np.random.RandomState(vb)
    raw = np.zeros((5, L.bytes), np.uint8)
    half = lambda x: np.asarray(x).astype(np.float16).view(np.uint8)  # noqa: E731
    raw[:, :L.ks] = r.randint(0, 256, (5, L.ks))
    raw[:, L.ks:L.kz] = half(r.uniform(0.01, 0.03, (5, 256)))
    raw[:, L.vc:L.vs] = r.randint(0, 256, (5, L.vs - L.vc))
    raw[:, L.vs:L.vz] = half(r.uniform(0.02, 0.2, (5, 256)))
    raw[:, L.vz:] = half(r.uniform(-1.0, -0.1, (5, 256)))
    for grp in range(4):
        at = L.vs + L.tables()["s"][2, grp]
        raw[0, at:at + 2] = half([large])
        at = L.kz + L.tables()["kz"][2, grp]
        raw[0, at:at + 2] = half([-60.0 / 128 * math.sqrt(D)])
    cache = native.PagedKVQCache(5, 1, 4, vb, page_tokens=P, rotate_k=0)
    cache.pages.copy_(torch.from_numpy(raw.reshape(-1)))
    kh, vh = (np.delete(x[:n], 2, 0) for x in held(cache, L, 0))
    q = torch.ones(B, G, D, device="cuda", dtype=TYPES[dtype])
    out = cache.decode(q, i32(np.tile(np.arange(5), (B, 1))), i32(np.full(B, n)), n)
    o = attention(np.ones(D), kh, vh, 1 / math.sqrt(D))
    bound = output_bound(o, np.ones(D), kh, vh, 1 / math.sqrt(D), dtype)
    for b in (0, B // 2, B - 1):
        for j in range(G):
            err = np.abs(out[b, j].double().cpu().numpy() - o)
            assert (err <= bound).all(), (b, j, float((err / bound).max()))


# ------------------------------------------------------------- one definition of the scale
@pytest.mark.parametrize("kb,vb,rot,ch0,rotv,clip,dtype", [(4, 4, 1, 0, 0, 1.0, "bf16"), (2, 4, 0, 1, 1, 0.92, "f32"),
                                                           (4, 2, 1, 1, 0, 0.9, "f16")])
def test_append_of_many_rows_holds_the_oracles_values_in_every_row(kb, vb, rot, ch0, rotv, clip, dtype):
    # the oracle's scale is the quotient (max - min) / L, which some 84 of a million 4-bit groups tell from a
    # product with 1 / L; rows next to a rounding boundary are no exception
    from test_gpu_paged import oracle_cache, rows
    n, H, P = 16384, 8, 256
    cache = native.PagedKVQCache(n // P, H, kb, vb, page_tokens=P, rotate_k=rot, keep_ch0=ch0, rotate_v=rotv, v_clip=clip)
    k, v = rows(31, n, H, dtype)
    slots = i32(np.random.RandomState(1).permutation(n))
    cache.append(k, v, slots)
    kd, vd = cache.gather(slots, torch.float32, rotate_back=False)
    oc = oracle_cache(k, v, kb, vb, rot, ch0, rotv, clip)
    for h in range(H):
        kh, vh = oc.dequantize(0, h, 0, n)
        for got, want in ((kd, kh), (vd, vh)):
            assert np.array_equal(got[:, h].cpu().numpy(), want.astype(np.float32)), h


# ------------------------------------------------------------- probabilities
@pytest.mark.parametrize("kb,vb", [(4, 4), (4, 2), (2, 2)])
@pytest.mark.parametrize("G", [1, 4, 8, 16])
@pytest.mark.parametrize("lens", [[1], [2, 7, 64, 65, 200]])
def test_the_divisor_holds_the_same_rounded_probabilities_as_the_sums(kb, vb, G, lens):
    # Value zeros near 1000 beside steps of some 3: an fp16 probability is off by up to 2^-11 of
    # itself, but the sum with the zeros and the divisor take the same one, so what is left is
    # P' = p * scale, 2^-11 of scale times the codes' distance from their middle, beside the final rounding.
    pool = Pool(kb * 7 + vb, 16, 1, 64, kb, vb, 0)
    L = pool.lay
    half = lambda x: np.asarray(x, np.float16).view(np.uint8)  # noqa: E731
    r = np.random.RandomState(5)
    shape = pool.raw[..., L.vs:L.vs + 512].shape
    m = shape[0] * 256
    pool.raw[..., L.vs:L.vs + 512] = half(r.uniform(1.5, 3.5, m)).reshape(shape)
    pool.raw[..., L.vz:L.vz + 512] = half(np.full(m, 1040.0)).reshape(shape)
    pool.cache.pages.copy_(torch.from_numpy(pool.raw.reshape(-1)))
    # scores: the fp32 sums' 2^-20 of |q| |k| scale, as in output_bound, times the values' spread about their mean
    order = np.random.RandomState(17).permutation(16)
    out, _ = decode_case(pool, G, "f16", lens, pad_pages=0)
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randn(len(lens), G, D, device="cuda", generator=g).half()
    at = 0
    for b, n in enumerate(lens):
        pages = order[at:at + -(-n // 64)]
        at += len(pages)
        k, v = (x[:n] for x in pool.values(pages, 0))
        for j in range(G):
            qr = hadamard() @ q[b, j].double().cpu().numpy()
            o = attention(qr, k, v, 1 / math.sqrt(D))
            spread = np.ptp(v)
            eps_s = 2.0 ** -20 * np.linalg.norm(qr) * np.linalg.norm(k, axis=1).max() / math.sqrt(D)
            bound = np.abs(o) * (2.0 ** -11 + 2.0 ** -20) + 3.5 * (1 << (vb - 1)) * 2.0 ** -11 + 2 * eps_s * spread
            err = np.abs(out[b, j].double().cpu().numpy() - o)
            assert (err <= bound).all(), (b, j, float((err / bound).max()))


# ------------------------------------------------------------- one long request among short ones
@pytest.mark.parametrize("G,dtype", [(4, "bf16"), (8, "f16"), (16, "f32")])
def test_decode_of_one_long_request_among_short_ones(G, dtype):
    # nearly all ranges belong to one request: its rows join hundreds of partials, the others' one or two
    lens = [200] * 30 + [40000] + [1, 0, 65] * 11
    pool = Pool(17, 400, 1, 256, 4, 4, 0)
    _, check = decode_case(pool, G, dtype, lens, seed=5)
    for b in (0, 29, 30, 31, 33, len(lens) - 1):
        for j in {0, G - 1}:
            check(b, j)


def test_captured_decodes_without_a_workspace_on_a_given_stream():
    # two graphs, each with the workspace and the output of its own memory, replayed in turn and beside eager calls
    pool = Pool(23, 40, 2, 64, 4, 4, 0)
    table, lens = i32(np.random.RandomState(2).permutation(40).reshape(4, 10)), i32([640, 33, 200, 64])
    qs = [torch.randn(4, 8, D, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    refs = [pool.cache.decode(q, table, lens, 640) for q in qs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(pool.cache.decode(q, table, lens, 640, stream=side))
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        eager = pool.cache.decode(qs[0], table, lens, 640)
        torch.cuda.synchronize()
        assert torch.equal(eager, refs[0]) and all(torch.equal(o, r) for o, r in zip(outs, refs))
    del graphs
