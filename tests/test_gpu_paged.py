"""The paged cache on the GPU against plain implementations: planning request by
request, appended bytes against the oracle, dense rows, and decode attention in
64 bits."""
import math

import numpy as np
import pytest
import torch

from oracle import oracle as orc
from paged_testlib import BT, D, Layout, attention, hadamard, output_bound, plan
from quantized_attention_kvq_b200 import native

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# --------------------------------------------------------------------- planning
def run_plan(num, P, ctx, new, done, table, free, count, n_slots, in_place=False):
    p = native.PagePlanner(num, P)
    t, f, c, ln = i32(table), i32(free), i32([count]), i32(ctx)
    out = None
    if in_place:
        e = lambda n: torch.full((n,), 77, dtype=torch.int32, device="cuda")  # noqa: E731
        out = native.PagePlan(e(n_slots), e(n_slots), e(len(ctx) + 1), ln, c)
    r = p.plan(ln, i32(new), t, f, c, n_slots, done=None if done is None else i32(done), out=out)
    torch.cuda.synchronize()
    return dict(slots=r.slots, positions=r.positions, cu_new=r.cu_new, seq_lens=r.seq_lens, table=t, free=f,
                count=r.free_count)


def check_plan(got, want):
    for k, v in want.items():
        g = got[k].cpu().numpy()
        assert np.array_equal(g, np.asarray(v).reshape(g.shape)), k


@pytest.mark.parametrize("seed,B,P,max_pages,short,n_cut", [
    (1, 1, 64, 1, 0, 0), (2, 1, 64, 3, 0, 0), (3, 7, 64, 20, 0, 0), (4, 7, 128, 5, 9, 0), (5, 64, 64, 40, 30, 0),
    (6, 511, 64, 12, 100, 0), (7, 513, 256, 6, 0, 700), (8, 3000, 64, 9, 500, 0), (9, 8192, 64, 4, 0, 3000),
    (10, 40, 64, 90, 0, 0), (11, 33, 4096, 2, 3, 0), (12, 700, 64, 3, 40, 10**6)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_requests_taken_one_by_one(seed, B, P, max_pages, short, n_cut, in_place):
    r = np.random.RandomState(seed)
    most = max_pages * P
    ctx = r.randint(0, most + 1, B)
    ctx[r.rand(B) < 0.2] = 0
    new = np.where(r.rand(B) < 0.6, 1, r.randint(0, max(2, min(most, 3 * P)), B))
    new[r.rand(B) < 0.1] = 0
    new[r.rand(B) < 0.03] = most + 1  # cannot fit its row
    ctx[r.rand(B) < 0.03] = -5
    new[r.rand(B) < 0.03] = -1
    done = (r.rand(B) < 0.25).astype(np.int32)
    new[(done > 0) & (r.rand(B) < 0.5)] = 0
    held = [-(-max(int(c), 0) // P) for c in ctx]
    extra = sum(-(-(max(int(c), 0) + max(int(n), 0)) // P) for c, n in zip(ctx, new)) - sum(held)
    num = max(1, sum(held) + max(extra - short, 0) + 2)
    perm = r.permutation(num).astype(np.int32)
    table = np.full((B, max_pages), -7, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += h
    free = np.full(num, -3, np.int32)
    free[:num - at] = perm[at:]
    n_slots = max(0, int(np.maximum(new, 0).sum()) + 5 - n_cut)
    args = (num, P, ctx, new, done if seed != 10 else None, table, free, num - at, n_slots)
    check_plan(run_plan(*args, in_place=in_place), plan(*args))


def test_plan_with_no_slots_and_an_empty_pool():
    table = np.full((3, 2), -1, np.int32)
    args = (4, 64, [0, 0, 0], [1, 0, 0], None, table, np.zeros(4, np.int32), 0, 0)
    check_plan(run_plan(*args), plan(*args))


# --------------------------------------------------------------------- appending
def rows(seed, n, H, dtype, Hq=0):
    """k, v [n, H, 128] as slices of one [n][Hq + 2H] projection, with a few strong channels."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(n, Hq + 2 * H, D, device="cuda", generator=g)
    x[:, Hq:Hq + H, 3] *= 12
    x[:, Hq:Hq + H, 77] *= 7
    x = x.to(TYPES[dtype])
    return x[:, Hq:Hq + H], x[:, Hq + H:]


def oracle_cache(k, v, kb, vb, rot, ch0, rotv, clip):
    """The oracle's cache of one sequence holding the tokens in order; its `near` flags the rows
    [which][head][token] with a value within 1e-6 of a rounding boundary.  The paged append forms its scale
    by a product that is one unit in the last place from the oracle's quotient, so such rows may differ."""
    n, H = k.shape[0], k.shape[1]
    oc = orc.Cache(1, H, D, -(-n // 128) * 128, kb, vb, rot, ch0, rotv, clip)
    f = lambda x: np.ascontiguousarray(x.float().cpu().numpy().transpose(1, 0, 2))[None]  # noqa: E731
    st = oc.append(f(k), f(v), 0, want_exempt=True)
    oc.near = (st["k_row_exempt"][0], st["v_row_exempt"][0])
    return oc


def token_places(slots, P):
    s = np.asarray(slots)
    return s // P, (s % P) // BT, s % BT


@pytest.mark.parametrize("kb,vb,rot,ch0,rotv,clip,dtype,H,P", [
    (4, 4, 1, 0, 0, 1.0, "bf16", 2, 64), (4, 2, 1, 1, 0, 1.0, "bf16", 1, 128), (2, 2, 1, 1, 1, 0.92, "f16", 3, 64),
    (2, 4, 0, 0, 1, 0.92, "f32", 2, 256), (4, 4, 1, 1, 1, 1.0, "f32", 2, 64)])
def test_appended_tokens_hold_the_oracles_bits(kb, vb, rot, ch0, rotv, clip, dtype, H, P):
    n, num = 301, 9
    lay = Layout(kb, vb, ch0)
    cache = native.PagedKVQCache(num, H, kb, vb, page_tokens=P, rotate_k=rot, keep_ch0=ch0, rotate_v=rotv, v_clip=clip)
    r = np.random.RandomState(n + kb)
    fill = torch.from_numpy(r.randint(0, 256, cache.pages.numel()).astype(np.uint8)).cuda()
    cache.pages.copy_(fill)
    # any distinct slots, some tokens skipped (padding and slots beyond the pool)
    slots = r.permutation(num * P)[:n].astype(np.int64)
    skip = r.rand(n) < 0.1
    slots[skip] = np.where(r.rand(skip.sum()) < 0.5, -1, num * P + r.randint(0, 99, skip.sum()))
    k, v = rows(5, n, H, dtype, Hq=3)
    if dtype == "bf16":  # a row of equal values: scale 0
        k[4], v[4] = 1.5, -2.0
    cache.append(k, v, i32(slots))
    torch.cuda.synchronize()
    got = cache.pages.cpu().numpy().reshape(num, H, P // BT, lay.bytes)
    oc = oracle_cache(k, v, kb, vb, rot, ch0, rotv, clip)
    want = fill.cpu().numpy().reshape(got.shape).copy()
    page, blk, t = token_places(slots, P)
    tb = lay.tables()
    s16 = lambda a, i: a.reshape(-1)[i]  # noqa: E731
    differ = 0
    for j in range(n):
        if skip[j]:
            continue
        for h in range(H):
            w = want[page[j], h, blk[j]]
            for which, bits, name in ((0, kb, "k"), (1, vb, "v")):
                codes = oc.unpack(0, h, j, which)
                place = tb[name][t[j]]
                for byte in np.unique(place[:, 0]):
                    w[byte] = sum(int(codes[c]) << int(place[c, 1]) for c in np.nonzero(place[:, 0] == byte)[0])
            N = oc.capacity
            for grp in range(4):
                ki = ((h * (N // 128) + j // 128) * 4 + grp) * 128 + j % 128
                vi = (h * N + j) * 4 + grp
                for base, at, val in ((lay.ks, tb["s"], s16(oc.k_scales, 2 * ki)), (lay.kz, tb["kz"], s16(oc.k_scales, 2 * ki + 1)),
                                      (lay.vs, tb["s"], s16(oc.v_scales, 2 * vi)), (lay.vz, tb["s"], s16(oc.v_scales, 2 * vi + 1))):
                    a = base + at[t[j], grp]
                    w[a], w[a + 1] = int(val) & 255, int(val) >> 8
            if ch0:
                val = int(oc.k_ch0[h * N + j])
                w[lay.k0 + 2 * t[j]], w[lay.k0 + 2 * t[j] + 1] = val & 255, val >> 8
            g = got[page[j], h, blk[j]]
            for which, (first, last, name, zname) in enumerate(((0, lay.k0, "k", "kz"), (lay.vc, lay.bytes, "v", "s"))):
                base = (lay.ks, lay.kz) if which == 0 else (lay.vs, lay.vz)
                at = np.concatenate([tb[name][t[j]][:, 0]] + [b + tb[x][t[j]] + o for b, x in zip(base, ("s", zname)) for o in (0, 1)])
                if oc.near[which][h, j] and not np.array_equal(w[at], g[at]):
                    assert (first <= at).all() and (at < last).all()
                    w[at] = g[at]
                    differ += 1
    assert differ <= 0.01 * 2 * n * H + 1
    assert np.array_equal(got, want)  # the tokens' bytes are the oracle's, every other byte is as it was


@pytest.mark.parametrize("kb,vb", [(4, 4), (4, 2), (2, 4), (2, 2)])
@pytest.mark.parametrize("start,P", [(0, 64), (1, 64), (3, 128), (6, 64), (61, 192)])
def test_tokens_in_a_row_hold_the_same_bytes_as_one_by_one(kb, vb, start, P):
    # a request's consecutive tokens from any place in their page, over page ends, with a
    # hole and a second request: the order in which a call lists them does not show
    H, num, n = 2, 12, 257
    table = np.array([7, 2, 3, 11, 0, 9])
    pos = start + np.arange(n)
    slots = table[pos // P] * P + pos % P
    slots[100] = -1
    slots[200:] = np.setdiff1d(np.arange(num * P), slots)[5:5 + n - 200]
    k, v = rows(9 + start, n, H, "bf16")
    perm = np.random.RandomState(start).permutation(n)
    pools = []
    for order in (np.arange(n), perm):
        cache = native.PagedKVQCache(num, H, kb, vb, page_tokens=P, keep_ch0=1)
        cache.pages.fill_(0x5A)
        o = torch.from_numpy(order).cuda()
        cache.append(k[o].contiguous(), v[o].contiguous(), i32(slots[order]))
        pools.append(cache.pages)
    one = native.PagedKVQCache(num, H, kb, vb, page_tokens=P, keep_ch0=1)
    one.pages.fill_(0x5A)
    for j in range(n):
        one.append(k[j:j + 1], v[j:j + 1], i32(slots[j:j + 1]))
    assert torch.equal(pools[0], one.pages) and torch.equal(pools[1], one.pages)


def test_append_one_token_and_none():
    cache = native.PagedKVQCache(2, 1, 4, 4)
    before = cache.pages.clone()
    k, v = rows(1, 1, 1, "bf16")
    cache.append(k[:0], v[:0], i32([]))
    cache.append(k, v, i32([-1]))
    assert torch.equal(cache.pages, before)
    cache.append(k, v, i32([127]))
    kd, vd = cache.gather(i32([127, 0]), torch.float32, rotate_back=False)
    oc = oracle_cache(k, v, 4, 4, 1, 0, 0, 1.0)
    kh, vh = oc.dequantize(0, 0, 0, 1)
    assert np.array_equal(kd[0, 0].cpu().numpy(), kh[0].astype(np.float32))
    assert np.array_equal(vd[0, 0].cpu().numpy(), vh[0].astype(np.float32))
    assert not kd[1].any() and not vd[1].any()


# --------------------------------------------------------------------- filled pools
class Pool:
    """A pool of random blocks (codes uniform, scales and zeros of plausible sizes), and its values in 64 bits."""

    def __init__(self, seed, num, H, P, kb, vb, ch0, rot=1, rotv=0):
        self.lay, self.P, self.H = Layout(kb, vb, ch0), P, H
        r = np.random.RandomState(seed)
        nb = P // BT
        raw = r.randint(0, 256, (num, H, nb, self.lay.bytes)).astype(np.uint8)
        half = lambda x: x.astype(np.float16).view(np.uint8)  # noqa: E731
        L = self.lay
        for a, lo, hi in ((L.ks, 0.02, 0.3), (L.vs, 0.02, 0.4)):
            raw[..., a:a + 512] = half(r.uniform(lo, hi, (num, H, nb, 256)) * np.exp(r.randn(num, H, nb, 256) * 0.3))
        for a, m in ((L.kz, -1.2), (L.vz, -1.0)):
            raw[..., a:a + 512] = half(m + 0.5 * r.randn(num, H, nb, 256))
        if ch0:
            f = (4 * r.randn(num, H, nb, BT)).astype(np.float32).view(np.uint32) >> 16
            raw[..., L.k0:L.k0 + 128] = f.astype(np.uint16).view(np.uint8)
        self.raw = raw
        self.cache = native.PagedKVQCache(num, H, kb, vb, page_tokens=P, rotate_k=rot, keep_ch0=ch0, rotate_v=rotv)
        self.cache.pages.copy_(torch.from_numpy(raw.reshape(-1)))

    def values(self, pages, h):
        """[len(pages) * P][128] keys and values of a page list."""
        kv = [self.lay.values(self.raw[p, h, b]) for p in pages for b in range(self.P // BT)]
        kv.append((np.zeros((0, D)), np.zeros((0, D))))
        return np.concatenate([x[0] for x in kv]), np.concatenate([x[1] for x in kv])


@pytest.mark.parametrize("kb,vb,ch0,dtype,back,rot,rotv", [
    (4, 4, 0, "f32", 0, 1, 1), (4, 2, 1, "f32", 1, 1, 0), (2, 4, 1, "bf16", 1, 0, 1), (2, 2, 0, "f16", 1, 1, 1),
    (4, 4, 1, "bf16", 0, 1, 0)])
def test_gather_reads_what_the_blocks_hold(kb, vb, ch0, dtype, back, rot, rotv):
    num, H, P = 5, 3, 128
    pool = Pool(kb * 10 + vb, num, H, P, kb, vb, ch0, rot, rotv)
    r = np.random.RandomState(4)
    slots = r.randint(0, num * P, 217)  # repetitions among them
    slots[::13] = -1
    slots[5], slots[6] = num * P, 2 ** 31 - 1
    k, v = pool.cache.gather(i32(slots), TYPES[dtype], rotate_back=bool(back))
    k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
    ok = (slots >= 0) & (slots < num * P)
    assert not k[~ok].any() and not v[~ok].any()
    page, blk, t = token_places(slots, P)
    Hm, half = hadamard(), torch.finfo(TYPES[dtype]).eps / 2
    for h in range(H):
        for j in np.nonzero(ok)[0]:
            kb_, vb_ = pool.lay.values(pool.raw[page[j], h, blk[j]])
            for got, x, turned in ((k, kb_[t[j]], back and rot), (v, vb_[t[j]], back and rotv)):
                want = Hm @ x if turned else x
                # one rounding of scale * code + zero in fp32 (2^-24), 7 fp32 butterfly sums and a product
                # (8 x 2^-24 of the row's norm), the type's rounding
                bound = 2.0 ** -24 * np.abs(want) + np.abs(want) * half * 1.01
                if turned:
                    bound = bound + 9 * 2.0 ** -24 * np.linalg.norm(x)
                bound = bound + (2.0 ** -25 if dtype == "f16" else 0)  # fp16 subnormals
                assert (np.abs(got[j, h] - want) <= bound).all()


def test_gather_of_one_side_only():
    pool = Pool(3, 3, 2, 64, 4, 2, 0)
    slots = i32([3, 70, 5])
    k, v = pool.cache.gather(slots, torch.float32)
    L = native.lib()
    only = torch.zeros_like(v)
    assert L.kvq_paged_gather(pool.cache._ref, slots.data_ptr(), 3, native.KVQ_F32, 1, None, only.data_ptr(),
                              torch.cuda.current_stream().cuda_stream) == native.KVQ_OK
    assert torch.equal(only, v)
    only.zero_()
    assert L.kvq_paged_gather(pool.cache._ref, slots.data_ptr(), 3, native.KVQ_F32, 1, only.data_ptr(), None,
                              torch.cuda.current_stream().cuda_stream) == native.KVQ_OK
    assert torch.equal(only, k)


# --------------------------------------------------------------------- decode
def decode_case(pool, G, dtype, lens, seed=0, keep=None, scale=1 / math.sqrt(D), q_mul=1.0, pad_pages=2, max_len=None,
                q_wide=0, bad=()):
    """Decode over shuffled block tables; returns (output, per-row check of it)."""
    H, P, B = pool.H, pool.P, len(lens)
    num = pool.cache.num_pages
    r = np.random.RandomState(seed + 17)
    n_pg = [-(-n // P) for n in lens]
    perm = r.permutation(num)
    assert sum(n_pg) <= num
    table = np.full((B, max(n_pg + [1]) + pad_pages), -1, np.int64)
    at = 0
    for b, m in enumerate(n_pg):
        table[b, :m] = perm[at:at + m]
        at += m
    for b, i, page in bad:
        table[b, i] = page
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = (q_mul * torch.randn(B, H * G + q_wide, D, device="cuda", generator=g)).to(TYPES[dtype])[:, :H * G]
    mask, keep_ch = None, np.ones((B, H, D))
    if keep is not None:
        words = np.array([[sum(1 << int(x) for x in r.permutation(32)[:keep]) for _ in range(H)] for _ in range(B)], np.uint64)
        mask = torch.from_numpy(words.astype(np.uint32).view(np.int32)).cuda()
        keep_ch = ((words[..., None] >> np.arange(32).astype(np.uint64)) & np.uint64(1)).astype(float).repeat(4, 2)
    out = pool.cache.decode(q, i32(table), i32(lens), max(lens + [0]) if max_len is None else max_len, mask=mask,
                            softmax_scale=scale)
    torch.cuda.synchronize()
    Hm = hadamard()

    def check(b, j):
        h = j // G
        n = max(0, min(lens[b], max_len if max_len is not None else lens[b]))
        pages = table[b, :-(-n // P)]
        good = (pages >= 0) & (pages < num)
        k, v = pool.values(np.where(good, pages, 0), h)
        on = good.repeat(P)[:n]
        k, v = k[:n][on], v[:n][on]
        qr = q[b, j].double().cpu().numpy()
        qr = Hm @ qr if pool.cache.desc.rotate_k else qr
        o = attention(qr, k, v, scale, keep_ch[b, h])
        bound = output_bound(o, qr, k, v, scale, dtype)
        if pool.cache.desc.rotate_v:  # rows rotated back: errors add up over the row
            bound = np.full(D, np.linalg.norm(bound)) + 2.0 ** -21 * np.linalg.norm(o)
            o = Hm @ o
            bound = bound + np.abs(o) * torch.finfo(TYPES[dtype]).eps / 2
        got = out[b, j].double().cpu().numpy()
        err = np.abs(got - o)
        assert (err <= bound).all(), (b, j, n, float((err / np.maximum(bound, 1e-300)).max()))

    return out, check


@pytest.mark.parametrize("kb,vb", [(4, 4), (4, 2), (2, 4), (2, 2)])
@pytest.mark.parametrize("G,dtype", [(1, "bf16"), (3, "f32"), (4, "f16"), (5, "bf16"), (8, "bf16"), (8, "f32"), (16, "f16"),
                                     (13, "f32")])
@pytest.mark.parametrize("ch0", [0, 1])
def test_decode_matches_attention_in_64_bits(kb, vb, G, dtype, ch0):
    lens = [0, 1, 63, 64, 65, 129, 500]
    pool = Pool(kb + vb, 16, 2, 64, kb, vb, ch0)
    out, check = decode_case(pool, G, dtype, lens, seed=G)
    assert not out[0].any()
    for b in range(len(lens)):
        for j in {0, G - 1, G, 2 * G - 1}:
            check(b, j)


@pytest.mark.parametrize("kb,vb,P,rot,rotv,keep,dtype", [
    (4, 4, 128, 1, 1, None, "bf16"), (2, 2, 256, 1, 1, 19, "f32"), (4, 2, 64, 0, 0, 24, "bf16"), (2, 4, 128, 0, 1, 1, "f16"),
    (2, 2, 64, 1, 0, 31, "bf16"), (4, 4, 64, 1, 0, 0, "f32"), (4, 2, 4096, 1, 0, 8, "f32")])
def test_decode_masks_page_sizes_and_rotations(kb, vb, P, rot, rotv, keep, dtype):
    lens = [P - 1, 2 * P, 1, 3 * P // 2]
    pool = Pool(P + kb, 8, 3, P, kb, vb, 1, rot, rotv)
    _, check = decode_case(pool, 4, dtype, lens, keep=keep, q_wide=3)
    for b in range(4):
        for j in (0, 3, 6, 11):
            check(b, j)


@pytest.mark.parametrize("G,dtype,B", [(4, "bf16", 1), (8, "f32", 1), (1, "f16", 2), (16, "bf16", 1)])
def test_decode_long_sequence_joins_many_partials(G, dtype, B):
    pool = Pool(8, 40 * B + 1, 1, 256, 4, 4, 0)
    _, check = decode_case(pool, G, dtype, [40 * 256 - 3] * B)
    for b in range(B):
        check(b, 0)
        check(b, G - 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_sharp_and_flat_queries(dtype):
    # scores of a hundred and more (one token takes all), and all equal
    pool = Pool(21, 12, 2, 64, 4, 4, 0)
    for mul in (40.0, 1e-6, 0.0):
        _, check = decode_case(pool, 4, dtype, [700], q_mul=mul)
        for j in range(8):
            check(0, j)


def test_decode_many_short_requests():
    lens = [int(x) for x in np.random.RandomState(3).randint(0, 130, 700)]
    pool = Pool(5, 2100, 2, 64, 4, 2, 0)
    out, check = decode_case(pool, 2, "bf16", lens)
    for b in range(0, 700, 37):
        for j in range(4):
            check(b, j)
    assert not out[[b for b, n in enumerate(lens) if n == 0]].any()


def test_decode_length_is_clamped_and_max_len_zero_gives_zero_rows():
    pool = Pool(6, 12, 1, 64, 4, 4, 0)
    _, check = decode_case(pool, 4, "bf16", [300, 40, 64], max_len=100)
    for b in range(3):
        check(b, 1)
    out, _ = decode_case(pool, 4, "bf16", [300, 40, 64], max_len=0)
    assert not out.any()


def test_decode_pages_outside_the_pool_take_no_part():
    pool = Pool(7, 12, 2, 64, 2, 4, 1)
    _, check = decode_case(pool, 4, "f32", [300, 200, 64], bad=((0, 1, -1), (0, 4, 12), (1, 0, 2 ** 31 - 1), (2, 0, -2 ** 31)))
    for b in range(2):
        for j in (0, 7):
            check(b, j)
    out, _ = decode_case(pool, 4, "f32", [300, 200, 64], bad=((2, 0, -2 ** 31),))
    assert not out[2].any()  # nothing of it is left


def test_decode_ignores_bytes_behind_the_last_token():
    pool = Pool(9, 4, 1, 64, 4, 4, 1)
    lay, n = pool.lay, 64 + 37
    out, _ = decode_case(pool, 4, "bf16", [n], seed=2)
    raw = pool.raw.copy()
    for t in range(37, 64):  # not-a-number and infinite scales, zeros and channel 0 behind every block's 37th token
        for g in range(4):
            for base, tab in ((lay.ks, "s"), (lay.kz, "kz"), (lay.vs, "s"), (lay.vz, "s")):
                a = base + lay.tables()[tab][t, g]
                raw[..., a:a + 2] = (0, 0x7E) if t % 2 else (0, 0x7C)
        raw[..., lay.k0 + 2 * t:lay.k0 + 2 * t + 2] = (0xC0, 0x7F)
    order = np.random.RandomState(2 + 17).permutation(4)
    keep = pool.raw[order[0]].copy()
    raw[order[0]] = keep  # the first page is whole
    pool.cache.pages.copy_(torch.from_numpy(raw.reshape(-1)))
    again, _ = decode_case(pool, 4, "bf16", [n], seed=2)
    assert torch.equal(out, again)


def test_value_scales_at_the_ends_of_fp16():
    # tiny, zero and huge value scales side by side: P' stays in range, nothing overflows
    for dtype in ("bf16", "f32"):
        pool = Pool(11, 9, 1, 64, 4, 4, 0)
        L = pool.lay
        half = lambda x: np.asarray(x, np.float16).view(np.uint8)  # noqa: E731
        n = pool.raw.shape[0] * 256
        sc = np.random.RandomState(0).choice([0.0, 6e-8, 1e-5, 0.2, 900.0, 4000.0], n)
        pool.raw[..., L.vs:L.vs + 512] = half(sc).reshape(pool.raw[..., L.vs:L.vs + 512].shape)
        pool.cache.pages.copy_(torch.from_numpy(pool.raw.reshape(-1)))
        _, check = decode_case(pool, 4, dtype, [513])
        for j in range(4):
            check(0, j)


def test_offsets_beyond_32_bits():
    # a pool of more than 4 GiB; the tokens sit in its last pages
    H, P, kb, vb = 8, 256, 4, 4
    per = 10240 * (P // BT) * H
    num = (1 << 32) // per + 40
    cache = native.PagedKVQCache(num, H, kb, vb, page_tokens=P, pages=torch.empty(num * per, dtype=torch.uint8, device="cuda"))
    n = 300
    k, v = rows(9, n, H, "bf16")
    slots = torch.arange((num - 2) * P, (num - 2) * P + n, device="cuda", dtype=torch.int32)
    cache.append(k, v, slots)
    kd, vd = cache.gather(slots, torch.float32, rotate_back=False)
    oc = oracle_cache(k, v, kb, vb, 1, 0, 0, 1.0)
    q = torch.randn(1, H * 2, D, device="cuda", dtype=torch.bfloat16)
    out = cache.decode(q, i32([[num - 2, num - 1]]), i32([n]), n)
    for h in range(H):
        kh, vh = oc.dequantize(0, h, 0, n)
        for got, x, near in ((kd, kh, oc.near[0]), (vd, vh, oc.near[1])):
            same = (got[:, h].cpu().numpy() == x.astype(np.float32)).all(1)
            assert (same | (near[h] != 0)).all() and same.mean() > 0.98
        kh, vh = kd[:, h].double().cpu().numpy(), vd[:, h].double().cpu().numpy()
        for g in range(2):
            qr = hadamard() @ q[0, 2 * h + g].double().cpu().numpy()
            o = attention(qr, kh, vh, 1 / math.sqrt(D))
            assert (np.abs(out[0, 2 * h + g].double().cpu().numpy() - o) <= output_bound(o, qr, kh, vh, 1 / math.sqrt(D), "bf16")).all()


# --------------------------------------------------------------------- the calls together
def step(cache, st):
    """One serving step: plan, append, select, decode."""
    p = cache.planner.plan(st["lens"], st["new"], st["table"], st["free"], st["count"], st["n_slots"], done=st["done"],
                           out=native.PagePlan(st["slots"], st["pos"], st["cu"], st["lens"], st["count"]))
    cache.append(st["k"], st["v"], p.slots)
    mask = cache.select(st["q"], 20, mask_out=st["mask"])
    return cache.decode(st["q"], st["table"], p.seq_lens, st["max_len"], mask=mask, out=st["out"], workspace=st["ws"])


def make_state(cache, B, H, G, max_pages, n_slots):
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    num, P = cache.num_pages, cache.page_tokens
    return dict(lens=z(B), new=z(B), done=z(B), table=z(B, max_pages) - 1, free=torch.arange(num, device="cuda", dtype=torch.int32),
                count=z(1) + num, slots=z(n_slots), pos=z(n_slots), cu=z(B + 1), n_slots=n_slots, max_len=max_pages * P,
                k=torch.zeros(n_slots, H, D, device="cuda", dtype=torch.bfloat16),
                v=torch.zeros(n_slots, H, D, device="cuda", dtype=torch.bfloat16),
                q=torch.zeros(B, H * G, D, device="cuda", dtype=torch.bfloat16), mask=z(B, H),
                out=torch.zeros(B, H * G, D, device="cuda", dtype=torch.bfloat16),
                ws=torch.empty(cache.workspace_bytes(B, H * G), dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps_follow_requests_that_come_and_go(captured):
    """Prompts, single tokens, finished requests and their successors over one pool, eagerly or as one
    replayed graph; every step's attention against the oracle's cache of each request's own tokens."""
    B, H, G, P, max_pages, n_slots = 5, 2, 4, 64, 6, 420
    kb, vb = 4, 2
    cache = native.PagedKVQCache(16, H, kb, vb, page_tokens=P, keep_ch0=1)
    st = make_state(cache, B, H, G, max_pages, n_slots)
    plan_steps = [  # (new tokens, finished) of each request
        ([130, 0, 64, 1, 0], [0, 0, 0, 0, 0]), ([1, 200, 1, 1, 0], [0] * 5), ([1, 1, 0, 62, 0], [0, 0, 1, 0, 0]),
        ([1, 1, 90, 1, 7], [0] * 5), ([0, 1, 1, 1, 1], [1, 0, 0, 0, 0]), ([70, 1, 1, 1, 1], [0] * 5), ([1, 0, 3, 1, 1], [0, 1, 1, 0, 0])]
    graph = None
    if captured:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            step(cache, st)  # nothing new yet: loads the kernels
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step(cache, st)
    held = [[] for _ in range(B)]
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for new, done in plan_steps:
        st["new"].copy_(i32(new))
        st["done"].copy_(i32(done))
        for name in ("k", "v", "q"):
            st[name].copy_(torch.randn(st[name].shape, device="cuda", generator=g))
        if captured:
            graph.replay()
        else:
            step(cache, st)
        torch.cuda.synchronize()
        at = 0
        for b in range(B):
            if done[b]:
                held[b] = []
            held[b] += [(st["k"][i].clone(), st["v"][i].clone()) for i in range(at, at + new[b])]
            at += new[b]
        assert st["lens"].tolist() == [len(x) for x in held]
        used = [p for b in range(B) for p in st["table"][b, :-(-len(held[b]) // P)].tolist()]
        assert len(set(used)) == len(used)
        assert sorted(used + st["free"][:int(st["count"])].tolist()) == list(range(16))
        for b in range(B):
            n = len(held[b])
            if n == 0:
                assert not st["out"][b].any()
                continue
            k, v = (torch.stack([x[i] for x in held[b]]) for i in (0, 1))
            oc = oracle_cache(k, v, kb, vb, 1, 1, 0, 1.0)
            q = st["q"][b:b + 1].float().cpu().numpy()
            mask, _ = orc.select(q, H, 1, 20)
            assert np.array_equal(mask[0], st["mask"][b].cpu().numpy().view(np.uint32))
            want = oc.attention(q, np.array([n]), mask, 1 / math.sqrt(D))
            for j in range(H * G):
                kh, vh = oc.dequantize(0, j // G, 0, n)
                bound = output_bound(want[j], hadamard() @ q[0, j].astype(float), kh, vh, 1 / math.sqrt(D), "bf16")
                assert (np.abs(st["out"][b, j].double().cpu().numpy() - want[j]) <= bound).all()
    del graph


def test_two_streams_and_a_repeated_call_give_the_same_bits():
    pool = Pool(13, 60, 2, 64, 4, 4, 0)
    B, Hq = 6, 8
    table = i32(np.random.RandomState(1).permutation(60).reshape(B, 10))
    lens = i32([640, 100, 7, 333, 64, 0])
    q = torch.randn(B, Hq, D, device="cuda", dtype=torch.bfloat16)
    ref = pool.cache.decode(q, table, lens, 640)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(pool.cache.workspace_bytes(B, Hq), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(ref) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, w, o in zip(streams, ws, outs):
            pool.cache.decode(q, table, lens, 640, workspace=w, out=o, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(ws, outs):
        assert torch.equal(o, ref)
        assert pool.cache.decode_status(B, Hq, w) == native.KVQ_OK


@pytest.mark.parametrize("captured", [False, True])
def test_work_joined_from_another_stream(captured):
    # the kernels may be placed early, but see what other streams' work before them left,
    # and leave what later work there must not touch
    H, G, T, P = 2, 4, 640, 64
    cache = native.PagedKVQCache(T // P, H, 4, 4)
    first, then = (rows(3 + i, T, H, "bf16") for i in range(2))
    slots, table = i32(np.arange(T)), i32([list(range(T // P))])
    q = torch.randn(1, H * G, D, device="cuda", dtype=torch.bfloat16)
    lens, ws = i32([T]), torch.empty(cache.workspace_bytes(1, H * G), dtype=torch.uint8, device="cuda")
    cache.append(*first, slots)
    want = cache.decode(q, table, lens, T, workspace=ws).clone()
    cache.append(*then, slots)
    other = cache.decode(q, table, lens, T, workspace=ws).clone()
    assert not torch.equal(want, other)
    out, out2, k, v = torch.empty_like(want), torch.empty_like(want), torch.empty(T, H, D, device="cuda"), torch.empty(T, H, D, device="cuda")
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        side.wait_stream(main)
        cache.gather(slots, torch.float32, k_out=k, v_out=v)  # a kernel that lets the next one start early
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.cuda._sleep(1000000)
            cache.append(*first, slots)
        out.zero_()
        main.wait_stream(side)
        cache.decode(q, table, lens, T, workspace=ws, out=out)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            cache.append(*then, slots)
            cache.gather(slots, torch.float32, k_out=k, v_out=v)
        main.wait_stream(side)
        cache.decode(q, table, lens, T, workspace=ws, out=out2)

    torch.cuda.synchronize()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=main):
            work()
    for _ in range(3):
        out.zero_()
        out2.zero_()
        torch.cuda.synchronize()
        if captured:
            g.replay()
        else:
            with torch.cuda.stream(main):
                work()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out2, other)


def test_tokens_that_are_no_numbers_stay_by_themselves():
    # infinities and not-a-numbers in some tokens of one head: no other token's bytes, no other
    # head's outputs change, and requests that do not hold them keep their outputs
    H, G, T, P = 2, 2, 256, 64
    k, v = rows(11, T, H, "bf16")
    bad = [(5, float("inf")), (6, float("nan")), (70, float("-inf"))]
    clean = native.PagedKVQCache(4, H, 4, 2, keep_ch0=1)
    dirty = native.PagedKVQCache(4, H, 4, 2, keep_ch0=1)
    slots = i32(np.arange(T))
    clean.append(k, v, slots)
    k2, v2 = k.clone(), v.clone()
    for t, x in bad:
        k2[t, 0, 9] = x
        v2[t, 0, 77] = x
    dirty.append(k2, v2, slots)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[t for t, _ in bad]] = False
    for a, b in zip(clean.gather(slots, torch.float32), dirty.gather(slots, torch.float32)):
        assert torch.equal(a[keep], b[keep]) and torch.equal(a[:, 1], b[:, 1])
    q = torch.randn(4, H * G, D, device="cuda", dtype=torch.bfloat16)
    table, lens = i32([[0, 1], [2, 3], [1, -1], [0, -1]]), i32([128, 100, 6, 5])
    a, b = clean.decode(q, table, lens, 128), dirty.decode(q, table, lens, 128)
    assert torch.equal(a[:, G:], b[:, G:])   # the other head
    assert torch.equal(a[1:], b[1:])         # requests that hold no such token, or end before it


def test_wrapper_refusals_on_the_device():
    pool = Pool(13, 6, 2, 64, 4, 4, 0)
    c = pool.cache
    q = torch.randn(2, 4, D, device="cuda", dtype=torch.bfloat16)
    table, lens = i32([[0, 1], [2, 3]]), i32([100, 20])
    with pytest.raises(native.KvqError) as e:
        c.decode(q, table, lens, 129)
    assert e.value.status == native.KVQ_ERR_CAPACITY
    with pytest.raises(native.KvqError) as e:
        c.decode(q, table, lens, 128, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert e.value.status == native.KVQ_ERR_WORKSPACE
    with pytest.raises(ValueError):
        c.decode(q, table.long(), lens, 128)
    with pytest.raises(ValueError):
        c.decode(q, table, lens.cpu(), 128)
    with pytest.raises(ValueError):
        c.decode(q, table, lens, 128, mask=i32([[1, 2, 3]]))
    with pytest.raises(ValueError):
        c.decode(q, table, lens, 128, out=torch.empty(2, 4, D, device="cuda"))
    with pytest.raises(ValueError):
        c.append(q[:, :2], q[:, :2].float(), i32([0, 1]))
    with pytest.raises(ValueError):
        c.append(q[:, :2], q[:, 2:], i32([0, 1, 2]))
    with pytest.raises(ValueError):
        c.append(q[:, :2, :64], q[:, :2, :64], i32([0, 1]))
    with pytest.raises(ValueError):
        c.append(q[:, :2].transpose(0, 1), q[:, :2].transpose(0, 1), i32([0, 1]))
    with pytest.raises(ValueError):
        c.append(q[:, :2].double(), q[:, :2].double(), i32([0, 1]))
    with pytest.raises(ValueError):
        c.gather(i32([0, 1]), torch.float16, k_out=q[:, :2].contiguous())
    with pytest.raises(ValueError):
        c.gather(i32([0, 1]).long())
    with pytest.raises(ValueError):
        c.decode(q, table, lens, 1 << 40)
    with pytest.raises(TypeError):
        c.decode(q, table, lens, 1.5)
    with pytest.raises(TypeError):
        c.decode(q, table, lens, 128, softmax_scale="x")
    before = c.pages.clone()
    c.append(q[:, :2], q[:, 2:], i32([0, 1]))  # heads out of a wider row: fine
    assert not torch.equal(before, c.pages)
