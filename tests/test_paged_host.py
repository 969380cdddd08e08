"""Host side of the paged cache (no GPU): pool sizes and the block layout follow
include/kvq.h, and bad arguments are refused with the documented status before
anything is enqueued (every call here is refused, so the placeholder pointers
are never used)."""
import ctypes

import numpy as np
import pytest

from paged_testlib import BT, D, Layout, plan
from quantized_attention_kvq_b200 import native

FAKE = 0x100000
INVALID, UNSUPPORTED, CAPACITY, WORKSPACE = (native.KVQ_ERR_INVALID_ARG, native.KVQ_ERR_UNSUPPORTED,
                                             native.KVQ_ERR_CAPACITY, native.KVQ_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def L():
    from quantized_attention_kvq_b200 import build
    build.build_kvq()
    build.build_binding()
    return native.lib()


def desc(**kw):
    d = native.KvqPagedStruct(8, 128, 2, 128, 4, 2, 32, 4, 1, 1, 0, 1.0, FAKE)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kb,vb,ch0", [(kb, vb, c) for kb in (2, 4) for vb in (2, 4) for c in (0, 1)])
def test_layout_gives_every_bit_one_owner(L, kb, vb, ch0):
    lay = Layout(kb, vb, ch0)
    used = np.zeros(lay.bytes * 8, np.int32)
    owner = np.full(lay.bytes, -1)
    tb = lay.tables()

    def claim(t, byte, bit, n):
        used[byte * 8 + bit: byte * 8 + bit + n] += 1
        for b in range(byte, byte + (bit + n + 7) // 8):
            assert owner[b] in (-1, t)  # a byte belongs to one token
            owner[b] = t

    for t in range(BT):
        for ch in range(D):
            claim(t, *tb["k"][t, ch], kb)
            claim(t, *tb["v"][t, ch], vb)
        for g in range(4):
            for base, at in ((lay.ks, "s"), (lay.kz, "kz"), (lay.vs, "s"), (lay.vz, "s")):
                claim(t, base + tb[at][t, g], 0, 16)
        if ch0:
            claim(t, lay.k0 + 2 * t, 0, 16)
    assert (used == 1).all()
    assert L.kvq_paged_bytes(ctypes.byref(desc(k_bits=kb, v_bits=vb, keep_ch0=ch0))) == 8 * 2 * 2 * lay.bytes


BAD = [("num_pages", 0, INVALID), ("kv_heads", 0, INVALID), ("page_tokens", 0, INVALID), ("page_tokens", 96, UNSUPPORTED),
       ("page_tokens", 8192, UNSUPPORTED), ("head_dim", 64, UNSUPPORTED), ("k_bits", 3, UNSUPPORTED),
       ("v_bits", 8, UNSUPPORTED), ("group_size", 64, UNSUPPORTED), ("prune_granule", 8, UNSUPPORTED),
       ("rotate_k", 2, UNSUPPORTED), ("rotate_k", 3, INVALID), ("rotate_k", -1, INVALID), ("keep_ch0", 2, INVALID),
       ("rotate_v", 2, INVALID), ("v_clip", 0.0, INVALID), ("v_clip", 1.5, INVALID), ("v_clip", float("nan"), INVALID),
       ("num_pages", 1 << 25, UNSUPPORTED), ("kv_heads", 65536, UNSUPPORTED)]


@pytest.mark.parametrize("field,value,status", BAD + [("pages", 0, INVALID), ("pages", FAKE + 64, INVALID)])
def test_bad_pool_refused_everywhere(L, field, value, status):
    d = ctypes.byref(desc(**{field: value}))
    assert L.kvq_paged_append(d, FAKE, 256, FAKE, 256, native.KVQ_BF16, 4, FAKE, None) == status
    assert L.kvq_paged_gather(d, FAKE, 4, native.KVQ_BF16, 0, FAKE, FAKE, None) == status
    assert L.kvq_paged_decode(d, FAKE, 1 << 20, native.KVQ_BF16, 1 << 10, 2, FAKE, 4, FAKE, 100, None, 0.1, FAKE, FAKE,
                              1 << 40, None) == status
    if field != "pages":
        assert L.kvq_paged_bytes(d) == 0
        assert L.kvq_paged_decode_workspace_bytes(d, 2, 8) == 0
        assert L.kvq_paged_decode_status(d, 2, 8, FAKE, 1 << 40, None) == status


def test_append_refusals(L):
    d = ctypes.byref(desc())

    def call(k=FAKE, ks=256, v=FAKE, vs=256, dt=native.KVQ_BF16, n=4, slots=FAKE):
        return L.kvq_paged_append(d, k, ks, v, vs, dt, n, slots, None)
    assert call(n=-1) == INVALID
    assert call(dt=9) == INVALID
    assert call(k=None) == INVALID and call(v=None) == INVALID and call(slots=None) == INVALID
    assert call(k=FAKE + 2) == INVALID and call(v=FAKE + 8) == INVALID and call(slots=FAKE + 2) == INVALID
    assert call(ks=255) == INVALID and call(vs=-256) == INVALID  # less than a row
    assert call(ks=260) == INVALID                               # rows off 16-byte boundaries
    assert call(n=0, k=None, v=None, slots=None) == native.KVQ_OK
    assert call(n=(1 << 30) + 1) == UNSUPPORTED


def test_gather_refusals(L):
    d = ctypes.byref(desc())

    def call(slots=FAKE, n=4, dt=native.KVQ_F16, back=0, k=FAKE, v=FAKE):
        return L.kvq_paged_gather(d, slots, n, dt, back, k, v, None)
    assert call(n=-1) == INVALID and call(dt=3) == INVALID and call(back=2) == INVALID
    assert call(slots=None) == INVALID and call(k=None, v=None) == INVALID
    assert call(k=FAKE + 4) == INVALID and call(v=FAKE + 8) == INVALID
    assert call(n=0, k=None, v=None, slots=None) == native.KVQ_OK
    assert call(n=(1 << 30) + 1) == UNSUPPORTED


def test_decode_refusals(L):
    dd = desc()
    d = ctypes.byref(dd)
    ws = L.kvq_paged_decode_workspace_bytes(d, 3, 8)
    assert ws >= (3 * 2 + 1) * 4 * (512 + 8)

    def call(q=FAKE, qs=1024, dt=native.KVQ_BF16, hq=8, B=3, table=FAKE, mp=4, lens=FAKE, ml=512, mask=None, scale=0.1,
             out=FAKE, w=FAKE, wb=ws):
        return L.kvq_paged_decode(d, q, qs, dt, hq, B, table, mp, lens, ml, mask, scale, out, w, wb, None)
    assert call(wb=ws - 1) == WORKSPACE
    assert call(ml=513) == CAPACITY and call(ml=-1) == INVALID
    assert call(hq=7) == INVALID and call(hq=0) == INVALID and call(hq=34, qs=34 * 128) == UNSUPPORTED
    assert call(B=0) == INVALID and call(mp=0) == INVALID
    assert call(scale=float("inf")) == INVALID and call(dt=5) == INVALID
    for name in ("q", "table", "lens", "out", "w"):
        assert call(**{name: None}) == INVALID, name
    assert call(q=FAKE + 8) == INVALID and call(out=FAKE + 8) == INVALID and call(w=FAKE + 128) == INVALID
    assert call(mask=FAKE + 2) == INVALID and call(lens=FAKE + 1) == INVALID
    assert call(qs=1023) == INVALID and call(qs=1028) == INVALID
    assert L.kvq_paged_decode(ctypes.byref(desc(num_pages=1, page_tokens=4096)), FAKE, 1024, native.KVQ_BF16, 8, 1 << 20,
                              FAKE, 1 << 19, FAKE, (1 << 31) - 1, None, 0.1, FAKE, FAKE, 1 << 60, None) == UNSUPPORTED
    assert L.kvq_paged_decode_status(d, 3, 8, None, ws, None) == INVALID
    assert L.kvq_paged_decode_status(d, 3, 8, FAKE, ws - 1, None) == WORKSPACE
    assert L.kvq_paged_decode_workspace_bytes(d, 0, 8) == 0 and L.kvq_paged_decode_workspace_bytes(d, 3, 7) == 0


def test_plan_refusals(L):
    def call(num=64, P=64, B=4, ctx=FAKE, new=FAKE, done=None, table=FAKE, mp=8, free=FAKE, cnt=FAKE, out=FAKE, slots=FAKE,
             pos=FAKE, n=16, cu=FAKE, lens=FAKE):
        return L.kvq_page_plan(num, P, B, ctx, new, done, table, mp, free, cnt, out, slots, pos, n, cu, lens, None)
    assert call(num=0) == INVALID and call(P=0) == INVALID and call(B=0) == INVALID and call(mp=0) == INVALID
    assert call(n=-1) == INVALID
    for name in ("ctx", "new", "table", "free", "cnt", "out", "slots", "cu", "lens"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: FAKE + 2}) == INVALID, name
    assert call(done=FAKE + 1) == INVALID and call(pos=FAKE + 1) == INVALID
    assert call(P=80) == UNSUPPORTED and call(P=8192) == UNSUPPORTED and call(B=8193) == UNSUPPORTED
    assert call(num=1 << 26) == UNSUPPORTED and call(mp=1 << 26) == UNSUPPORTED


def test_wrapper_refuses_host_tensors_and_wrong_shapes(L):
    import torch
    with pytest.raises(native.KvqError):
        native.PagedKVQCache(4, 2, 3, 4)
    with pytest.raises(ValueError):
        native.PagedKVQCache(4, 2, 4, 4, pages=torch.zeros(16, dtype=torch.uint8))
    cache = native.PagedKVQCache.__new__(native.PagedKVQCache)  # no device memory is needed to refuse
    cache.desc, cache.H, cache.pages = desc(), 2, torch.zeros(8, dtype=torch.uint8)
    cache._at, cache._dev = ctypes.addressof(cache.desc), -1
    fast = native._binding()
    cache._append, cache._gather, cache._decode = fast.append, fast.gather, fast.decode
    k, i = torch.zeros(3, 2, 128), torch.zeros(3, dtype=torch.int32)
    for bad in (lambda: cache.append(k, k, i), lambda: cache.gather(i), lambda: cache.append(k, None, i),
                lambda: cache.append(k, k, [1, 2, 3]), lambda: cache.decode(k, i[None], i, 3),
                lambda: native.PagePlanner(4).plan(i, i, i[:, None], i, i[:1], 3),
                lambda: native.PagePlanner(4).plan(i, i, i, i, i[:1], 3)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fast.append(1, 2), lambda: cache.gather(i, rotate_back="x"), lambda: fast.bind("x", 1, 1, 1, 1, 1)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(ValueError):
        native._i32(torch.zeros(3), "slots", 3)
    with pytest.raises(ValueError):
        native._i32(torch.zeros(4, dtype=torch.int32), "slots", 3)


def test_plan_model_hands_pages_out_in_request_order():
    # the model the GPU tests compare with, on a step worked out by hand: pages
    # of 64, free stack [5, 9, 2] (top 2); request 1 is finished and gives 7
    table = np.array([[1, -1, -1], [7, -1, -1], [-1, -1, -1], [4, -1, -1]], np.int32)
    r = plan(10, 64, [64, 10, 0, 63], [1, 0, 130, 2], [0, 1, 0, 0], table, np.array([5, 9, 2, 0, 0, 0, 0, 0, 0, 0], np.int32), 3, 140)
    assert r["free"][3] == 7
    assert r["table"][0, 1] == 7 and list(r["table"][2]) == [2, 9, 5]
    assert list(r["seq_lens"]) == [65, 0, 130, 63]  # request 3 needs a fifth page: not served
    assert r["count"] == 0 and list(r["cu_new"]) == [0, 1, 1, 131, 133]
    assert r["slots"][0] == 7 * 64 and r["slots"][1] == 2 * 64 and r["slots"][130] == 5 * 64 + 1
    assert (r["slots"][131:] == -1).all()
