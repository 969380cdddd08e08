"""Plain implementations the paged-cache tests compare with: the pool layout as
include/kvq.h words it, the planning step request by request, attention in 64
bits, and the error bounds of the decode."""
from __future__ import annotations

import math

import numpy as np

BT, D = 64, 128


class Layout:
    """Byte places of a 64-token block."""

    def __init__(self, kb, vb, ch0):
        self.kb, self.vb, self.ch0 = kb, vb, ch0
        self.ks = BT * D * kb // 8
        self.kz = self.ks + 512
        self.k0 = self.kz + 512
        self.vc = self.k0 + (128 if ch0 else 0)
        self.vs = self.vc + BT * D * vb // 8
        self.vz = self.vs + 512
        self.bytes = self.vz + 512

    def k_code(self, t, ch):
        """(byte, bit) of channel ch of token t."""
        p, u = ch // 4, t // 8
        if self.kb == 4:
            i, e = (t % 8) // 2, t % 2
            return p * 128 + 16 * (u ^ (2 * (p & 3))) + 4 * i + e + (2 if ch % 4 >= 2 else 0), 4 * (ch % 2)
        return p * 64 + 8 * (u ^ (4 * ((p >> 1) & 1))) + t % 8, 2 * (ch % 4)

    def v_code(self, t, ch):
        per = 8 // self.vb
        byte = 16 * (t // 16) + 4 * ((t % 8) // 2) + 2 * ((t % 16) // 8) + t % 2
        return self.vc + (ch // per) * 64 + byte, self.vb * (ch % per)

    def scale(self, t, grp):
        """byte of an fp16 inside a scales part (also the value zeros)"""
        u, i, e = t // 8, (t % 8) // 2, t % 2
        return 2 * (((i * 8 + u) * 2 + e) * 4 + grp)

    def k_zero(self, t, grp):
        u, i, e = t // 8, (t % 8) // 2, t % 2
        return 2 * ((((((i // 2) * 8 + u) * 2 + grp // 2) * 2 + i % 2) * 2 + e) * 2 + grp % 2)

    def tables(self):
        """index arrays of all tokens: code bytes and bits [64][128], scale and zero bytes [64][4]"""
        if not hasattr(self, "_tab"):
            f = lambda fn, n: np.array([[fn(t, c) for c in range(n)] for t in range(BT)])  # noqa: E731
            self._tab = dict(k=f(self.k_code, D), v=f(self.v_code, D), s=f(self.scale, 4), kz=f(self.k_zero, 4))
        return self._tab

    def unpack(self, block):
        """One block (uint8 [bytes]) -> codes, scales, zeros of keys and values, channel-0 bits."""
        tb = self.tables()
        half = lambda base, at: (block[base + at].astype(np.uint16) | (block[base + at + 1].astype(np.uint16) << 8))  # noqa: E731
        out = {}
        for n, bits in (("k", self.kb), ("v", self.vb)):
            at = tb[n]
            out[n + "c"] = (block[at[..., 0]] >> at[..., 1].astype(np.uint8)) & ((1 << bits) - 1)
        out["ks"], out["kz"] = half(self.ks, tb["s"]), half(self.kz, tb["kz"])
        out["vs"], out["vz"] = half(self.vs, tb["s"]), half(self.vz, tb["s"])
        if self.ch0:
            out["k0"] = half(self.k0, 2 * np.arange(BT))
        return out

    def values(self, block):
        """Keys and values [64][128] in 64 bits, as the block holds them."""
        u = self.unpack(block)
        f = lambda x: x.astype(np.uint16).view(np.float16).astype(np.float64).repeat(32, 1)  # noqa: E731
        with np.errstate(invalid="ignore", over="ignore"):
            k = u["kc"] * f(u["ks"]) + f(u["kz"])
            v = u["vc"] * f(u["vs"]) + f(u["vz"])
        if self.ch0:
            k[:, 0] = (u["k0"].astype(np.uint32) << 16).view(np.float32)
        return k, v


def hadamard():
    h = np.ones((1, 1))
    for _ in range(7):
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(D)


def plan(num_pages, P, ctx, new, done, table, free, count, n_slots):
    """kvq_page_plan, one request after another.  Returns everything it writes."""
    B, max_pages = table.shape
    table, free = table.copy(), free.copy()
    ctx = [max(int(x), 0) for x in ctx]
    new = [max(int(x), 0) for x in new]
    pages = lambda n: -(-n // P)  # noqa: E731
    for b in range(B):
        if done is not None and done[b]:
            for i in range(min(pages(ctx[b]), max_pages)):
                free[count] = table[b, i]
                count += 1
            ctx[b] = 0
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    slots = np.full(n_slots, -1, np.int32)
    pos = np.full(n_slots, -1, np.int32)
    lens = np.array(ctx, np.int32)
    asked, top = 0, count
    for b in range(B):
        end = ctx[b] + new[b]
        if end > max_pages * P or cu[b + 1] > n_slots:
            continue
        need = pages(end) - pages(ctx[b])
        asked += need
        if need and asked > top:
            continue
        for i in range(need):
            count -= 1
            table[b, pages(ctx[b]) + i] = free[count]
        for i in range(new[b]):
            p = ctx[b] + i
            slots[cu[b] + i] = table[b, p // P] * P + p % P
            pos[cu[b] + i] = p
        lens[b] = end
    return dict(slots=slots, positions=pos, cu_new=cu.astype(np.int32), seq_lens=lens, table=table, free=free, count=count)


def attention(q, k, v, scale, keep_ch=None):
    """One query row over [n][128] keys and values, in 64 bits."""
    if k.shape[0] == 0:
        return np.zeros(D)
    q = q if keep_ch is None else q * keep_ch
    s = k @ q * scale
    w = np.exp(s - s.max())
    return (w / w.sum()) @ v


def output_bound(o, q, k, v, scale, dtype):
    """How far a decode output row may be from its 64-bit value, element by element.

    Type: the final rounding, |o| eps/2.  Score: q is fp32 butterflies (7 sums
    of relative error 2^-24 each, bounded by 2^-21 |q|_2) and two fp16 pieces
    (2^-22 of an element), the products are summed in fp32 over 128 channels:
    together below 2^-20 |q|_2 |k|_2 scale per score, taken twice (the softmax's
    numerator and denominator), times the values' spread.  P': one fp16 rounding
    2^-11 (16-bit types; 2^-22 for fp32) of p * scale * code, i.e. of at most the
    spread of the values.  Exponential and sums in fp32: 2^-20 of the spread."""
    import torch
    t = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dtype]
    half = torch.finfo(t).eps / 2
    if k.shape[0] == 0:
        return np.zeros(D)
    spread = np.abs(v).max() * 2
    eps_s = 2.0 ** -20 * np.linalg.norm(q) * np.linalg.norm(k, axis=1).max() * scale
    p = 2.0 ** -11 if dtype != "f32" else 2.0 ** -22
    return np.abs(o) * half + spread * (2 * eps_s + p + 2.0 ** -20) + torch.finfo(t).tiny
