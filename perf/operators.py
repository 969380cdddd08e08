"""The paged low-bit KV cache's operators: plan, append, gather, decode.

Each case is one call a serving step makes of the cache: building the step's
block tables and slot map, quantizing new tokens into pages, reading cached
tokens back as dense rows, and one decode step.  ``run`` computes the plain
form (elementary torch operations) or, with ``own`` set, the library's calls.

The cache format the cases share (also in ``include/kvq.h``): pages are
[page][kv head][64-token block][block bytes]; a block holds the key codes, the
key scales, the key zeros, channel 0 in bf16 (optional), the value codes, the
value scales and the value zeros of its 64 tokens.
"""
import math
import random

import torch

own = False

D = 128           # head dim
BT = 64           # tokens per block
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step's bookkeeping for a handful of requests: latency
        dict(name="plan_step_b8", op="plan", B=8, P=64, max_pages=256, finished=1, admitted=0, prompt=0, seed_len=3),
        # a step that admits long prompts into a large batch
        dict(name="plan_prompts_b512", op="plan", B=512, P=128, max_pages=512, finished=40, admitted=48, prompt=2500,
             seed_len=4),
        # a decode step's append: one new token per request
        dict(name="append_step_b64_int4", op="append", n=64, H=8, G=4, P=64, kb=4, vb=4, rot=1, ch0=0, rotv=0,
             clip=1.0, dtype="bf16", pad=3, back=0),
        # a batch of prompts (ragged, arbitrary offsets in their pages), INT4 keys and INT2 values
        dict(name="append_prompts_32k_k4v2", op="append", n=32768, H=8, G=4, P=128, kb=4, vb=2, rot=1, ch0=0, rotv=0,
             clip=1.0, dtype="bf16", pad=0, back=0),
        # the Dual-QK recipe's INT2 cache (channel 0 kept, values rotated and clipped), odd token count, fp16
        dict(name="append_odd_int2_f16", op="append", n=5003, H=5, G=1, P=64, kb=2, vb=2, rot=1, ch0=1, rotv=1,
             clip=0.92, dtype="f16", pad=5, back=0),
        # dense rows of cached prefixes for prompt attention, in the model's basis
        dict(name="gather_prefix_24k_int4", op="gather", n=24576, H=8, P=64, kb=4, vb=4, rot=1, ch0=0, rotv=0,
             dtype="bf16", pad=0, back=1),
        # a short odd prefix in fp32, INT2 with channel 0
        dict(name="gather_odd_int2_f32", op="gather", n=777, H=3, P=128, kb=2, vb=2, rot=1, ch0=1, rotv=1,
             dtype="f32", pad=7, back=1),
        # one sequence of 1024 tokens, one head, fp32: the smallest decode
        dict(name="decode_tiny_f32", op="decode", B=1, H=1, G=1, P=64, lo=1024, hi=1024, kb=4, vb=4, rot=1, ch0=0,
             rotv=0, keep=32, dtype="f32", seed_len=1),
        # grouped-query decode at 32K tokens, INT4
        dict(name="decode_gqa_int4_b8_32k", op="decode", B=8, H=8, G=4, P=64, lo=32768, hi=32768, kb=4, vb=4, rot=1,
             ch0=0, rotv=0, keep=32, dtype="bf16", seed_len=1),
        # Dual-QK INT2 at 128K tokens: channel 0 in bf16, 19 of 32 channel groups kept
        dict(name="decode_int2_b4_128k_keep19", op="decode", B=4, H=8, G=4, P=128, lo=131072, hi=131072, kb=2, vb=2,
             rot=1, ch0=1, rotv=0, keep=19, dtype="bf16", seed_len=1),
        # a ragged batch of 64 requests, eight query heads per kv head
        dict(name="decode_ragged_b64_keep24", op="decode", B=64, H=8, G=8, P=64, lo=1024, hi=16384, kb=4, vb=2, rot=1,
             ch0=1, rotv=0, keep=24, dtype="bf16", seed_len=4),
        # many short requests (some empty), five query heads per kv head, values rotated
        dict(name="decode_short_b200_g5_f16", op="decode", B=200, H=4, G=5, P=128, lo=0, hi=700, kb=4, vb=4, rot=1,
             ch0=0, rotv=1, keep=32, dtype="f16", seed_len=9),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "gather", "decode", "decode"])
    P = rng.choice([64, 64, 128, 256])
    kb, vb = rng.choice([2, 4]), rng.choice([2, 4])
    base = dict(op=op, P=P)
    if op == "plan":
        B = log_int(rng, 1, 1000)
        fin = rng.randint(0, B // 4)
        return dict(base, B=B, max_pages=log_int(rng, 16, 700), finished=fin, admitted=rng.randint(0, (B - fin) // 3),
                    prompt=log_int(rng, 1, 4000), seed_len=rng.randint(0, 1 << 20))
    flags = dict(kb=kb, vb=vb, rot=rng.choice([0, 1, 1]), ch0=rng.randint(0, 1), rotv=rng.randint(0, 1))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("append", "gather"):
        H = rng.choice([1, 2, 3, 5, 8])
        n = log_int(rng, 1, 32768 * 8 // (H * (2 if dtype == "f32" else 1)) // 2)
        case = dict(base, n=n, H=H, dtype=dtype, pad=rng.randint(0, 9), back=rng.randint(0, 1), **flags)
        return dict(case, G=rng.choice([1, 2, 4, 8]), clip=rng.choice([1.0, 0.92])) if op == "append" else case
    B, H, G = log_int(rng, 1, 256), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    hi = log_int(rng, 1, max(1, min(65536, 4000000 // (B * H))))
    return dict(base, B=B, H=H, G=G, lo=rng.choice([0, hi // 3, hi]), hi=hi, keep=rng.choice([32, rng.randint(6, 32)]),
                dtype=dtype, seed_len=rng.randint(0, 1 << 20), **flags)


def seq_lens(c):
    """The requests' cached lengths: part of the case, not of the seed."""
    r = random.Random("lens %d %d %d %d" % (c["B"], c["lo"], c["hi"], c["seed_len"]))
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]


def plan_lens(c):
    """ctx, new and done of each request of a planning step."""
    r = random.Random("plan %d %d %d" % (c["B"], c["max_pages"], c["seed_len"]))
    most = c["max_pages"] * c["P"]
    role = ["done"] * c["finished"] + ["admit"] * c["admitted"]
    role += ["step"] * (c["B"] - len(role))
    r.shuffle(role)
    ctx, new, done = [], [], []
    for x in role:
        done.append(int(x == "done"))
        ctx.append(0 if x == "admit" else r.randint(1, most - 1))
        new.append(0 if x == "done" else min(most, r.randint(max(1, c["prompt"] // 2), c["prompt"])) if x == "admit" else 1)
    return ctx, new, done


# --------------------------------------------------------------------- the format
def code_bytes(c):
    kc, vc = BT * D * c["kb"] // 8, BT * D * c["vb"] // 8
    ch0 = BT * 2 if c["ch0"] else 0
    at = {}
    off = 0
    for name, size in (("kc", kc), ("ks", BT * 8), ("kz", BT * 8), ("k0", ch0), ("vc", vc), ("vs", BT * 8), ("vz", BT * 8)):
        at[name] = (off, off + size)
        off += size
    return at, off


def k_swizzle(kb, device):
    """chunk position of token group g (8 tokens) in key row p: g xor this."""
    p = torch.arange(32, device=device)[:, None]
    g = torch.arange(8, device=device)[None, :]
    return p, g ^ (2 * (p & 3) if kb == 4 else 4 * ((p >> 1) & 1))


def pack_blocks(c, kcode, ks, kz, k0, vcode, vs, vz):
    """codes [N, 64, 128] uint8, scales and zeros [N, 64, 4] fp16, k0 [N, 64] bf16 -> [N, block bytes] uint8."""
    N = kcode.shape[0]
    p, pos = k_swizzle(c["kb"], kcode.device)
    if c["kb"] == 4:
        b = kcode.view(N, 8, 4, 2, 32, 2, 2)  # g, i, e, p, half, channel
        b = b[..., 0] | (b[..., 1] << 4)
        b = b.permute(0, 4, 1, 2, 5, 3).reshape(N, 32, 8, 16)
    else:
        b = kcode.view(N, 64, 32, 4)
        b = b[..., 0] | (b[..., 1] << 2) | (b[..., 2] << 4) | (b[..., 3] << 6)
        b = b.view(N, 8, 8, 32).permute(0, 3, 1, 2)
    parts = [b[:, p, pos].reshape(N, -1)]
    by_pair = lambda x: x.view(N, 8, 4, 8).permute(0, 2, 1, 3).reshape(N, -1).view(torch.uint8)  # noqa: E731
    parts.append(by_pair(ks))
    z = kz.view(N, 8, 2, 2, 2, 2, 2)  # g, j, i & 1, e, c', group & 1
    parts.append(z.permute(0, 2, 1, 5, 3, 4, 6).reshape(N, -1).view(torch.uint8))
    if c["ch0"]:
        parts.append(k0.contiguous().view(torch.uint8))
    if c["vb"] == 4:
        v = vcode.view(N, 64, 64, 2)
        v = v[..., 0] | (v[..., 1] << 4)
    else:
        v = vcode.view(N, 64, 32, 4)
        v = v[..., 0] | (v[..., 1] << 2) | (v[..., 2] << 4) | (v[..., 3] << 6)
    v = v.view(N, 4, 2, 4, 2, v.shape[-1])  # 16-token chunk, half, i, e, row
    parts.append(v.permute(0, 5, 1, 3, 2, 4).reshape(N, -1))
    parts += [by_pair(vs), by_pair(vz)]
    return torch.cat(parts, 1)


def unpack_blocks(c, blocks):
    """[N, block bytes] -> dequantized keys and values [N, 64, 128] fp32, as the blocks hold them."""
    N = blocks.shape[0]
    at, _ = code_bytes(c)
    part = lambda name: blocks[:, at[name][0]:at[name][1]]  # noqa: E731
    half = lambda name: part(name).contiguous().view(torch.float16)  # noqa: E731
    p, pos = k_swizzle(c["kb"], blocks.device)
    if c["kb"] == 4:
        b = part("kc").reshape(N, 32, 8, 16)[:, p, pos].view(N, 32, 8, 4, 2, 2)  # p, g, i, half, e
        b = torch.stack((b & 15, b >> 4), -1).permute(0, 2, 3, 5, 1, 4, 6)
    else:
        b = part("kc").reshape(N, 32, 8, 8)[:, p, pos].view(N, 32, 64)
        b = torch.stack((b & 3, (b >> 2) & 3, (b >> 4) & 3, b >> 6), -1).permute(0, 2, 1, 3)
    kcode = b.reshape(N, 64, 4, 32)
    by_pair = lambda name: half(name).view(N, 4, 8, 2, 4).permute(0, 2, 1, 3, 4).reshape(N, 64, 4, 1).float()  # noqa: E731
    kz = half("kz").view(N, 2, 8, 2, 2, 2, 2).permute(0, 2, 1, 4, 5, 3, 6).reshape(N, 64, 4, 1).float()
    k = (kcode.float() * by_pair("ks") + kz).view(N, 64, D)
    if c["ch0"]:
        k[..., 0] = part("k0").contiguous().view(torch.bfloat16).float()
    v = part("vc").reshape(N, -1, 4, 4, 2, 2)  # row, chunk, i, half, e
    v = v.permute(0, 2, 4, 3, 5, 1).reshape(N, 64, -1)
    v = torch.stack((v & 15, v >> 4) if c["vb"] == 4 else (v & 3, (v >> 2) & 3, (v >> 4) & 3, v >> 6), -1)
    return k, (v.reshape(N, 64, 4, 32).float() * by_pair("vs") + by_pair("vz")).view(N, 64, D)


def hadamard(device):
    h = torch.ones(1, 1, dtype=torch.float64, device=device)
    two = torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64, device=device)
    return torch.kron(torch.kron(torch.kron(torch.kron(torch.kron(torch.kron(torch.kron(h, two), two), two), two), two), two), two)


def rotated(x):
    """The orthonormal Walsh-Hadamard transform of rows, products in 64 bits, rounded to 32."""
    return (x.double() @ hadamard(x.device) * (1.0 / math.sqrt(D))).float()


def quantized(x, bits, skip0, clip):
    """x [.., 128] fp32 -> codes uint8 [.., 128], scale and zero fp16 [.., 4]."""
    L = (1 << bits) - 1
    g = x.reshape(*x.shape[:-1], 4, 32)
    r = g
    if skip0:  # channel 0 is kept apart: outside its group's range
        r = g.clone()
        r[..., 0, 0] = g[..., 0, 1]
    mn, mx = (r.amin(-1) + 0.0) * clip, (r.amax(-1) + 0.0) * clip
    s = ((mx - mn) / L).clamp(max=65504.0).half()
    z = mn.clamp(-65504.0, 65504.0).half()
    sf = s.float()[..., None]
    q = torch.where(sf > 0, (g - z.float()[..., None]) / sf, torch.zeros_like(g))
    code = q.round().clamp(0, L).to(torch.uint8).reshape(x.shape)
    if skip0:
        code[..., 0] = 0
    return code, s, z


# --------------------------------------------------------------------- inputs
def token_rows(gen, n, H, dtype):
    """Keys with a few strong channels per head, as models have them, and values, [n, H, 128]."""
    dev = gen.device
    scale = torch.exp(0.5 * torch.randn(H, D, device=dev, generator=gen))
    strong = torch.rand(H, D, device=dev, generator=gen).argsort(1)[:, :4]
    scale.scatter_(1, strong, scale.gather(1, strong) * 10)
    k = torch.randn(n, H, D, device=dev, generator=gen) * scale
    return k.to(dtype), torch.randn(n, H, D, device=dev, generator=gen).to(dtype)


def fill_pages(c, gen, pages):
    """Every block of the pool, made and quantized a slice of pages at a time."""
    n_pages, H, nb, size = pages.shape
    step = max(1, (1 << 19) // (H * nb * BT))
    for a in range(0, n_pages, step):
        part = pages[a:a + step]
        n = part.shape[0] * nb * BT
        k, v = token_rows(gen, n, H, torch.bfloat16)
        k, v = (x.float().view(part.shape[0], nb * BT, H, D).transpose(1, 2).reshape(-1, BT, D) for x in (k, v))
        h = (hadamard(k.device) / math.sqrt(D)).float()
        k = k @ h if c["rot"] else k
        v = v @ h if c["rotv"] else v
        kc, ks, kz = quantized(k, c["kb"], c["ch0"], 1.0)
        vc, vs, vz = quantized(v, c["vb"], 0, 1.0)
        part.copy_(pack_blocks(c, kc, ks, kz, k[..., 0].bfloat16(), vc, vs, vz).view(part.shape))


def handle(c, pages):
    """The program's handle on its pool (the page memory is the program's own)."""
    from quantized_attention_kvq_b200 import native
    return native.PagedKVQCache(pages.shape[0], c["H"], c["kb"], c["vb"], page_tokens=c["P"], rotate_k=c["rot"],
                                keep_ch0=c["ch0"], rotate_v=c["rotv"], v_clip=c.get("clip", 1.0), pages=pages)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 1)
    st = {"c": c}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    P = c["P"]
    if c["op"] == "plan":
        ctx, new, done = plan_lens(c)
        held = sum(-(-x // P) for x in ctx)
        need = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(ctx, new))
        released = sum(-(-x // P) for x, d in zip(ctx, done) if d)
        # a pool that serves the step with little to spare, its free list in the order requests left it
        num = held + max(need - released, 0) + c["B"] // 2 + 1
        perm = torch.randperm(num, device="cuda", generator=gen).to(torch.int32)
        table = torch.full((c["B"], c["max_pages"]), -1, dtype=torch.int32, device="cuda")
        n_pages = i32([-(-x // P) for x in ctx])
        col = torch.arange(c["max_pages"], device="cuda", dtype=torch.int32)
        has = col[None, :] < n_pages[:, None]
        table[has] = perm[:held]
        free = torch.full((num,), -1, dtype=torch.int32, device="cuda")
        free[:num - held] = perm[held:]
        st.update(ctx=i32(ctx), new=i32(new), done=i32(done), table=table, free=free, count=i32([num - held]),
                  num_pages=num, n_slots=sum(new) + 5)
        if own:
            from quantized_attention_kvq_b200 import native
            st["plan"] = native.PagePlanner(num, P)
        return st
    _, size = code_bytes(c)
    nb = P // BT
    dtype = DTYPES[c["dtype"]]
    if c["op"] == "decode":
        lens = seq_lens(c)
        n_pg = [-(-x // P) for x in lens]
        num = max(1, sum(n_pg)) + 3
        pages = torch.empty((num, c["H"], nb, size), dtype=torch.uint8, device="cuda")
        fill_pages(c, gen, pages)
        table = torch.full((c["B"], max(1, max(n_pg))), -1, dtype=torch.int32, device="cuda")
        perm = torch.randperm(num, device="cuda", generator=gen).to(torch.int32)
        has = torch.arange(table.shape[1], device="cuda")[None, :] < i32(n_pg)[:, None]
        table[has] = perm[:sum(n_pg)]
        q = torch.randn(c["B"], c["H"] * c["G"], D, device="cuda", generator=gen).to(dtype)
        st.update(pages=pages, table=table, lens=i32(lens), max_len=max(lens), q=q, mask=None)
        if c["keep"] < 32:  # the step's channel selection: the groups with the largest query energy
            qr = rotated(q.float()) if c["rot"] else q.float()
            e = qr.double().view(c["B"], c["H"], c["G"], 32, 4).square().sum((2, 4))
            bits = torch.zeros_like(e, dtype=torch.int64).scatter_(2, e.topk(c["keep"], 2).indices, 1)
            word = (bits << torch.arange(32, device="cuda")).sum(2)
            st["mask"] = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
        if own:
            st["cache"] = handle(c, pages)
            st["ws"] = torch.empty(st["cache"].workspace_bytes(c["B"], c["H"] * c["G"]), dtype=torch.uint8, device="cuda")
        return st
    # token slots: runs of consecutive positions of several requests, each run starting anywhere in a page
    n, pad = c["n"], c["pad"]
    r = random.Random(seed)
    runs, left = [], n
    while left > 0:
        take = min(left, 1 if n <= 256 else r.randint(1, max(1, n // 8)))
        runs.append((r.randrange(P), take))
        left -= take
    pages_of = [-(-(o + t) // P) for o, t in runs]
    num = sum(pages_of) + 2
    perm = torch.randperm(num, device="cuda", generator=gen)
    slots, base = [], 0
    for (o, t), m in zip(runs, pages_of):
        pos = o + torch.arange(t, device="cuda")
        slots.append(perm[base + pos // P] * P + pos % P)
        base += m
    slots = torch.cat(slots + [torch.full((pad,), -1, device="cuda")]).to(torch.int32)  # padding of a captured step
    st["slots"] = slots
    if c["op"] == "gather":
        pages = torch.empty((num, c["H"], nb, size), dtype=torch.uint8, device="cuda")
        fill_pages(c, gen, pages)
    else:
        # keys and values are slices of the step's fused projection
        H, Hq = c["H"], c["H"] * c["G"]
        pages = torch.zeros((num, H, nb, size), dtype=torch.uint8, device="cuda")
        qkv = torch.zeros((n + pad, (Hq + 2 * H) * D), dtype=dtype, device="cuda")
        k, v = token_rows(gen, n + pad, H, dtype)
        qkv[:, Hq * D:(Hq + H) * D] = k.view(n + pad, -1)
        qkv[:, (Hq + H) * D:] = v.view(n + pad, -1)
        st["k"] = qkv[:, Hq * D:(Hq + H) * D].view(n + pad, H, D)
        st["v"] = qkv[:, (Hq + H) * D:].view(n + pad, H, D)
    st["pages"] = pages
    if own:
        st["cache"] = handle(c, pages)
    return st


# --------------------------------------------------------------------- one pass
def run(state):
    c = state["c"]
    if own:
        return run_own(c, state)
    return {"plan": plain_plan, "append": plain_append, "gather": plain_gather, "decode": plain_decode}[c["op"]](c, state)


def run_own(c, st):
    if c["op"] == "plan":
        p = st["plan"].plan(st["ctx"], st["new"], st["table"], st["free"], st["count"], st["n_slots"], done=st["done"])
        return {"slots": p.slots, "positions": p.positions, "cu_new": p.cu_new, "seq_lens": p.seq_lens,
                "count": p.free_count, "table": st["table"], "free": st["free"]}
    if c["op"] == "append":
        st["cache"].append(st["k"], st["v"], st["slots"])
        return st["cache"].gather(st["slots"], st["k"].dtype, rotate_back=bool(c["back"]))
    if c["op"] == "gather":
        return st["cache"].gather(st["slots"], DTYPES[c["dtype"]], rotate_back=bool(c["back"]))
    return st["cache"].decode(st["q"], st["table"], st["lens"], st["max_len"], mask=st["mask"], workspace=st["ws"])


def plain_plan(c, st):
    P, B = c["P"], c["B"]
    dev = st["ctx"].device
    table, free = st["table"].clone(), st["free"].clone()
    max_pages, num = table.shape[1], st["num_pages"]
    ctx, new, done = st["ctx"].long().clamp(min=0), st["new"].long().clamp(min=0), st["done"] != 0
    count = st["count"].long()
    held = (ctx + P - 1) // P
    # finished requests give their pages back, in request order
    give = torch.where(done, held.clamp(max=max_pages), torch.zeros_like(held))
    col = torch.arange(max_pages, device=dev)
    rel = table[col[None, :] < give[:, None]]
    at = count + torch.arange(rel.shape[0], device=dev)
    free[at[at < num]] = rel[at < num]
    top = count + rel.shape[0]
    ctx = torch.where(done, torch.zeros_like(ctx), ctx)
    held = torch.where(done, torch.zeros_like(held), held)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), new.cumsum(0)])
    fits = (ctx + new <= max_pages * P) & (cu[1:] <= st["n_slots"])
    need = torch.where(fits, (ctx + new + P - 1) // P - held, torch.zeros_like(held))
    upto = need.cumsum(0)
    served = fits & ((need == 0) | (upto <= top))
    taken = torch.where(served & (need > 0), upto, torch.zeros_like(upto)).amax()
    # the new pages, popped from the top of the stack
    want = served[:, None] & (col[None, :] >= held[:, None]) & (col[None, :] < (held + need)[:, None])
    j = (upto - need)[:, None] + col[None, :] - held[:, None]
    page = free[(top - 1 - j).clamp(0, num - 1)]
    table = torch.where(want, page, table)
    # the slot of every new token
    t = torch.arange(st["n_slots"], device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
    real = (t < cu[-1]) & served[b]
    pos = ctx[b] + t - cu[b]
    slot = table[b, (pos // P).clamp(0, max_pages - 1)].long() * P + pos % P
    none = torch.full_like(slot, -1)
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"slots": i32(torch.where(real, slot, none)), "positions": i32(torch.where(real, pos, none)), "cu_new": i32(cu),
            "seq_lens": i32(torch.where(served, ctx + new, ctx)), "count": i32(top - taken), "table": table, "free": free}


def plain_append(c, st):
    k, v = st["k"].float(), st["v"].float()
    k = rotated(k) if c["rot"] else k
    v = rotated(v) if c["rotv"] else v
    out = []
    for x, bits, skip0, clip, rot in ((k, c["kb"], c["ch0"], 1.0, c["rot"]), (v, c["vb"], 0, c["clip"], c["rotv"])):
        code, s, z = quantized(x, bits, skip0, clip)
        y = (code.view(*x.shape[:-1], 4, 32).float() * s.float()[..., None] + z.float()[..., None]).view(x.shape)
        if skip0:
            y[..., 0] = x[..., 0].bfloat16().float()
        out.append(dense_rows(c, y, rot, st["slots"], st["k"].dtype))
    return out[0], out[1]


def dense_rows(c, y, rot, slots, dtype):
    """Rows as the caller gets them: rotated back when asked, zero where there is no token."""
    y = rotated(y) if rot and c["back"] else y
    return torch.where((slots >= 0)[:, None, None], y, torch.zeros_like(y)).to(dtype)


def plain_gather(c, st):
    pages, slots = st["pages"], st["slots"].long()
    n_pages, H, nb, size = pages.shape
    P = c["P"]
    s = slots.clamp(min=0)
    blocks, inverse = torch.unique(s // BT, return_inverse=True)  # each touched block once
    part = pages.permute(0, 2, 1, 3)[blocks // nb, blocks % nb].reshape(-1, size)
    k, v = unpack_blocks(c, part)
    row = lambda x: x.view(-1, H, BT, D)[inverse, :, s % BT]  # noqa: E731
    return tuple(dense_rows(c, row(x), rot, slots, DTYPES[c["dtype"]]) for x, rot in ((k, c["rot"]), (v, c["rotv"])))


def plain_decode(c, st):
    pages, table, q = st["pages"], st["table"].long().clamp(min=0), st["q"]
    n_pages, H, nb, size = pages.shape
    B, G, P = c["B"], c["G"], c["P"]
    T = table.shape[1] * P
    k, v = unpack_blocks(c, pages[table].transpose(1, 2).reshape(-1, size))
    k, v = k.view(B, H, T, D), v.view(B, H, T, D)
    qr = (rotated(q.float()) if c["rot"] else q.float()).view(B, H, G, D)
    if st["mask"] is not None:
        keep = (st["mask"].long()[:, :, None] >> torch.arange(32, device=q.device)) & 1
        qr = qr * keep.repeat_interleave(4, 2)[:, :, None, :].float()
    s = torch.matmul(qr, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    off = torch.arange(T, device=q.device)[None, :] >= st["lens"][:, None]
    s = s.masked_fill(off[:, None, None, :], -math.inf)
    m = s.amax(3, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    o = torch.matmul(e, v) / e.sum(3, keepdim=True).clamp(min=1e-30)  # an empty request's row is zero
    o = rotated(o) if c["rotv"] else o
    return o.view(B, H * G, D).to(q.dtype)


# --------------------------------------------------------------------- what a pass cannot do without
def token_bytes(c, keep=32):
    return keep * c["kb"] // 2 + 16 + (2 if c["ch0"] else 0) + D * c["vb"] // 8 + 16


def work(case):
    c = case
    if c["op"] == "plan":
        ctx, new, done = plan_lens(c)
        P = c["P"]
        moved = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(ctx, new)) + sum(-(-a // P) for a, d in zip(ctx, done) if d)
        return {"bytes": 4.0 * (5 * c["B"] + 2 * moved + 2 * (sum(new) + 5)), "flops": 0}
    if c["op"] == "decode":
        n = sum(seq_lens(c))
        e = 4 if c["dtype"] == "f32" else 2
        return {"bytes": float(n * c["H"] * token_bytes(c, c["keep"]) + 2 * e * c["B"] * c["H"] * c["G"] * D),
                "flops": 2.0 * n * c["H"] * c["G"] * (4 * c["keep"] + D)}
    e = 4 if c["dtype"] == "f32" else 2
    rows = c["n"] * c["H"]
    move = rows * (token_bytes(c) + 2 * D * e)
    if c["op"] == "append":  # the tokens in, their pages out, and the values they now stand for
        move += rows * 2 * D * e
    flops = 2.0 * rows * D * 7 * ((c["rot"] + c["rotv"]) * (2 if c["op"] == "append" and c["back"] else 1)) + 8.0 * rows * D
    return {"bytes": float(move), "flops": flops}


# --------------------------------------------------------------------- the same in 64 bits
def butterflies(x):
    x = x.double()
    h = 1
    while h < D:
        y = x.reshape(*x.shape[:-1], D // (2 * h), 2, h)
        x = torch.stack((y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]), -2).reshape(x.shape)
        h *= 2
    return x / math.sqrt(D)


def r32(x):
    return x.float().double()


def exact_values(x, bits, skip0, clip):
    """The values a row's codes stand for, in 64 bits: every rounding of the definition is made by name."""
    L = (1 << bits) - 1
    out = torch.empty_like(x, dtype=torch.float64)
    x = x.double()
    for g in range(4):
        y = x[..., 32 * g:32 * g + 32]
        rng = y[..., 1:] if skip0 and g == 0 else y
        c32 = float(torch.tensor(clip, dtype=torch.float32))
        lo, hi = r32(rng.min(-1, keepdim=True).values * c32), r32(rng.max(-1, keepdim=True).values * c32)
        s = r32(r32(hi - lo) / L).clamp(max=65504.0).half().double()
        z = lo.clamp(-65504.0, 65504.0).half().double()
        code = torch.where(s > 0, r32(r32(y - z) / s.clamp(min=1e-30)), torch.zeros_like(y)).round().clamp(0, L)
        out[..., 32 * g:32 * g + 32] = code * s + z
    if skip0:
        out[..., 0] = x[..., 0].float().bfloat16().double()
    return out


def exact_block_values(c, blocks):
    """Keys and values [N, 64, 128] in 64 bits, each code read at its byte and bit."""
    at, _ = code_bytes(c)
    dev = blocks.device
    t = torch.arange(BT, device=dev)[:, None]
    ch = torch.arange(D, device=dev)[None, :]
    p, g, i, e = ch // 4, t // 8, (t % 8) // 2, t % 2
    if c["kb"] == 4:
        byte = p * 128 + 16 * (g ^ (2 * (p & 3))) + 4 * i + 2 * ((ch % 4) // 2) + e
        bit = 4 * (ch % 2) + 0 * t
    else:
        byte = p * 64 + 8 * (g ^ (4 * ((p >> 1) & 1))) + t % 8
        bit = 2 * (ch % 4) + 0 * t
    kcode = (blocks[:, at["kc"][0]:][:, byte.reshape(-1)].long() >> bit.reshape(-1)) & ((1 << c["kb"]) - 1)
    vpos = 16 * (t // 16) + 4 * i + 2 * ((t % 16) // 8) + e
    per = 8 // c["vb"]
    vbyte = (ch // per) * 64 + vpos
    vcode = (blocks[:, at["vc"][0]:][:, vbyte.reshape(-1)].long() >> (c["vb"] * (ch % per) + 0 * t).reshape(-1)) & ((1 << c["vb"]) - 1)

    def halves(name):
        lo, hi = at[name]
        return blocks[:, lo:hi].contiguous().view(torch.float16).double()

    grp = torch.arange(4, device=dev)[None, :]
    pair = (((i * 8 + g) * 2 + e) * 4 + grp).reshape(-1)
    kz_at = (((((i // 2) * 8 + g) * 2 + grp // 2) * 2 + i % 2) * 2 + e) * 2 + grp % 2
    wide = lambda x: x.view(-1, BT, 4).repeat_interleave(32, 2)  # noqa: E731
    N = blocks.shape[0]
    k = kcode.view(N, BT, D).double() * wide(halves("ks")[:, pair]) + wide(halves("kz")[:, kz_at.reshape(-1)])
    v = vcode.view(N, BT, D).double() * wide(halves("vs")[:, pair]) + wide(halves("vz")[:, pair])
    if c["ch0"]:
        lo, hi = at["k0"]
        k[..., 0] = blocks[:, lo:hi].contiguous().view(torch.bfloat16).double()
    return k, v


def exact(case, seed):
    c = dict(case)
    if c["op"] == "plan":
        return None  # whole numbers only
    st = prepare(c, seed)
    if c["op"] == "append":
        got = []
        for x, bits, skip0, clip, rot in ((st["k"], c["kb"], c["ch0"], 1.0, c["rot"]), (st["v"], c["vb"], 0, c["clip"], c["rotv"])):
            x = x.double()
            x = butterflies(x).float() if rot else x.float()
            y = exact_values(x, bits, skip0, clip)
            y = butterflies(y) if rot and c["back"] else y
            got.append(y * (st["slots"] >= 0)[:, None, None])
        return got[0], got[1]
    pages = st["pages"]
    n_pages, H, nb, size = pages.shape
    if c["op"] == "gather":
        slots = st["slots"].long()
        out = [torch.zeros(slots.shape[0], H, D, dtype=torch.float64, device=pages.device) for _ in range(2)]
        for a in range(0, slots.shape[0], 2048):  # a slice of tokens at a time
            s = slots[a:a + 2048]
            on = s >= 0
            s = s[on]
            blk = s // BT
            used, inv = torch.unique(blk, return_inverse=True)
            for h in range(H):
                kv = exact_block_values(c, pages[used // nb, h, used % nb])
                for o, x, rot in zip(out, kv, (c["rot"], c["rotv"])):
                    y = x[inv, s % BT]
                    o[a:a + 2048, h][on] = butterflies(y) if rot and c["back"] else y
        return out[0], out[1]
    G, P = c["G"], c["P"]
    q = st["q"].double()
    q = butterflies(q).float().double() if c["rot"] else q
    out = torch.zeros(c["B"], H * G, D, dtype=torch.float64, device=pages.device)
    lens = seq_lens(c)
    for b in range(c["B"]):
        n = lens[b]
        if n == 0:
            continue
        ids = st["table"][b, :-(-n // P)].long()
        for h in range(H):
            k, v = exact_block_values(c, pages[ids, h].reshape(-1, size))
            k, v = k.view(-1, D)[:n], v.view(-1, D)[:n]
            qh = q[b, h * G:(h + 1) * G]
            if st["mask"] is not None:
                word = int(st["mask"][b, h]) & 0xFFFFFFFF
                qh = qh * torch.tensor([(word >> (x // 4)) & 1 for x in range(D)], dtype=torch.float64, device=q.device)
            w = torch.softmax(qh @ k.T / math.sqrt(D), 1)
            o = w @ v
            out[b, h * G:(h + 1) * G] = butterflies(o) if c["rotv"] else o
    return out
