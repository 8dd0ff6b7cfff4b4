"""Measured cases of the quantised paged KV cache: writing it, reading it back, attending over it.

A request's prompt cache is compressed once (``jolt_compress``); what is generated after it, and
whole caches that are not compressed with factors, live in pages of block-quantised rows.  One
cache serves three operators, and each case is one pass through them as a serving loop makes it:

  store   new rows of keys and values are quantised into their pages and read back as values (a
          prompt whose attention is to see the values that later steps will see)
  read    stored rows are read back as dense rows
  attend  new query rows (one per sequence, a tree of drafted tokens, or a chunk of a prompt)
          attend over the pages
  step    a decode step: the new rows are written, then attended over

With ``own`` false, ``run`` computes the same in elementary torch operations in 32 bits (the
quantiser in 64: its codes sit next to ties), rounded once at the end.
"""
import math
import random

import torch

own = False

BLK = 16          # values that share one (lo, step) pair
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _c(name, op, batch, ctx, new, heads, group, dim, page, bits_k, bits_v, dtype, **kw):
    c = dict(name=name, op=op, batch=batch, ctx=ctx, new=new, heads=heads, group=group, dim=dim, page=page,
             bits_k=bits_k, bits_v=bits_v, dtype=dtype, ragged=False, softcap=0.0, window=0, bias=False, tree=False,
             prefix=False)
    c.update(kw)
    return c


def listed():
    return [
        # the rows of one decode step of a batch: latency only
        _c("store_step", "store", 64, 1000, 1, 8, 4, 128, 16, 4, 4, "bf16", ragged=True),
        # a whole long prompt written at once, keys at 8 bits, values at 4
        _c("store_prompt", "store", 1, 65536, 65536, 8, 4, 128, 64, 8, 4, "bf16"),
        # several fp32 prompts of odd lengths, 2 bits
        _c("store_ragged", "store", 8, 1021, 1021, 8, 4, 64, 32, 2, 2, "fp32", ragged=True),
        # a batch of 40-head caches read back in half precision
        _c("read_batch", "read", 4, 4096, 4096, 40, 1, 128, 64, 4, 4, "fp16", ragged=True),
        # one long 8-bit cache read back to fp32
        _c("read_long", "read", 1, 32768, 32768, 8, 4, 128, 256, 8, 8, "fp32"),
        # one short sequence, one token: the shortest call of a serving loop
        _c("step_short", "step", 1, 1000, 1, 8, 4, 128, 16, 4, 4, "bf16"),
        # one long context, one token
        _c("attend_long", "attend", 1, 65536, 1, 8, 4, 128, 64, 4, 4, "bf16"),
        # a ragged batch with capped scores and a sliding window, keys at 8 bits
        _c("attend_batch", "attend", 64, 8192, 1, 8, 4, 128, 32, 8, 4, "bf16", ragged=True, softcap=30.0, window=4096),
        # no grouped heads, a distance bias, 2 bits; behind a prefix attended elsewhere
        _c("attend_mha", "attend", 8, 4096, 1, 40, 1, 128, 128, 2, 2, "fp16", ragged=True, bias=True, prefix=True),
        # small trees of drafted tokens over 64-wide heads
        _c("tree_small", "step", 4, 16384, 8, 8, 4, 64, 64, 8, 8, "fp16", ragged=True, tree=True, bias=True),
        # wide trees over a batch
        _c("tree_batch", "step", 16, 8192, 32, 8, 4, 128, 64, 4, 4, "bf16", ragged=True, tree=True),
        # a chunk of a prompt over what was written before it
        _c("chunk", "attend", 1, 16384, 2048, 8, 4, 128, 64, 4, 4, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "read", "attend", "attend", "step", "step"])
    heads, group = rng.choice([(8, 4), (8, 4), (8, 1), (40, 1), (4, 7), (1, 8), (8, 8), (2, 16)])
    c = _c("", op, 1, 1, 1, heads, group, rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128, 256]),
           rng.choice([2, 4, 4, 8]), rng.choice([2, 4, 4, 8]), rng.choice(["bf16", "bf16", "fp16"]), ragged=rng.random() < 0.7)
    del c["name"]
    if op in ("store", "read"):
        if rng.random() < 0.3:
            c["dtype"] = "fp32"
        rows = min(_log(rng, 1, 65536), (65536 * 8) // heads)
        c["batch"] = min(rows, _log(rng, 1, 64))
        c["new"] = max(1, rows // c["batch"])
        c["ctx"] = c["new"] + (rng.randrange(200) if rng.random() < 0.5 else 0)
        return c
    c["batch"] = _log(rng, 1, 64)
    kind = rng.random()
    c["new"] = 1 if kind < 0.5 else _log(rng, 2, 64) if kind < 0.85 else _log(rng, 65, 2048)
    tokens = 65536 * 8 // heads                       # of context, over the batch
    if c["new"] > 64:                                 # a chunk: at most the listed one's products
        c["batch"] = rng.choice([1, 1, 2])
        tokens = min(tokens, int(2048 * 16384 * 32 / (c["new"] * heads * group)))
        c["ragged"] = False
    c["ctx"] = max(c["new"], min(_log(rng, 16, 65536), tokens // c["batch"]))
    c["tree"] = 1 < c["new"] <= 64 and rng.random() < 0.7
    c["softcap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
    c["window"] = rng.choice([0, 0, 128, 1024, 4096])
    c["bias"] = rng.random() < 0.3
    c["prefix"] = rng.random() < 0.2
    return c


# ---- sizes that the case alone fixes ------------------------------------------------------
def _lengths(case):
    """(length of each sequence with its new rows, new rows of each sequence)."""
    r = random.Random("%d %d %d" % (case["batch"], case["ctx"], case["new"]))
    lens, news = [], []
    for b in range(case["batch"]):
        n = case["new"]
        if case["ragged"] and b and n > 1:
            n = r.randint((n + 1) // 2, n)
        old = case["ctx"] - case["new"]
        if case["ragged"] and b and old:
            old = r.randint(old // 4, old)
        lens.append(old + n)
        news.append(n)
    return lens, news


def _row_bytes(case):
    """Stored bytes of one token's keys and values over all heads."""
    d = case["dim"]
    return case["heads"] * (d * (case["bits_k"] + case["bits_v"]) // 8 + 2 * 4 * d // BLK)


def work(case):
    lens, news = _lengths(case)
    rows, esz, d = sum(news), 4 if case["dtype"] == "fp32" else 2, case["dim"]
    dense = 2 * rows * case["heads"] * d * esz
    stored = rows * _row_bytes(case)
    if case["op"] == "store":       # in, stored, stored read again, out
        return {"bytes": 2 * dense + 2 * stored, "flops": 0}
    if case["op"] == "read":
        return {"bytes": stored + dense, "flops": 0}
    nq = case["heads"] * case["group"]
    seen = pairs = 0
    for length, n in zip(lens, news):
        old = length - n
        kept = min(old, case["window"] - 1) if case["window"] else old
        seen += kept + n
        pairs += n * kept + n * (n + 1) // 2
    w = {"bytes": seen * _row_bytes(case) + 2 * rows * nq * d * esz + (rows * nq * (d + 1) * 4 if case["prefix"] else 0),
         "flops": 4 * d * nq * pairs}
    if case["op"] == "step":
        w["bytes"] += dense         # the new rows come in (they are among the stored ones above)
    return w


# ---- inputs -------------------------------------------------------------------------------
def _fill(g, pages, heads, page, dim, bits, spread):
    """A pool of written pages: Gaussian rows with a scale per channel, as codes and (lo, step)."""
    dev, lev = "cuda", (1 << bits) - 1
    gain = torch.exp(torch.randn(heads, 1, dim, generator=g, device=dev) * spread)
    codes = torch.empty(pages, heads, page, dim * bits // 8, dtype=torch.uint8, device=dev)
    scales = torch.empty(pages, heads, page, dim // BLK, 2, dtype=torch.float16, device=dev)
    shift = torch.arange(0, 8, bits, device=dev, dtype=torch.uint8)
    step_pages = max(1, (1 << 25) // (heads * page * dim))
    for p in range(0, pages, step_pages):
        n = min(step_pages, pages - p)
        x = (torch.randn(n, heads, page, dim, generator=g, device=dev) * gain).view(n, heads, page, dim // BLK, BLK)
        mn, mx = x.aminmax(dim=-1)
        lo = mn.half()
        step = ((mx - lo.float()) / lev).half()
        c = ((x - lo.float()[..., None]) / step.float()[..., None]).round_().clamp_(0, lev).to(torch.uint8)
        c = c.view(n, heads, page, dim * bits // 8, 8 // bits)
        codes[p:p + n] = (c << shift).sum(-1, dtype=torch.uint8)
        scales[p:p + n] = torch.stack((lo, step), -1)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    dev, dt = "cuda", DTYPES[case["dtype"]]
    lens, news = _lengths(case)
    H, D, P, B = case["heads"], case["dim"], case["page"], case["batch"]
    need = [-(-n // P) for n in lens]
    pages = sum(need) + 3                       # a few pages belong to nobody
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[:sum(need)].to(torch.int32)
    table = torch.zeros(B, max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    rows, nq = starts[-1], H * case["group"]
    s = {"case": case, "table": table.to(dev), "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "starts": torch.tensor(starts, dtype=torch.int32, device=dev), "max_len": max(lens), "max_new": max(news),
         "rows": rows}
    s["k_codes"], s["k_scales"] = _fill(g, pages, H, P, D, case["bits_k"], 1.0)
    s["v_codes"], s["v_scales"] = _fill(g, pages, H, P, D, case["bits_v"], 0.0)
    if case["op"] in ("store", "step"):
        gain = torch.exp(torch.randn(H, D, generator=g, device=dev))
        s["k"] = (torch.randn(rows, H, D, generator=g, device=dev) * gain).to(dt)
        s["v"] = torch.randn(rows, H, D, generator=g, device=dev).to(dt)
    if case["op"] in ("attend", "step"):
        s["q"] = (torch.randn(rows, nq, D, generator=g, device=dev) * 0.5).to(dt)
        s["slopes"] = None
        if case["bias"]:
            s["slopes"] = torch.tensor([2.0 ** (-8.0 * (j + 1) / nq) for j in range(nq)], device=dev)
        s["mask"] = s["positions"] = None
        if case["tree"]:
            words = -(-max(news) // 32)
            mask, pos = [], []
            for length, n in zip(lens, news):
                seen, depth = [], []
                for i in range(n):
                    parent = r.randint(max(0, i - 6), i - 1) if i else -1
                    seen.append((seen[parent] if i else 0) | (1 << i))
                    depth.append(depth[parent] + 1 if i else 0)
                mask += [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for m in seen]
                pos += [length - n + d for d in depth]
            mask = torch.tensor(mask, dtype=torch.int64)
            s["mask"] = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32).to(dev)
            s["positions"] = torch.tensor(pos, dtype=torch.int32, device=dev)
        s["prefix"] = None
        if case["prefix"]:
            s["prefix"] = (torch.randn(rows, nq, D, generator=g, device=dev) * 0.1,
                           torch.randn(rows, nq, generator=g, device=dev) + 6.0)
    if own:
        from kv_cache_compression_group_b200 import jolt
        s["cache"] = jolt.QuantCache(1, H, D, pages, P, (case["bits_k"], case["bits_v"]),
                                     pools=tuple(s[n][None] for n in ("k_codes", "k_scales", "v_codes", "v_scales")))
        s["batch"] = jolt.CacheBatch(s["table"], s["lens"], s["starts"], s["max_new"])
    return s


# ---- one pass -----------------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        cache, batch = s["cache"], s["batch"]
        if op in ("store", "step"):
            cache.write(0, s["k"], s["v"], batch)
        if op in ("store", "read"):
            return cache.read(0, batch, s["rows"], DTYPES[case["dtype"]])
        return cache.attend(0, s["q"], batch, softcap=case["softcap"], window=case["window"], slopes=s["slopes"],
                            positions=s["positions"], mask=s["mask"], prefix=s["prefix"])
    if op in ("store", "step"):
        b, i = _rows(s)
        page, slot = _place(s, b, i)
        for x, codes, scales, bits in ((s["k"], s["k_codes"], s["k_scales"], case["bits_k"]),
                                       (s["v"], s["v_codes"], s["v_scales"], case["bits_v"])):
            c, sc = _quantise(x, bits)
            codes[page, :, slot] = c
            scales[page, :, slot] = sc
    if op in ("store", "read"):
        b, i = _rows(s)
        page, slot = _place(s, b, i)
        dt = DTYPES[case["dtype"]]
        return (_values(s["k_codes"][page, :, slot], s["k_scales"][page, :, slot], case["bits_k"]).to(dt),
                _values(s["v_codes"][page, :, slot], s["v_scales"][page, :, slot], case["bits_v"]).to(dt))
    return _attend(s)


def _rows(s):
    """Sequence and place within it of every new row."""
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["starts"], r, right=True) - 1
    return b, r - s["starts"][b]


def _place(s, b, i):
    """Page and slot of new row i of sequence b: the new rows are the last of their sequence."""
    at = s["lens"][b] - (s["starts"][b + 1] - s["starts"][b]) + i
    return s["table"][b, at // s["case"]["page"]].long(), at % s["case"]["page"]


def _next_half(h, up):
    """The next fp16 number above (or below) h."""
    i = h.view(torch.int16).to(torch.int32)
    ordered = torch.where(i < 0, -32768 - i, i) + (1 if up else -1)   # -0 and +0 are the same place
    back = torch.where(ordered < 0, -32768 - ordered, ordered)
    return back.to(torch.int16).view(torch.float16)


def _quantise(x, bits):
    lev = (1 << bits) - 1
    x = x.double().view(*x.shape[:-1], -1, BLK)
    mn, mx = x.aminmax(dim=-1)
    lo = mn.half()
    lo = torch.where(lo.double() > mn, _next_half(lo, False), lo)
    ideal = (mx - lo.double()) / lev
    step = ideal.half()
    step = torch.where(step.double() < ideal, _next_half(step, True), step)
    div = torch.where(step > 0, step, torch.ones_like(step)).double()
    c = ((x - lo.double()[..., None]) / div[..., None]).round().clamp(0, lev)
    c = (c * (step > 0)[..., None]).to(torch.uint8).view(*x.shape[:-2], -1, 8 // bits)
    shift = torch.arange(0, 8, bits, device=c.device, dtype=torch.uint8)
    return (c << shift).sum(-1, dtype=torch.uint8), torch.stack((lo, step), -1)


def _values(codes, scales, bits):
    shift = torch.arange(0, 8, bits, device=codes.device, dtype=torch.uint8)
    c = ((codes[..., None] >> shift) & ((1 << bits) - 1)).float()
    c = c.view(*scales.shape[:-1], BLK)
    return (scales[..., 0].float()[..., None] + c * scales[..., 1].float()[..., None]).flatten(-2)


def _attend(s):
    case = s["case"]
    B, H, G, D, L, n = case["batch"], case["heads"], case["group"], case["dim"], s["max_len"], s["max_new"]
    t = torch.arange(L, device="cuda")
    page, slot = s["table"][:, t // case["page"]].long(), (t % case["page"]).expand(B, L)
    kx = _values(s["k_codes"][page, :, slot], s["k_scales"][page, :, slot], case["bits_k"])       # [B, L, H, D]
    b, i = _rows(s)
    q = torch.zeros(B, n, H * G, D, device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    sc = torch.matmul(q, kx.permute(0, 2, 3, 1)).view(B, H, G, n, L) / math.sqrt(D)
    del kx
    if case["softcap"]:
        sc = case["softcap"] * torch.tanh(sc / case["softcap"])
    count = (s["starts"][1:] - s["starts"][:-1]).long()
    old = (s["lens"] - count).long()
    node = t[None, :] - old[:, None]                                   # [B, L] which new row a key is
    row = torch.arange(n, device="cuda")
    pos_q = old[:, None] + row                                         # [B, n]
    pos_k = t.expand(B, L)
    if s["positions"] is not None:
        pos_q = torch.zeros(B, n, dtype=torch.long, device="cuda")
        pos_q[b, i] = s["positions"].long()
        pos_k = torch.where(node < 0, pos_k, torch.gather(pos_q, 1, node.clamp(0, n - 1)))
    if s["mask"] is not None:
        words = torch.zeros(B, n, s["mask"].shape[1], dtype=torch.int32, device="cuda")
        words[b, i] = s["mask"]
        at = node.clamp(0, n - 1)
        w = torch.gather(words, 2, (at // 32)[:, None].expand(B, n, L))
        seen = ((w >> (at % 32)[:, None].int()) & 1) == 1
    else:
        seen = node[:, None] <= row[:, None]
    seen = (node[:, None] < 0) | (seen & (node < count[:, None])[:, None])
    far = pos_q[:, :, None] - pos_k[:, None]                           # [B, n, L]
    if case["window"]:
        seen = seen & (far < case["window"])
    if s["slopes"] is not None:
        sc = sc - s["slopes"].view(H, G)[None, :, :, None, None] * far[:, None, None].float()
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    if s["prefix"] is not None:
        p_out = torch.zeros(B, n, H * G, D, device="cuda")
        p_lse = torch.full((B, n, H * G), -math.inf, device="cuda")
        p_out[b, i], p_lse[b, i] = s["prefix"]
        p_out = p_out.view(B, n, H, G, D).permute(0, 2, 3, 1, 4)
        p_lse = p_lse.view(B, n, H, G).permute(0, 2, 3, 1)[..., None]
        top = torch.maximum(top, p_lse)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(sc - top)
    del sc
    total = p.sum(-1, keepdim=True)
    vx = _values(s["v_codes"][page, :, slot], s["v_scales"][page, :, slot], case["bits_v"])
    vx = vx.masked_fill((t[None] >= s["lens"][:, None])[:, :, None, None], 0.0)
    out = torch.matmul(p.view(B, H, G * n, L), vx.permute(0, 2, 1, 3)).view(B, H, G, n, D)
    if s["prefix"] is not None:
        w = torch.exp(p_lse - top)
        out, total = out + w * p_out, total + w
    out = out / torch.where(total > 0, total, torch.ones_like(total))
    return out.permute(0, 3, 1, 2, 4).reshape(B, n, H * G, D)[b, i].to(s["q"].dtype)


# ---- the definition in 64 bits ------------------------------------------------------------
def _round_half(x, up):
    """x rounded towards +inf (up) or -inf to a multiple of the fp16 spacing at |x|."""
    _, e = torch.frexp(x)
    ulp = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-14) - 10)
    return (torch.ceil(x / ulp) if up else torch.floor(x / ulp)) * ulp


def _stored_values(x, bits):
    """The values that rows x stand for once they are stored with this many bits."""
    x = x.double()
    blocks = x.unflatten(-1, (-1, BLK))
    lo = _round_half(blocks.min(-1, keepdim=True).values, False)
    step = _round_half((blocks.max(-1, keepdim=True).values - lo) / (2 ** bits - 1), True)
    code = torch.where(step > 0, torch.round((blocks - lo) / step), torch.zeros_like(blocks))
    return (lo + code.clamp(0, 2 ** bits - 1) * step).flatten(-2)


def _pool_values(codes, scales, bits):
    """Values of pool entries, by a table of what each byte holds."""
    per = 8 // bits
    held = torch.tensor([[(v >> (bits * j)) % (1 << bits) for j in range(per)] for v in range(256)],
                        dtype=torch.float64, device=codes.device)
    c = held[codes.long()].flatten(-2).unflatten(-1, (-1, BLK))
    sc = scales.double()
    return (c * sc[..., 1:] + sc[..., :1]).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    lens, news = _lengths(case)
    H, G, D, P = case["heads"], case["group"], case["dim"], case["page"]
    if case["op"] == "store":
        return _stored_values(s["k"], case["bits_k"]), _stored_values(s["v"], case["bits_v"])
    outs, first = [], 0
    for b, (length, n) in enumerate(zip(lens, news)):
        t = torch.arange(length - n if case["op"] == "read" else 0, length, device="cuda")
        page, slot = s["table"][b][t // P].long(), t % P
        kx = _pool_values(s["k_codes"][page, :, slot], s["k_scales"][page, :, slot], case["bits_k"])   # [L, H, D]
        vx = _pool_values(s["v_codes"][page, :, slot], s["v_scales"][page, :, slot], case["bits_v"])
        mine = slice(first, first + n)
        first += n
        if case["op"] == "read":
            outs.append((kx, vx))
            continue
        if case["op"] == "step":
            kx[length - n:] = _stored_values(s["k"][mine], case["bits_k"])
            vx[length - n:] = _stored_values(s["v"][mine], case["bits_v"])
        seen = torch.ones(n, length, dtype=torch.bool, device="cuda")
        pos_k = torch.arange(length, device="cuda", dtype=torch.float64)
        if s["positions"] is not None:
            pos_k[length - n:] = s["positions"][mine].double()
        pos_q = pos_k[length - n:].clone()
        if s["mask"] is not None:
            bits = [[(int(w) >> j) & 1 for w in row for j in range(32)][:n] for row in s["mask"][mine].cpu().tolist()]
            seen[:, length - n:] = torch.tensor(bits, device="cuda") == 1
        else:
            seen[:, length - n:] = torch.ones(n, n, device="cuda").tril() == 1
        far = pos_q[:, None] - pos_k
        if case["window"]:
            seen &= far < case["window"]
        out = torch.empty(n, H * G, D, dtype=torch.float64, device="cuda")
        for j in range(H * G):
            sc = s["q"][mine, j].double() @ kx[:, j // G].T * D ** -0.5
            if case["softcap"]:
                sc = torch.tanh(sc / case["softcap"]) * case["softcap"]
            if s["slopes"] is not None:
                sc = sc - s["slopes"][j].double() * far
            sc[~seen] = -math.inf
            values = vx[:, j // G]
            if s["prefix"] is not None:     # the prefix is one more key, whose value is its output
                o, lse = s["prefix"][0][mine, j].double(), s["prefix"][1][mine, j].double()
                p = torch.softmax(torch.cat((sc, lse[:, None]), 1), 1)
                out[:, j] = p[:, :-1] @ values + p[:, -1:] * o
            else:
                out[:, j] = torch.softmax(sc, 1) @ values
        outs.append(out)
    if case["op"] == "read":
        return torch.cat([o[0] for o in outs]), torch.cat([o[1] for o in outs])
    return torch.cat(outs)
