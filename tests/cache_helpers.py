"""A plain paged cache in float64 for the tests: the stored values by the oracle's quantiser, and
attention with every option written out key by key, with a bound on what the kernels may be off by."""
import math

import numpy as np
import torch

import oracle as O
from kv_cache_compression_group_b200 import jolt as J

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def quantised(x, bits):
    """(packed codes, scales, values) of rows x [..., D] float64, by the oracle."""
    c, lo, step, val, ok = O.quantize(x, bits)
    assert ok.all()
    shape = x.shape[:-1]
    packed = O.pack_codes(c.reshape(-1, 16), bits).reshape(*shape, x.shape[-1] * bits // 8)
    scales = np.stack((lo, step), -1).reshape(*shape, x.shape[-1] // 16, 2)
    return packed, scales, val.reshape(x.shape)


class Paged:
    """A QuantCache of one layer with a batch over it, and the same in float64 on the host.

    lens, news: lengths with, and numbers of, the new rows.  Pages come in random order; what no row
    was written to holds NaN scales and random codes."""

    def __init__(self, lens, news, H, D, page, bits, seed=0, spare=2, spread=0.5, rows_behind=0, max_new=None,
                 extra_columns=0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.news, self.H, self.D, self.page = rng, list(lens), list(news), H, D, page
        self.bits = bits
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages)[:sum(need)]
        table = np.full((len(lens), max(need + [0]) + extra_columns), -7, np.int32)   # entries behind a sequence: never read
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table
        self.starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
        self.rows = int(self.starts[-1]) + rows_behind
        gain = np.exp(rng.standard_normal((H, D)) * spread)
        self.values = []                       # per sequence (K, V) [len, H, D] float64: what is stored
        self.dense = []
        pools = []
        for kv in range(2):
            b = bits[kv]
            codes = rng.integers(0, 256, (self.n_pages, H, page, D * b // 8)).astype(np.uint8)
            scales = np.full((self.n_pages, H, page, D // 16, 2), np.nan, np.float16)
            vals, dens = [], []
            for s, n in enumerate(lens):
                x = (rng.standard_normal((n, H, D)) * (gain if kv == 0 else 1.0)).astype(np.float32)
                x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
                dens.append(x)
                p, sc, v = quantised(x, b) if n else (None, None, np.zeros((0, H, D)))
                vals.append(v)
                for t in range(n):
                    codes[table[s, t // page], :, t % page] = p[t]
                    scales[table[s, t // page], :, t % page] = sc[t]
            self.values.append(vals)
            self.dense.append(dens)
            pools += [codes, scales]
        self.pools_np = pools
        self.pools = tuple(torch.from_numpy(p)[None].cuda() for p in pools)
        self.cache = J.QuantCache(1, H, D, self.n_pages, page, bits, pools=self.pools)
        self.batch = J.CacheBatch(torch.from_numpy(table).cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(),
                                  torch.from_numpy(self.starts).cuda(),
                                  max(self.news + [0]) if max_new is None else max_new)

    def new_rows(self, dtype, kv):
        """The new rows of K (0) or V (1) as they were before they were stored."""
        x = [d[n - m:] for d, n, m in zip(self.dense[kv], self.lens, self.news)]
        return torch.from_numpy(np.concatenate(x)).to(dtype)


def refill(p, kv, rows):
    """Store rows (one [len, H, D] array per sequence) as the keys (0) or values (1) of p."""
    for s, x in enumerate(rows):
        codes, scales, p.values[kv][s] = quantised(np.asarray(x, np.float64), p.bits[kv])
        t = np.arange(p.lens[s])
        at = p.table[s, t // p.page], slice(None), t % p.page
        p.pools_np[2 * kv][at], p.pools_np[2 * kv + 1][at] = codes, scales
    for i in (2 * kv, 2 * kv + 1):
        p.pools[i][0].copy_(torch.from_numpy(p.pools_np[i]))


def tree(rng, news, width):
    """(mask words, depths) of a random tree of drafted tokens for every sequence."""
    words = max(1, -(-max(news + [0]) // 32))
    mask, depth = [], []
    for n in news:
        seen, deep = [], []
        for i in range(n):
            parent = int(rng.integers(max(0, i - width), i)) if i else -1
            seen.append((seen[parent] if i else 0) | (1 << i))
            deep.append(deep[parent] + 1 if i else 0)
        mask += [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for m in seen]
        depth += deep
    return np.array(mask, np.uint32).reshape(-1, words), np.array(depth, np.int32)


def magnitude(v):
    """|v| + (v - lo) of stored values [..., D], numpy or torch; lo, the block's lower end, is its least
    value, or below it by less than fp16's step there, 2^-10 |lo|, which |v| covers."""
    blocks = v.reshape(*v.shape[:-1], v.shape[-1] // 16, 16)
    low = blocks.min(-1, keepdims=True) if isinstance(v, np.ndarray) else blocks.min(-1, keepdim=True).values
    return (abs(blocks) + (blocks - low)).reshape(v.shape)


def plain_attend(p, q, scale=0.0, softcap=0.0, window=0, slopes=None, positions=None, mask=None, prefix=None,
                 skip=(), lost=()):
    """(output, bound) float64 [rows, n_q_heads, D].  q float64.  skip: sequences the call leaves
    out; lost: (sequence, page column) pairs whose keys nobody sees.

    The bound, with u = 2^-11 (half a step of fp16; 2^-25 for a value below its normal range): the
    stored values enter the products rounded to fp16, so a score is off by at most
    d = u scale sum |q_d k_d| (+ fp32 sums), every normalised weight by a factor e^(2d), and the
    output by (e^(2d) - 1) 2 sum p|v|.  Beside that, either the weights and the values are rounded, 2 u
    sum p|v|; or, where the products take the codes, v = lo + c step is summed as sum fl(p) lo +
    sum fl(fl(p) step) c: the first rounding of p is common to both and costs u sum p|v|, the second
    u sum p c step = u sum p (v - lo).  Both are at most 2 u sum p (|v| + v - lo) (see magnitude)."""
    rows, nq, D = q.shape
    G = nq // p.H
    out, tol = np.full(q.shape, np.nan), np.zeros(q.shape)
    scale = scale or 1.0 / math.sqrt(D)
    for b, (length, n) in enumerate(zip(p.lens, p.news)):
        if b in skip:
            continue
        r0, old = int(p.starts[b]), length - n
        pos_k = np.arange(length)
        if positions is not None:
            pos_k[old:] = positions[r0:r0 + n]
        for i in range(n):
            pq = int(pos_k[old + i])
            seen = np.ones(length, bool)
            for j in range(n):
                seen[old + j] = (j <= i) if mask is None else bool((int(mask[r0 + i, j // 32]) >> (j % 32)) & 1)
            if window:
                seen &= pq - pos_k < window
            for s, col in lost:
                if s == b:
                    seen[col * p.page:(col + 1) * p.page] = False
            for h in range(nq):
                k, v = p.values[0][b][:, h // G][seen], p.values[1][b][:, h // G][seen]
                x = q[r0 + i, h]
                s = scale * (k @ x)
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - float(slopes[h]) * (pq - pos_k[seen])
                d = scale * (np.abs(k) @ np.abs(x)) * (2.0 ** -11 + 2.0 ** -20) + 2.0 ** -20 * np.abs(s) + scale * 2.0 ** -24 * np.abs(x).sum()
                vs, ms, d = v, magnitude(v), (d.max() if d.size else 0.0)
                if prefix is not None:
                    s = np.append(s, prefix[1][r0 + i, h])
                    vs = np.concatenate((v, prefix[0][r0 + i, h][None]))
                    ms = np.concatenate((ms, np.abs(prefix[0][r0 + i, h])[None]))
                if not s.size or s.max() == -np.inf:
                    out[r0 + i, h] = 0.0
                    continue
                w = np.exp(s - s.max())
                w /= w.sum()
                out[r0 + i, h] = w @ vs
                mag = w @ ms + 2.0 ** -14
                tol[r0 + i, h] = mag * (2 * math.expm1(2 * d) + 2 * 2.0 ** -11 + 2.0 ** -18)
    return out, tol


def check_attend(p, dtype, nq, seed=1, q_scale=1.0, stream=None, **kw):
    """One call against plain_attend; returns the output."""
    rng = np.random.default_rng(seed)
    q = torch.from_numpy(rng.standard_normal((p.rows, nq, p.D)) * q_scale).to(dtype)
    dev = {}
    for name, dt in (("slopes", torch.float32), ("positions", torch.int32)):
        if kw.get(name) is not None:
            dev[name] = torch.from_numpy(np.asarray(kw[name])).to(dt).cuda()
    if kw.get("mask") is not None:
        dev["mask"] = torch.from_numpy(np.ascontiguousarray(kw["mask"]).view(np.int32)).cuda()
    if kw.get("prefix") is not None:
        dev["prefix"] = tuple(torch.from_numpy(x).float().cuda() for x in kw["prefix"])
    calls = {k: v for k, v in kw.items() if k in ("scale", "softcap", "window")}
    before = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    got = p.cache.attend(0, q.cuda(), p.batch, out=before, **calls, **dev)
    want, tol = plain_attend(p, q.double().numpy(), **kw)
    got64 = got.double().cpu().numpy()
    told = ~np.isnan(want)
    assert (got64[~told] == 7.0).all(), "a row that belongs to no sequence was written"
    off = np.abs(got64 - want)[told] - (tol + HALF_STEP[dtype] * (np.abs(want) + tol))[told] - 1e-7
    assert off.size == 0 or off.max() <= 0, (off.max(), int((off > 0).sum()), off.size)
    return got
