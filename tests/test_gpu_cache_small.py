"""Attention of the paged cache over rows of small values, in each of its kernels, against float64.

A stored value is lo + code * step of its block.  Where it enters the products in fp16, it does as
2 fl(fl(lo / 2) + step code / 2): the sum is rounded by at most 2^-11 of itself or 2^-25, below fp16's
normal range lo / 2 by at most 2^-25 before it, so the value is off by at most 2^-11 |v| + 2^-23."""
import numpy as np
import pytest
import torch

from cache_helpers import Paged, quantised

pytestmark = pytest.mark.gpu

VALUE, LEAST = 2.0 ** -11, 2.0 ** -23
# query heads of the one KV head: one row to two n-tiles in the codes' kernel, one to four in the next,
# jobs of 128 and of 256 rows on the tensor cores
ROWS = [1, 4, 7, 12, 24, 40, 160]
SIZES = [1.0, 1e-2, 1e-3, 1e-4, 1e-5]


def refill(p, kv, rows):
    """Store rows (one [len, H, D] array per sequence) as the keys (0) or values (1) of p."""
    for s, x in enumerate(rows):
        codes, scales, p.values[kv][s] = quantised(np.asarray(x, np.float64), p.bits[kv])
        for t in range(p.lens[s]):
            at = p.table[s, t // p.page], slice(None), t % p.page
            p.pools_np[2 * kv][at], p.pools_np[2 * kv + 1][at] = codes[t], scales[t]
    for i in (2 * kv, 2 * kv + 1):
        p.pools[i][0].copy_(torch.from_numpy(p.pools_np[i]))


def fp16_out(want, tol):
    """Bound of an fp16 output whose value before its rounding is want, off by at most tol."""
    return tol + np.maximum(VALUE * (np.abs(want) + tol), 2.0 ** -25) + 2.0 ** -18 * (np.abs(want) + tol)


def check(got, want, tol):
    off = np.abs(got.double().cpu().numpy() - want) - fp16_out(want, tol)
    assert off.max() <= 0, (off.max(), int((off > 0).sum()), off.size)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("G", ROWS)
def test_a_lone_value(G, bits, D, size):
    """A row that sees one key gives that key's value, whatever the number of rows."""
    p = Paged([1] * 4, [1] * 4, 1, D, 16, (4, bits))
    rng = np.random.default_rng(bits)
    refill(p, 1, [rng.standard_normal((1, 1, D)) * size for _ in range(4)])
    q = torch.from_numpy(rng.standard_normal((4, G, D))).half()
    got = p.cache.attend(0, q.cuda(), p.batch)
    want = np.concatenate(p.values[1]).repeat(G, 1)
    check(got, want, VALUE * np.abs(want) + LEAST)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("G", ROWS)
def test_small_keys(G, bits, D, size):
    """Two keys with the values 1 and -1: the output is tanh((s0 - s1) / 2), off by at most half of what
    the scores are off by, and by both weights' rounding, 2^-11 each."""
    p = Paged([2] * 4, [1] * 4, 1, D, 16, (bits, 4))
    rng = np.random.default_rng(bits)
    refill(p, 0, [rng.standard_normal((2, 1, D)) * size for _ in range(4)])
    refill(p, 1, [np.array([1.0, -1.0])[:, None, None] * np.ones((2, 1, D))] * 4)
    q = torch.from_numpy(rng.standard_normal((4, G, D))).half()
    scale = float(np.float32(1.0 / size / D ** 0.5))
    got = p.cache.attend(0, q.cuda(), p.batch, scale=scale)
    k, x = np.stack([v[:, 0] for v in p.values[0]]), q.double().numpy()      # [4, 2, D], [4, G, D]
    s = scale * np.einsum("btd,bgd->bgt", k, x)
    off = scale * np.einsum("btd,bgd->bgt", VALUE * np.abs(k) + LEAST, np.abs(x)) + 2.0 ** -18 * (1 + np.abs(s))
    want, tol = np.tanh((s[..., 0] - s[..., 1]) / 2), off.sum(-1) / 2 + 2.0 ** -10
    check(got, np.repeat(want[..., None], D, -1), np.repeat(tol[..., None], D, -1))
