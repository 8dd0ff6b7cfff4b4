"""Attention of the paged cache over rows of small values, in each of its kernels, against float64.

A stored value is lo + code * step of its block.  Where it enters the products in fp16, it does as
2 fl(fl(lo / 2) + step code / 2): the sum is rounded by at most 2^-11 of itself or 2^-25, below fp16's
normal range lo / 2 by at most 2^-25 before it, so the value is off by at most 2^-11 |v| + 2^-23."""
import numpy as np
import pytest
import torch

from cache_helpers import Paged, refill
from kv_cache_compression_group_b200 import jolt as J

pytestmark = pytest.mark.gpu

VALUE, LEAST = 2.0 ** -11, 2.0 ** -23
# query heads of the one KV head: one row to two n-tiles in the codes' kernel, one to four in the next,
# jobs of 128 and of 256 rows on the tensor cores
ROWS = [1, 4, 7, 12, 24, 40, 160]
SIZES = [1.0, 1e-2, 1e-3, 1e-4, 1e-5]


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


@pytest.mark.parametrize("size", [1e4, 1.0, 1e-2, 1e-4, "blocks", "growing", "shrinking"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("G", ROWS)
def test_low_weights_of_small_values(G, bits, D, size):
    """16 keys of weight 1 among the first 256, then 65280 with those between them of weight 2^-12: half of the
    output is theirs.  Sequences enough that a thread block, and in it every warp, has some of the
    high ones and thousands of the low ones.  size: of all values; "blocks": from 1e4 to 1e-4 by blocks of
    features; "growing", "shrinking": the later keys' 1000 times as large, or as small.

    Off by: a weight's rounding, 2^-11 of it (all are above fp16's subnormal numbers), and either the
    value's (see above), or, where the products take the codes, that of weight times step, 2^-11 of it: sum
    p (v - lo) 2^-11, where v - lo is code times step."""
    seqs, page, pages = 600, 64, 1024
    p = Paged([2 * page], [1], 1, D, page, (4, bits))
    rng = np.random.default_rng(bits)
    high = np.arange(2 * page) % 16 == 5
    high[page:] = False
    # one value per block: stored exactly
    refill(p, 0, [high[:, None, None] * np.ones((2 * page, 1, D))])
    if size == "blocks":
        size = np.array([1e4, 1e-4, 1.0, 1e-2] * (D // 64)).repeat(16)
    elif size in ("growing", "shrinking"):
        size = np.array([1e-2, 10.0] if size == "growing" else [10.0, 1e-2]).repeat(page)[:, None, None]
    # of one sign, so that the low weights' part of the sum does not cancel
    refill(p, 1, [(0.5 + rng.random((2 * page, 1, D))) * size * np.array([1.0, -1.0]).repeat(D // 2)])
    which = torch.tensor([0] * 4 + [1] * (pages - 4))
    table = p.batch.page_table[0].cpu()[which].repeat(seqs, 1).cuda()
    batch = J.CacheBatch(table, torch.full((seqs,), page * pages, dtype=torch.int32, device="cuda"),
                         torch.arange(seqs + 1, dtype=torch.int32, device="cuda"), 1)
    scale = float(np.float32(12 * np.log(2.0) / D))
    got = p.cache.attend(0, torch.ones(seqs, G, D, device="cuda").half(), batch, scale=scale)
    p.cache.check()
    times = np.where(np.arange(2 * page) < page, 4.0, pages - 4.0)            # how often each stored row is seen
    w = times * np.exp(np.where(high, 0.0, -scale * D))
    w /= w.sum()
    vals = p.values[1][0][:, 0]
    lo = vals.reshape(2 * page, D // 16, 16).min(-1).repeat(16, -1)
    lo = lo - 2.0 ** -10 * np.abs(lo)                    # at least the block's lower end (a code may not be 0)
    want = w @ vals
    # Scores and weights in fp32: 2^-18 covers 12 ln 2 of them.  The sums in fp32: a product adds 16 keys to them,
    # and each of the page pages / 16 = 4096 additions in a row is off by less than the last place of what has been
    # summed, 2^-23 of at most sum p |v|: 2^-11 of it together.  (It is needed: what is added later and is
    # small, as in "shrinking", loses its last bits the same way every time, as the products' sums are cut off.)
    sums = page * pages // 16 * 2.0 ** -23
    tol = w @ ((2 * VALUE + 2.0 ** -18 + sums) * np.abs(vals) + VALUE * (vals - lo) + LEAST)
    check(got, np.tile(want, (1, G, 1)), np.tile(tol, (1, G, 1)))
