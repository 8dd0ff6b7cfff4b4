"""How the attention over the paged cache is split and joined: nothing lost, nothing twice, the same in every
run; and the forms that the kernels of more rows are compiled in."""
import numpy as np
import pytest
import torch

from cache_helpers import Paged, check_attend, refill, tree
from kv_cache_compression_group_b200 import jolt as J

pytestmark = pytest.mark.gpu

U = 2.0 ** -11
GROUP = 16            # tokens of a stage of the narrow kernels


# ---- every group of 16 keys counts once ----------------------------------------------------
# (new rows, query heads per KV head): a row and two n-tiles of the codes' kernel, two and four of the next, jobs of
# 128 rows (one and several) and of 256
SHAPES = [(1, 1), (1, 4), (4, 4), (3, 4), (6, 4), (40, 1), (12, 8), (100, 3)]


@pytest.mark.parametrize("n,G", SHAPES)
@pytest.mark.parametrize("bits,lens", [((4, 8), [20000, 1, 777, 5000, 64]), ((2, 2), [20000, 1, 777, 5000, 64]),
                                       ((8, 4), [33333]), ((4, 8), [33333])])
@pytest.mark.parametrize("D,page", [(64, 64), (128, 32)])
def test_every_group_of_keys_counts_once(n, G, bits, D, page, lens):
    """Keys with one value each for 16 tokens, so that scores are known exactly, between -1 and 1; values that are
    1 in one feature, another one for every 16 tokens, and 0 elsewhere.  A feature's output is then a sum over a
    few dozen groups at most, of one sign, known to about 5 u of itself, while any group is
    more than twice that.

    Off by: the weight's rounding u, the value's (or the weight's times the step) u, v - lo <= v: 3 u, another u
    for scores and sums in fp32 (scores within 2^-18; at most 2^11 additions in a row, 2^-23 each)."""
    H = 2
    lens = [x + n for x in lens]
    p = Paged(lens, [n] * len(lens), H, D, page, bits, spread=0.0)
    rng = np.random.default_rng(n)
    rel, level, ks, vs = 4 * U, [], [], []
    for length in lens:
        groups = -(-length // GROUP)
        c = rng.integers(-64, 65, (groups, H)) / 64.0
        level.append(np.repeat(c, GROUP, 0)[:length])
        ks.append(np.repeat(level[-1][:, :, None], D, -1))
        which = np.repeat((np.arange(groups) * 7 + 3) % D, GROUP)[:length]     # 7: neighbours in other blocks
        v = np.zeros((length, H, D))
        v[np.arange(length), :, which] = 1.0
        vs.append(v)
    refill(p, 0, ks)
    refill(p, 1, vs)
    q = torch.ones(p.rows, H * G, D, device="cuda").half()
    got = p.cache.attend(0, q, p.batch, scale=1.0 / D).double().cpu().numpy()
    p.cache.check()
    for b, length in enumerate(lens):
        w = np.exp(level[b])                                            # [len, H]
        val = p.values[1][b]
        parts = np.cumsum(w[:, :, None] * val, 0)                       # sums over the keys up to each
        sums = np.cumsum(w, 0)
        for i in {0, n // 2, n - 1}:
            end = length - n + i
            want = parts[end] / sums[end][:, None]                      # [H, D]
            mine = got[p.starts[b] + i].reshape(H, G, D)
            tol = rel * want + np.maximum(U * want * (1 + rel), 2.0 ** -25)
            assert (np.abs(mine - want[:, None]) <= tol[:, None]).all(), (b, i)
            # what the bound is worth: an output without any one of the groups would be outside, and zeros are
            first = np.arange(0, end + 1, GROUP)
            part = np.add.reduceat((w[:, :, None] * val)[:end + 1], first, 0) / sums[end][:, None]
            whole = np.add.reduceat(np.ones(end + 1), first) == GROUP
            assert (part.max(-1)[whole] > 2 * np.take_along_axis(
                np.broadcast_to(tol, part.shape), part.argmax(-1)[..., None], -1)[..., 0][whole]).all()


# ---- the same in every run; what the other sequences of a batch may change -----------------
@pytest.mark.parametrize("n,G", SHAPES)
def test_every_run_of_a_call_gives_the_same_bits(n, G):
    p = Paged([9000 + n, 30 + n, 2500 + n], [n] * 3, 2, 128, 64, (4, 4))
    q = torch.randn(p.rows, 2 * G, 128, device="cuda").half()
    first = p.cache.attend(0, q, p.batch)
    for _ in range(5):
        assert torch.equal(p.cache.attend(0, q, p.batch), first)


@pytest.mark.parametrize("n,G", SHAPES)
def test_a_sequence_alone_and_among_others(n, G):
    """Alone, in another order and among other neighbours a sequence's work is split in other places.  The
    weights are then rounded to fp16 relative to another maximum: both results are off by at most 3 u sum p (|v| + v
    - lo) (and fp32 sums, within another u), the keys' rounding being the same."""
    lens, H, D = [9000 + n, 30 + n, 2500 + n, 700 + n], 2, 64
    p = Paged(lens, [n] * 4, H, D, 64, (4, 8))
    q = torch.randn(p.rows, H * G, D).half()
    rows = [q[p.starts[b]:p.starts[b + 1]] for b in range(4)]

    def attend(order):
        """Results of the sequences in this order, each on its own."""
        batch = J.CacheBatch(p.batch.page_table[order].contiguous(), p.batch.lens[order].contiguous(),
                             torch.arange(0, n * len(order) + 1, n, dtype=torch.int32, device="cuda"), n)
        out = p.cache.attend(0, torch.cat([rows[b] for b in order]).cuda(), batch).double().cpu()
        return dict(zip(order, out.split(n)))
    together = attend([0, 1, 2, 3])
    for order in ([0], [1], [2], [3], [3, 1, 0], [2, 3]):
        for b, got in attend(order).items():
            want, length = together[b], lens[b]
            v = torch.from_numpy(p.values[1][b])
            low = v.view(length, H, D // 16, 16).min(-1, keepdim=True).values
            mag = v.abs() + (v.view(length, H, D // 16, 16) - low + 2.0 ** -10 * low.abs()).reshape(v.shape)
            s = torch.einsum("nhgd,lhd->nhgl", rows[b].double().view(n, H, G, D), torch.from_numpy(p.values[0][b])) / D ** 0.5
            s.masked_fill_((torch.arange(length) > length - n + torch.arange(n)[:, None])[:, None, None], -float("inf"))
            tol = torch.einsum("nhgl,lhd->nhgd", s.softmax(-1), mag).reshape(want.shape) * 4 * U
            assert ((got - want).abs() <= 2 * (tol + U * (want.abs() + tol))).all(), (order, b)


# ---- the kernels of more rows: every pair of bit-widths, every option ----------------------
@pytest.mark.parametrize("rows", [7, 12, 24, 40, 160])
@pytest.mark.parametrize("bits", [(k, v) for k in (2, 4, 8) for v in (2, 4, 8)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_bit_widths_of_the_kernels_of_more_rows(rows, bits, D, page):
    p = Paged([1, 17, 130, 300], [1] * 4, 1, D, page, bits, seed=rows)
    check_attend(p, torch.float16, rows, seed=rows)
    p.cache.check()


@pytest.mark.parametrize("n,G", [(40, 8), (150, 2), (300, 1)])
@pytest.mark.parametrize("opts", [dict(softcap=5.0), dict(softcap=1e6), dict(scale=0.3), dict(window=1), dict(window=37),
                                  dict(window=200), dict(window=5000), dict(slopes=True),
                                  dict(softcap=20.0, window=100, slopes=True, scale=0.2), dict(prefix=True),
                                  dict(prefix=True, softcap=8.0, window=64)])
def test_options_of_jobs_of_256_rows(n, G, opts):
    lens = [n, n + 40, 290 + n]
    p = Paged(lens, [n, n - 7, n], 1, 64, 32, (4, 8), seed=n)
    opts, rng = dict(opts), np.random.default_rng(9)
    if opts.pop("slopes", None):
        opts["slopes"] = rng.standard_normal(G).astype(np.float32) * 0.2
    if opts.pop("prefix", None):
        lse = rng.standard_normal((p.rows, G)).astype(np.float32) * 3
        lse[0], lse[1:2] = -np.inf, 60.0
        opts["prefix"] = (rng.standard_normal((p.rows, G, 64)).astype(np.float32), lse)
    check_attend(p, torch.float16, G, **opts)
    p.cache.check()


@pytest.mark.parametrize("n,G", [(8, 4), (40, 4), (90, 3)])
@pytest.mark.parametrize("bits", [(2, 2), (2, 8), (8, 2)])
def test_trees_at_two_bits(n, G, bits):
    news = [n, n, max(1, n // 2)]
    lens = [n, 150 + n, 300]
    p = Paged(lens, news, 1, 128, 64, bits, seed=n)
    rng = np.random.default_rng(n)
    mask, depth = tree(rng, news, 5)
    positions = np.concatenate([np.full(m, length - m) for length, m in zip(lens, news)]) + depth
    slopes = 2.0 ** -np.arange(1, G + 1, dtype=np.float32)
    check_attend(p, torch.bfloat16, G, mask=mask, positions=positions, slopes=slopes, window=90)
    check_attend(p, torch.float16, G, mask=mask, softcap=10.0)
