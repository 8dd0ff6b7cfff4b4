"""The paged cache of block-quantised rows through its public entry points: rows written (codes and
scales bit for bit the oracle's), read back, and attended over, against float64."""
import numpy as np
import pytest
import torch

import oracle as O
from cache_helpers import HALF_STEP, Paged, magnitude, check_attend, plain_attend, quantised, tree
from kv_cache_compression_group_b200 import jolt as J
from kv_cache_compression_group_b200 import synth

pytestmark = pytest.mark.gpu


def raises(name, f):
    with pytest.raises(J.JoltError) as e:
        f()
    assert e.value.name == name, e.value


# ---- writing and reading ------------------------------------------------------------------
def _strided(x, how):
    """x [rows, H, D] with the same values in another layout."""
    rows, H, D = x.shape
    if how == "dense":
        return x.contiguous()
    if how == "fused":                                    # a slice of rows that hold more than x
        wide = torch.zeros(rows, 3, H, D, dtype=x.dtype, device=x.device)
        wide[:, 1] = x
        return wide[:, 1]
    if how == "odd":                                      # rows that start at odd elements
        flat = torch.zeros(rows * (H * D + 3) + 1, dtype=x.dtype, device=x.device)[1:]
        y = flat.as_strided((rows, H, D), (H * D + 3, D, 1))
        y.copy_(x)
        return y
    y = torch.empty(H, rows, D, dtype=x.dtype, device=x.device)   # the compressor's layout, heads first
    return y.copy_(x.transpose(0, 1)).transpose(0, 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("bits", [(2, 8), (4, 4), (8, 2)])
@pytest.mark.parametrize("how,D,page", [("dense", 128, 16), ("fused", 64, 64), ("odd", 128, 32), ("heads", 64, 256)])
def test_write_and_read_are_the_oracles(dtype, bits, how, D, page):
    lens, news, H = [33, 5, 0, 100, 1], [17, 5, 0, 0, 1], 3
    p = Paged(lens, news, H, D, page, bits, rows_behind=2)
    before = [t.clone() for t in p.pools]
    rng = np.random.default_rng(5)
    rows = [torch.from_numpy(rng.standard_normal((p.rows, H, D)) * np.exp(rng.standard_normal((p.rows, H, 1)) * 3)).to(dtype)
            for _ in range(2)]
    p.cache.write(0, _strided(rows[0].cuda(), how), _strided(rows[1].cuda(), how), p.batch)
    p.cache.check()
    want_pools = [t.cpu().numpy()[0] for t in before]
    want_vals = []
    for kv in range(2):
        packed, scales, val = quantised(rows[kv].double().numpy(), bits[kv])
        want_vals.append(val)
        for b, (length, n) in enumerate(zip(lens, news)):
            for i in range(n):
                t, r = length - n + i, p.starts[b] + i
                want_pools[2 * kv][p.table[b, t // page], :, t % page] = packed[r]
                want_pools[2 * kv + 1][p.table[b, t // page], :, t % page] = scales[r]
    for got, want in zip(p.pools, want_pools):
        assert np.array_equal(got[0].cpu().numpy(), want, equal_nan=want.dtype == np.float16)
    n = int(p.starts[-1])
    for dt in (torch.bfloat16, torch.float16, torch.float32):
        fill = torch.full((p.rows, H, D), 3.0, dtype=dt, device="cuda")
        outs = (_strided(fill, how), _strided(fill.clone(), how))
        got = p.cache.read(0, p.batch, p.rows, dt, out=outs)
        for kv in range(2):
            want = torch.from_numpy(want_vals[kv][:n]).float().to(dt)
            assert torch.equal(got[kv][:n].cpu(), want)
            assert (got[kv][n:] == 3.0).all()


def test_whole_sequences_read_back():
    lens = [70, 1, 129, 16]
    p = Paged(lens, lens, 2, 128, 64, (8, 4))
    k, v = p.cache.read(0, p.batch, sum(lens), torch.float32)
    for got, vals in ((k, p.values[0]), (v, p.values[1])):
        assert np.array_equal(got.cpu().numpy(), np.concatenate(vals).astype(np.float32))


@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_at_the_ends_of_the_range(bits, dtype):
    H, D = 1, 64
    rows = torch.zeros(12, H, D, dtype=torch.float64)
    rng = np.random.default_rng(3)
    rows[1] = 1.5                                             # one value: step 0
    rows[2] = -0.0
    rows[3] = torch.from_numpy(rng.standard_normal((H, D))) * 2.0 ** -20    # below fp16's normal range
    rows[4] = torch.from_numpy(rng.standard_normal((H, D))) * 2.0 ** -40    # below fp16
    rows[5, 0, ::2], rows[5, 0, 1::2] = -65504.0, 65504.0
    rows[6, 0, ::2], rows[6, 0, 1::2] = 65280.0, 65024.0
    rows[7] = torch.arange(D).double()                        # exact ties between codes
    rows[8] = torch.arange(D).double() / 2
    rows[9] = torch.from_numpy(rng.integers(0, 31, (H, D))).double() / 2    # ties for 15 levels
    rows[10, 0, 3] = 1e30
    rows[11] = torch.from_numpy(rng.standard_normal((H, D))) * 1e4
    rows[10] = rows[10].clamp(-65504.0, 65504.0)
    rows = rows.to(dtype).clamp(-65504.0, 65504.0) if dtype == torch.float32 else rows.to(dtype)
    if dtype == torch.bfloat16:                               # bf16 has no 65504
        rows[5] = rows[5].sign() * 65280.0
        rows[10] = rows[10].clamp(-65280.0, 65280.0)
    p = Paged([12], [12], H, D, 16, (bits, bits))
    p.cache.write(0, rows.cuda(), rows.cuda(), p.batch)
    p.cache.check()
    _, scales, want = quantised(rows.double().numpy(), bits)
    k, v = p.cache.read(0, p.batch, 12, torch.float32)
    assert np.array_equal(k.cpu().numpy(), want.astype(np.float32))
    assert torch.equal(k, v)


def test_write_of_nan_and_infinities():
    H, D = 2, 64
    x = torch.randn(4, H, D)
    bad = x.clone()
    bad[1, 0, 5], bad[2, 1, 7], bad[2, 1, 40], bad[3, 0, 0] = float("nan"), float("inf"), -float("inf"), 1e9
    good = bad.nan_to_num(nan=0.0).clamp(-65504.0, 65504.0)
    p = Paged([4], [4], H, D, 16, (4, 8))
    p.cache.write(0, bad.cuda(), bad.cuda(), p.batch)
    raises("NUMERIC", p.cache.check)
    p.cache.check()                                            # told once
    got = p.cache.read(0, p.batch, 4, torch.float32)
    for kv, bits in ((0, 4), (1, 8)):
        assert np.array_equal(got[kv].cpu().numpy(), quantised(good.double().numpy(), bits)[2].astype(np.float32))


def test_pool_beyond_32_bit_offsets():
    """The last pages of a pool whose codes take more than 2^32 bytes."""
    H, D, page, pages = 8, 128, 256, 17000
    cache = J.QuantCache(1, H, D, pages, page, (8, 8))
    assert cache.k_codes.numel() > 2 ** 32
    rng = np.random.default_rng(0)
    p = Paged([300], [300], H, D, page, (8, 8), spare=0)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    batch = J.CacheBatch(table, p.batch.lens, p.batch.starts, 300)
    k, v = (p.new_rows(torch.bfloat16, kv).cuda() for kv in range(2))
    cache.write(0, k, v, batch)
    got = cache.read(0, batch, 300, torch.float32)
    for kv in range(2):
        assert np.array_equal(got[kv].cpu().numpy(), p.values[kv][0].astype(np.float32))
    q = torch.from_numpy(rng.standard_normal((1, 16, D))).bfloat16().cuda()
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    a = cache.attend(0, q, J.CacheBatch(table, p.batch.lens, one, 1))
    b = p.cache.attend(0, q, J.CacheBatch(p.batch.page_table, p.batch.lens, one, 1))
    assert torch.equal(a, b)
    cache.check()


# ---- attention ----------------------------------------------------------------------------
@pytest.mark.parametrize("bits", [(2, 2), (4, 4), (8, 8), (8, 4), (4, 2), (2, 8)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attend_single_tokens(bits, D, page, dtype):
    p = Paged([1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 300], [1] * 13, 2, D, page, bits)
    check_attend(p, dtype, 8)
    p.cache.check()


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 33])
def test_attend_query_groups(G):
    p = Paged([1, 40, 131], [1] * 3, 2, 128, 16, (4, 4))
    check_attend(p, torch.float16, 2 * G)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32, 33, 40, 64, 65, 100])
@pytest.mark.parametrize("G", [1, 4])
def test_attend_chunks(n, G):
    """Causal rows, over committed keys of several lengths and none."""
    lens, news = [n, n + 1, n + 63, n + 130, 200], [n, n, n, n - 1, min(3, n)]
    p = Paged(lens, news, 2, 64, 32, (8, 4), seed=n)
    check_attend(p, torch.float16, 2 * G, seed=n)
    p.cache.check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [4, 9, 32, 40, 70])
def test_attend_trees(n, D):
    lens, news = [n, n + 5, 150 + n, 300], [n, n, n, max(1, n // 2)]
    p = Paged(lens, news, 2, D, 64, (4, 8), seed=n)
    rng = np.random.default_rng(n)
    mask, depth = tree(rng, news, 5)
    positions = np.concatenate([np.full(m, length - m) for length, m in zip(lens, news)]) + depth
    slopes = 2.0 ** -np.arange(1, 9, dtype=np.float32)
    check_attend(p, torch.bfloat16, 8, mask=mask, positions=positions, slopes=slopes)
    check_attend(p, torch.float16, 4, mask=mask, positions=positions, window=20)
    check_attend(p, torch.float16, 4, mask=mask)
    p.cache.check()


@pytest.mark.parametrize("n,G", [(1, 4), (2, 8), (3, 8), (12, 8)])
@pytest.mark.parametrize("opts", [dict(softcap=5.0), dict(softcap=1e6), dict(softcap=0.01), dict(scale=0.3), dict(window=1), dict(window=37), dict(window=5000),
                                  dict(slopes=True), dict(softcap=20.0, window=100, slopes=True, scale=0.2),
                                  dict(prefix=True), dict(prefix=True, softcap=8.0, window=64)])
def test_attend_options(n, G, opts):
    lens = [n, n + 40, 290, 128 + n]
    p = Paged(lens, [n] * 4, 2, 128, 32, (4, 4), seed=n)
    opts = dict(opts)
    nq, rng = 2 * G, np.random.default_rng(9)
    if opts.pop("slopes", None):
        opts["slopes"] = rng.standard_normal(nq).astype(np.float32) * 0.2      # either sign
    if opts.pop("prefix", None):
        lse = rng.standard_normal((p.rows, nq)).astype(np.float32) * 3
        lse[0] = -np.inf                                                       # a prefix that saw nothing
        lse[1:2] = 60.0                                                        # one that outweighs all
        opts["prefix"] = (rng.standard_normal((p.rows, nq, 128)).astype(np.float32), lse)
    check_attend(p, torch.float16, nq, **opts)


@pytest.mark.parametrize("G", [2, 16])
def test_attend_rows_that_see_nothing(G):
    """Trees whose nodes have no bits set, with and without committed keys, and a prefix."""
    lens, news = [4, 40, 4], [4, 4, 4]
    p = Paged(lens, news, 1, 64, 16, (4, 4), rows_behind=3)
    mask = np.zeros((p.rows, 1), np.uint32)
    mask[1], mask[6] = 0b0011, 0b0101
    got = check_attend(p, torch.float16, G, mask=mask)
    assert (got[0] == 0).all() and (got[2:4] == 0).all()
    rng = np.random.default_rng(0)
    prefix = (rng.standard_normal((p.rows, G, 64)).astype(np.float32), np.full((p.rows, G), -np.inf, np.float32))
    prefix[1][2:] = -400.0                        # far below any score, but all that rows 2 and 3 have
    got = check_attend(p, torch.float16, G, mask=mask, prefix=prefix)
    assert (got[0] == 0).all()
    assert torch.equal(got[2].cpu(), torch.from_numpy(prefix[0][2]).half())
    check_attend(p, torch.float16, G, mask=mask, window=1)


def test_attend_large_and_small_queries():
    """Queries at the ends of bf16's range, where fp16 has no such numbers."""
    p = Paged([70, 9], [1, 1], 1, 64, 16, (8, 8))
    for q_scale, scale in ((1e-30, 1e30), (1e20, 1e-20), (3e4, 1e-4), (1.0, 1.0)):
        check_attend(p, torch.bfloat16, 4, q_scale=q_scale, scale=scale)


def test_attend_large_values():
    """Stored values at the ends of fp16's range."""
    p = Paged([40], [40], 1, 64, 16, (8, 8))
    x = (torch.rand(40, 1, 64) * 2 - 1) * 65504.0
    p.cache.write(0, x.cuda(), x.cuda(), p.batch)
    val = quantised(x.double().numpy(), 8)[2]
    p.values = [[val], [val]]
    check_attend(p, torch.bfloat16, 2, scale=1e-5)


def test_attend_nan_queries_stay_in_their_rows():
    p = Paged([50, 60], [3, 2], 1, 128, 16, (4, 4))
    q = torch.randn(5, 4, 128).half().cuda()
    want = p.cache.attend(0, q, p.batch)
    q[1, 2, 7], q[3, 0, 0] = float("nan"), float("inf")
    got = p.cache.attend(0, q, p.batch)
    hit = torch.zeros(5, 4, dtype=torch.bool)
    hit[1, 2] = hit[3, 0] = True
    assert torch.equal(got[~hit], want[~hit])
    assert got[1, 2].isnan().all()


def test_attend_long_and_ragged():
    """Work split over many thread blocks, joined: long next to short sequences, 64-bit check on the device."""
    lens, H, D, G = [20000, 1, 777, 5000, 64], 2, 128, 4
    for n in (1, 4, 24):
        p = Paged([x + n for x in lens], [n] * 5, H, D, 64, (4, 8), seed=n)
        q = torch.randn(p.rows, H * G, D, dtype=torch.float64).to(torch.float16)
        got = p.cache.attend(0, q.cuda(), p.batch).double().cpu()
        for b in range(5):
            k, v = (torch.from_numpy(p.values[kv][b]).cuda() for kv in range(2))
            x = q[p.starts[b]:p.starts[b + 1]].double().cuda()
            s = torch.einsum("nhgd,lhd->nhgl", x.view(n, H, G, D), k) / D ** 0.5
            i, t = torch.arange(n, device="cuda"), torch.arange(lens[b] + n, device="cuda")
            s.masked_fill_((t[None] > lens[b] + i[:, None])[:, None, None], -float("inf"))
            want = torch.einsum("nhgl,lhd->nhgd", s.softmax(-1), v).reshape(n, H * G, D).cpu()
            mag = torch.einsum("nhgl,lhd->nhgd", s.softmax(-1), magnitude(v)).reshape(n, H * G, D).cpu()
            d = float(2.0 ** -11 * torch.einsum("nhgd,lhd->nhgl", x.view(n, H, G, D).abs(), k.abs()).max() / D ** 0.5)
            tol = mag * (2 * np.expm1(2 * d) + 2.0 ** -10 + 2.0 ** -17) + 2.0 ** -11 * want.abs() + 1e-6
            assert ((got[p.starts[b]:p.starts[b + 1]] - want).abs() <= tol).all()


@pytest.mark.parametrize("n,G,heads", [(16, 4, 1), (40, 1, 2), (33, 4, 1), (70, 8, 1)])
@pytest.mark.parametrize("lens", [[70000], [9000, 40000, 130, 33000]])
def test_attend_many_tiles_in_one_block(n, G, heads, lens):
    """Rows by the dozen over enough keys that every thread block has many tiles of a job, and parts
    of several jobs; the keys repeat, so the answer is that of one repetition."""
    D, page, rep = 64, 64, 128
    p = Paged([rep], [1], heads, D, page, (4, 4))
    reps = [x // rep for x in lens]
    table = torch.zeros(len(lens), max(reps) * 2 + 2, dtype=torch.int32, device="cuda")
    for b, r in enumerate(reps):
        table[b, :2 * r] = p.batch.page_table[0].repeat(r)[:2 * r]
    starts = torch.arange(0, n * len(lens) + 1, n, dtype=torch.int32, device="cuda")
    batch = J.CacheBatch(table, torch.tensor([r * rep for r in reps], dtype=torch.int32, device="cuda"), starts, n)
    mask = torch.full((n * len(lens), -(-n // 32)), -1, dtype=torch.int32, device="cuda")    # all new rows seen
    q = torch.randn(n * len(lens), heads * G, D).half()
    got = p.cache.attend(0, q.cuda(), batch, mask=mask)
    p.cache.check()
    k, v = (torch.from_numpy(p.values[kv][0]) for kv in range(2))
    s = torch.einsum("nhgd,lhd->nhgl", q.double().view(-1, heads, G, D), k) / D ** 0.5
    w = s.softmax(-1)
    want = torch.einsum("nhgl,lhd->nhgd", w, v).reshape(q.shape)
    mag = torch.einsum("nhgl,lhd->nhgd", w, magnitude(v)).reshape(q.shape)
    d = float(2.0 ** -11 * torch.einsum("nhgd,lhd->nhgl", q.double().view(-1, heads, G, D).abs(), k.abs()).max() / D ** 0.5)
    tol = mag * (2 * np.expm1(2 * d) + 2.0 ** -10 + 2.0 ** -17) + 2.0 ** -11 * want.abs() + 1e-6
    assert ((got.double().cpu() - want).abs() <= tol).all()


def test_strided_queries_and_outputs():
    p = Paged([30, 50], [2, 2], 2, 64, 16, (4, 4))
    x = torch.randn(4, 8, 64, device="cuda").bfloat16()
    want = p.cache.attend(0, x, p.batch)
    for how in ("fused", "odd", "heads"):
        out = _strided(torch.zeros_like(x), how)
        got = p.cache.attend(0, _strided(x, how), p.batch, out=out)
        assert got is out and torch.equal(got, want), how


@pytest.mark.parametrize("n,G", [(1, 4), (3, 8), (9, 8)])
def test_many_sequences(n, G):
    """More sequences than threads that look for them, empty ones and ones without new rows among them."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 40, 700).tolist()
    news = [min(x, int(rng.integers(0, n + 1))) for x in lens]
    lens[311], news[311] = 900, n
    p = Paged(lens, news, 1, 64, 16, (4, 4), seed=n, max_new=n)
    check_attend(p, torch.float16, G)
    before = [t.clone() for t in p.pools]
    rows = [p.new_rows(torch.float32, kv).cuda() for kv in range(2)]
    k, v = p.cache.read(0, p.batch, p.rows, torch.float32)
    p.cache.write(0, *rows, p.batch)
    for t, was in zip(p.pools, before):
        assert torch.equal(t.view(torch.uint8), was.view(torch.uint8))
    for got, vals in ((k, p.values[0]), (v, p.values[1])):
        want = np.concatenate([x[len(x) - m:] for x, m in zip(vals, news)])
        assert np.array_equal(got.cpu().numpy(), want.astype(np.float32))
    p.cache.check()


def test_output_in_place_of_the_queries():
    p = Paged([5000, 40, 700], [2, 2, 2], 2, 128, 64, (4, 4))
    q = torch.randn(6, 8, 128, device="cuda").half()
    want = p.cache.attend(0, q, p.batch)
    assert torch.equal(p.cache.attend(0, q, p.batch, out=q), want)


def test_batch_grows_within_its_bounds():
    """One batch object whose tensors change between calls: fewer rows than max_new, and more sequences' pages."""
    p = Paged([100, 60], [8, 1], 2, 64, 16, (8, 8), max_new=40)
    check_attend(p, torch.bfloat16, 8)                       # max_new * 4 rows choose the wide kernel
    q = torch.randn(p.rows, 8, 64, device="cuda").bfloat16()
    wide = p.cache.attend(0, q, p.batch)
    p.batch = J.CacheBatch(p.batch.page_table, p.batch.lens, p.batch.starts, 8)
    check_attend(p, torch.bfloat16, 8)
    assert (wide.float() - p.cache.attend(0, q, p.batch).float()).abs().max() < 0.05


# ---- how calls stand next to one another --------------------------------------------------
def test_batches_that_name_what_is_not_there():
    lens, news = [40, 50, 60, 30], [2, 3, 1, 2]
    p = Paged(lens, news, 2, 64, 16, (4, 4))
    table = p.batch.page_table.clone()
    p.batch.page_table[1, 1] = p.n_pages                   # one page of sequence 1 is not there
    p.batch.page_table[3, 0] = -1
    check_attend(p, torch.float16, 4, lost=((1, 1), (3, 0)))
    raises("INVALID_ARG", p.cache.check)
    k, _ = p.cache.read(0, J.CacheBatch(p.batch.page_table, p.batch.lens, torch.tensor(
        np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda"), 60), sum(lens), torch.float32)
    want = np.concatenate(p.values[0]).astype(np.float32)
    want[40 + 16:40 + 32] = 0
    want[150:150 + 16] = 0
    assert np.array_equal(k.cpu().numpy(), want)
    raises("INVALID_ARG", p.cache.check)
    p.batch.page_table.copy_(table)
    p.cache.check()
    for change in ("short", "long", "negative", "rows"):
        p = Paged(lens, news, 2, 64, 16, (4, 4))
        before = [t.clone() for t in p.pools]
        if change == "short":
            p.batch.lens[1] = 2                             # fewer than its new rows
        elif change == "long":
            p.batch.lens[1] = 16 * p.table.shape[1] + 1
        elif change == "negative":
            p.batch.lens[1] = -5
        else:
            p.batch = J.CacheBatch(p.batch.page_table, p.batch.lens, p.batch.starts, 2)   # max_new below sequence 1's rows
        check_attend(p, torch.float16, 4, skip=(1,))
        raises("INVALID_ARG", p.cache.check)
        x = torch.randn(p.rows, 2, 64, device="cuda")
        p.cache.write(0, x, x, p.batch)
        raises("INVALID_ARG", p.cache.check)
        for t, was in zip(p.pools, before):                 # sequence 1's pages are as they were
            mine = torch.from_numpy(p.table[1][p.table[1] >= 0]).long().cuda()
            assert torch.equal(t[0, mine].view(torch.uint8), was[0, mine].view(torch.uint8))
    p = Paged(lens, news, 2, 64, 16, (4, 4))
    q = torch.randn(p.rows, 4, 64, device="cuda").half()
    want = p.cache.attend(0, q, p.batch)
    p.batch.starts[2] = 100                                 # beyond the rows, and no longer ascending
    out = torch.full_like(q, 7.0)
    p.cache.attend(0, q, p.batch, out=out)
    assert torch.equal(out[:2], want[:2])
    assert (out[2:6] == 7.0).all()
    assert torch.equal(out[6:], want[6:]) or (out[6:] == 7.0).all()
    raises("INVALID_ARG", p.cache.check)


def test_nothing_to_do():
    p = Paged([20, 30], [0, 0], 1, 64, 16, (4, 4))
    assert p.cache.attend(0, torch.zeros(0, 2, 64, device="cuda").half(), p.batch).shape == (0, 2, 64)
    p.cache.write(0, torch.zeros(0, 1, 64, device="cuda"), torch.zeros(0, 1, 64, device="cuda"), p.batch)
    q = torch.ones(3, 2, 64, device="cuda").half()
    out = torch.full_like(q, 5.0)
    p.cache.attend(0, q, J.CacheBatch(p.batch.page_table, p.batch.lens, p.batch.starts, 4), out=out)
    assert (out == 5.0).all()
    none = J.CacheBatch(torch.zeros(0, 0, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int32, device="cuda"), 1)
    p.cache.attend(0, q, none, out=out)
    assert (out == 5.0).all()
    p.cache.check()


def test_results_repeat_and_do_not_depend_on_the_batch():
    lens, news = [9000, 30, 2500], [1, 1, 1]
    p = Paged(lens, news, 2, 128, 64, (4, 4))
    q = torch.randn(3, 8, 128, device="cuda").half()
    first = p.cache.attend(0, q, p.batch)
    for _ in range(3):
        assert torch.equal(p.cache.attend(0, q, p.batch), first)


@pytest.mark.parametrize("n", [1, 2, 6, 40])
def test_captured_step_replays_on_new_contents(n):
    """Written and attended in a captured graph, replayed after lengths and rows changed in place; two
    such graphs at once on two streams."""
    lens = [190, 110]
    p = Paged(lens, [n, n], 2, 128, 32, (4, 8))
    q = torch.zeros(2 * n, 8, 128, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.zeros(2 * n, 2, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    saved = [t.clone() for t in p.pools]
    p.cache.write(0, k, v, p.batch)
    p.cache.attend(0, q, p.batch)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.cache.write(0, k, v, p.batch)
            out = p.cache.attend(0, q, p.batch)
        graphs.append((g, out))
    for t, s in zip(p.pools, saved):
        t.copy_(s)
    qs = torch.randn(2 * n, 8, 128).bfloat16()
    for shorter in (0, 40):
        p.lens = [x - shorter for x in lens]
        p.batch.lens.copy_(torch.tensor(p.lens, dtype=torch.int32))
        for kv in range(2):
            p.values[kv] = [x[:m] for x, m in zip(p.values[kv], p.lens)]
            p.dense[kv] = [x[:m] for x, m in zip(p.dense[kv], p.lens)]
        q.copy_(qs)
        k.copy_(p.new_rows(torch.bfloat16, 0))
        v.copy_(p.new_rows(torch.bfloat16, 1))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        want, tol = plain_attend(p, qs.double().numpy())
        for _, out in graphs:
            off = np.abs(out.double().cpu().numpy() - want)
            assert (off <= tol + HALF_STEP[torch.bfloat16] * (np.abs(want) + tol) + 1e-7).all()
    p.cache.check()


def test_calls_on_other_streams_at_once():
    p = Paged([5000, 300], [1, 1], 2, 128, 64, (4, 4))
    q = [torch.randn(2, 8, 128, device="cuda").half() for _ in range(4)]
    want = [p.cache.attend(0, x, p.batch) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(5):
        got = []
        for x, st in zip(q, streams):
            with torch.cuda.stream(st):
                got.append(p.cache.attend(0, x, p.batch))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        got = [p.cache.attend(0, x, p.batch, stream=st) for x, st in zip(q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_layers_are_apart():
    p = Paged([40], [1], 2, 64, 16, (4, 4))
    many = J.QuantCache(3, 2, 64, p.n_pages, 16, (4, 4))
    for t, one in zip((many.k_codes, many.k_scales, many.v_codes, many.v_scales), p.pools):
        t[1].copy_(one[0])
    q = torch.randn(1, 4, 64, device="cuda").half()
    assert torch.equal(many.attend(1, q, p.batch), p.cache.attend(0, q, p.batch))
    x = torch.randn(1, 2, 64, device="cuda")
    before = many.k_codes.clone()
    many.write(2, x, x, p.batch)
    assert torch.equal(many.k_codes[:2], before[:2]) and not torch.equal(many.k_codes[2], before[2])


# ---- a compressed prompt with generated rows behind it -------------------------------------
@pytest.mark.parametrize("n", [1, 3])
def test_generation_behind_a_compressed_prompt(n):
    """The prompt in JoLT's factors, the generated rows in pages: attention over both is attention
    over the decompressed prompt and the stored rows."""
    w = synth.small_workload("mistral7b", n_layers=4, n_heads=2, T=256)
    K, V = synth.make_cache(w, 0)
    opts = J.Options((32, 64), (64, 128), (0, 2, 4), "randomized")
    comp = J.Compressor(w.n_layers, w.n_heads, w.T, w.D, w.layers_per_group, K.dtype, opts)
    blob = comp.compress(K.cuda(), V.cuda(), w.bf16_bytes() // 2, 0)
    Kh, Vh = comp.decompress(blob, torch.float32)
    att = J.Attention(comp, blob, 8)
    lens = [37]
    p = Paged(lens, [n], 2, 128, 16, (8, 4))
    for layer in (0, 3):
        q = (torch.randn(n, 8, 128) * 0.3).bfloat16().cuda()
        states = [att.attend_state(layer, x) for x in q]
        for x, (o, lse) in zip(q, states):
            assert torch.equal(o, att.attend(layer, x))
        prefix = (torch.stack([o for o, _ in states]), torch.stack([s for _, s in states]))
        got = p.cache.attend(0, q, p.batch, prefix=prefix).double().cpu()
        for i in range(n):
            end = lens[0] - n + i + 1
            for h in range(8):
                k = torch.cat((Kh[layer, h // 4].double().cpu(), torch.from_numpy(p.values[0][0][:end, h // 4])))
                v = torch.cat((Vh[layer, h // 4].double().cpu(), torch.from_numpy(p.values[1][0][:end, h // 4])))
                x = q[i, h].double().cpu()
                s = (k @ x) / 128 ** 0.5
                wgt = s.softmax(0)
                want, mag = wgt @ v, wgt @ magnitude(v)
                d = float((k.abs() @ x.abs()).max()) / 128 ** 0.5 * 2.0 ** -11
                tol = mag * (2 * np.expm1(2 * d) + 2.0 ** -10 + 2e-5) + 2.0 ** -8 * (want.abs() + mag * 0.01) + 1e-6
                assert ((got[i, h] - want).abs() <= tol).all()
            assert abs(float(states[i][1][0]) - float(torch.logsumexp(
                (Kh[layer, 0].double().cpu() @ q[i, 0].double().cpu()) / 128 ** 0.5, 0))) < 1e-4
