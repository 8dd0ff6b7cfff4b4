"""First calls of the paged cache in a process that are captured into a graph, and the largest pages."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from cache_helpers import Paged, check_attend

pytestmark = pytest.mark.gpu

FIRST = """
import torch
from kv_cache_compression_group_b200 import jolt as J
n, G = {n}, {G}
torch.manual_seed(0)
cache = J.QuantCache(1, 2, 64, 16, 16, (4, 8))
i32 = dict(dtype=torch.int32, device="cuda")
batch = J.CacheBatch(torch.arange(16, **i32)[None], torch.tensor([150], **i32), torch.tensor([0, n], **i32), n)
whole = J.CacheBatch(batch.page_table, batch.lens, torch.tensor([0, 150], **i32), 150)
q, k, v = (torch.randn(n, h, 64, device="cuda").half() for h in (2 * G, 2, 2))
old = [torch.randn(150, 2, 64, device="cuda").half() for _ in range(2)]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    cache.write(0, *old, whole)
    cache.write(0, k, v, batch)
    out = cache.attend(0, q, batch)
    rows = cache.read(0, batch, n)
g.replay()
torch.cuda.synchronize()
cache.check()
first = [t.clone() for t in (out, *rows)]
again = (cache.attend(0, q, batch), *cache.read(0, batch, n))
assert out.abs().sum() > 0 and all(torch.equal(a, b) for a, b in zip(first, again))
print("captured")
"""


@pytest.mark.parametrize("n,G", [(1, 4), (3, 8), (20, 2), (100, 4)])
def test_the_first_calls_of_a_process_may_be_captured(n, G):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST.format(n=n, G=G)], cwd=root, capture_output=True, text=True,
                          timeout=300)
    assert done.returncode == 0 and "captured" in done.stdout, done.stderr[-2000:]


@pytest.mark.parametrize("page", [512, 4096])
def test_the_largest_pages(page):
    lens = [page, page + 1, page - 1, 2 * page + 100]
    p = Paged(lens, [1] * 4, 1, 64, page, (4, 8))
    for rows in (2, 24, 40, 160):
        check_attend(p, torch.float16, rows, window=300)
        check_attend(p, torch.float16, rows, slopes=np.full(rows, 0.05, np.float32))
    k, v = p.cache.read(0, p.batch, 4, torch.float32)
    for got, vals in ((k, p.values[0]), (v, p.values[1])):
        assert np.array_equal(got.cpu().numpy(), np.stack([x[-1] for x in vals]).astype(np.float32))
    p.cache.check()
