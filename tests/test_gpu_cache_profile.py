"""Stage timing of the paged cache's calls, captured ones among them."""
import pytest
import torch

from cache_helpers import Paged
from kv_cache_compression_group_b200 import jolt as J

pytestmark = pytest.mark.gpu


def test_captured_calls_are_not_timed():
    """Events that are captured into a graph cannot be read: calls on a capturing stream leave none."""
    p = Paged([300, 20], [1, 1], 2, 64, 16, (4, 4))
    q = torch.randn(2, 8, 64, device="cuda").half()
    k = torch.randn(2, 2, 64, device="cuda").half()
    p.cache.write(0, k, k, p.batch)
    want = p.cache.attend(0, q, p.batch)
    J.profile_begin()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.cache.write(0, k, k, p.batch)
        got = p.cache.attend(0, q, p.batch)
    g.replay()
    p.cache.attend(0, q, p.batch)
    p.cache.read(0, p.batch, 2)
    told = J.profile_end()
    assert {name: (n, rows) for name, (_, n, rows) in told.items()} == {"cache_attend": (1, 2), "cache_read": (1, 2)}
    assert torch.equal(got, want)
    J.profile_begin()
    assert J.profile_end() == {}
