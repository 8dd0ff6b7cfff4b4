"""Sizes that the binding's 32-bit fields cannot hold are refused, not cut off."""
import pytest
import torch

from cache_helpers import Paged, check_attend
from kv_cache_compression_group_b200 import jolt as J

pytestmark = pytest.mark.gpu


def test_sizes_beyond_32_bits_are_refused():
    p = Paged([40, 9], [2, 1], 1, 64, 16, (4, 4))
    q = torch.zeros(3, 2, 64, device="cuda").half()
    for window in (1 << 31, (1 << 32) + 5, 1 << 64):
        with pytest.raises(ValueError, match="window"):
            p.cache.attend(0, q, p.batch, window=window)
    many = torch.zeros(1, 1, 64, device="cuda").half().expand((1 << 32) + 3, 1, 64)
    with pytest.raises(ValueError, match="rows"):
        p.cache.write(0, many, many, p.batch)
    with pytest.raises(ValueError, match="rows"):
        p.cache.read(0, p.batch, many.shape[0], torch.float16, out=(many, many))
    with pytest.raises(ValueError, match="rows"):
        p.cache.attend(0, many, p.batch, out=many)
    for max_new in (1 << 31, (1 << 32) + 2):
        with pytest.raises(ValueError, match="max_new"):
            J.CacheBatch(p.batch.page_table, p.batch.lens, p.batch.starts, max_new)
    with pytest.raises(J.JoltError):                      # fits, but more than a call takes
        p.cache.write(0, many[:(1 << 30) + 1], many[:(1 << 30) + 1], p.batch)


def test_the_largest_window():
    p = Paged([40, 9], [2, 1], 1, 64, 16, (4, 4))
    for G in (2, 20, 40):
        check_attend(p, torch.float16, G, window=(1 << 31) - 1)
