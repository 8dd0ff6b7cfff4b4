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


def test_outputs_that_overlap_are_refused():
    """Rows or heads of an output in one place would be written by several threads at once."""
    p = Paged([40, 9], [2, 1], 2, 64, 16, (4, 4))
    q = torch.randn(3, 4, 64, device="cuda").half()
    want = p.cache.attend(0, q, p.batch)
    rows = p.cache.read(0, p.batch, 3, torch.float16)
    room = torch.full((1000,), 7.0, device="cuda").half()

    def view(heads, row, head):
        return room.as_strided((3, heads, 64), (row, head, 1))
    for row, head in ((0, 64), (256, 0), (64, 64), (255, 64), (256, 63), (32, 96), (64, 191), (1, 64)):
        with pytest.raises(ValueError, match="overlap"):
            p.cache.attend(0, q, p.batch, out=view(4, row, head))
    for row, head in ((0, 64), (128, 0), (64, 64), (127, 64), (64, 191)):
        for outs in ((view(2, row, head), torch.empty_like(rows[0])), (torch.empty_like(rows[0]), view(2, row, head))):
            with pytest.raises(ValueError, match="overlap"):
                p.cache.read(0, p.batch, 3, torch.float16, out=outs)
    with pytest.raises(ValueError, match="overlap"):
        p.cache.read(0, p.batch, 3, torch.float16, out=(view(2, 128, 64), view(2, 128, 64)))
    assert (room == 7.0).all()
    for row, head in ((256, 64), (64, 192), (300, 70), (65, 196)):
        assert torch.equal(p.cache.attend(0, q, p.batch, out=view(4, row, head)), want)
    one = torch.empty(1, 4, 64, device="cuda").half()             # a stride of nothing but one row does not count
    batch = J.CacheBatch(p.batch.page_table[:1].contiguous(), p.batch.lens[:1].contiguous(),
                         torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1)
    a = p.cache.attend(0, q[1:2], batch, out=one.as_strided((1, 4, 64), (0, 64, 1)))
    assert torch.equal(a, p.cache.attend(0, q[1:2], batch))
