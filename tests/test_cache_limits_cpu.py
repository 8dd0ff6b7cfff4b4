"""The largest sizes of the paged cache's batches: what its kernels' 32-bit indices cannot hold is refused on
the host, before any launch."""
import pytest

from test_cache_cpu import PTR, attend, batch, cache, options, read, scratch, write


def refused(c, b):
    """What every call makes of a batch."""
    return {write(c, b), read(c, b), scratch(c, b, 4)[0], attend(c, b, options())}


@pytest.mark.parametrize("page,pages", [(16, (1 << 26) + 1), (4096, (1 << 18) + 1), (4096, (1 << 31) - 1)])
def test_more_tokens_than_a_sequence_may_have(page, pages):
    """A length near 2^31, rounded up to whole units, would be negative."""
    assert refused(cache(page_size=page), batch(max_pages=pages)) == {"UNSUPPORTED_SHAPE"}


@pytest.mark.parametrize("page,pages", [(16, 1 << 26), (4096, 1 << 18)])
def test_most_tokens_of_a_sequence(page, pages):
    assert scratch(cache(page_size=page), batch(max_pages=pages), 4)[0] == "OK"


@pytest.mark.parametrize("name", ["n_rows", "n_seqs"])
def test_more_rows_or_sequences_than_a_batch_may_have(name):
    """Rows may be that many without as much memory (a row stride of 0); the last block's first row would
    be negative."""
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        assert refused(cache(), batch(**{name: n})) == {"UNSUPPORTED_SHAPE"}
    assert scratch(cache(), batch(**{name: 1 << 30}), 4)[0] == "OK"
