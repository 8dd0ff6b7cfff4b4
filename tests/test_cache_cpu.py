"""Refusals of the paged cache's C ABI: every one is decided on the host, before any launch."""
import ctypes

import pytest

from kv_cache_compression_group_b200 import jolt as J

PTR = 1 << 20        # stands for device memory: no call here gets far enough to use it


def cache(**kw):
    c = dict(n_heads=2, head_dim=128, page_size=64, n_pages=10, bits_k=4, bits_v=4, k_codes=PTR, k_scales=PTR,
             v_codes=PTR, v_scales=PTR)
    return J.CCache(**{**c, **kw})


def batch(**kw):
    b = dict(n_seqs=1, max_pages=4, max_new=2, n_rows=2, page_table=PTR, lens=PTR, starts=PTR, status=PTR)
    return J.CCacheBatch(**{**b, **kw})


def options(**kw):
    return J.CAttendOptions(**kw)


def status(name, *args):
    return J.STATUS_NAMES[getattr(J.lib(), name)(*args)]


def write(c, b, k=PTR, v=PTR, dtype=J.JOLT_BF16):
    return status("jolt_cache_write", c, b, k, v, dtype, 256, 128, 256, 128, None)


def read(c, b, k=PTR, v=PTR, dtype=J.JOLT_BF16):
    return status("jolt_cache_read", c, b, dtype, k, v, 256, 128, 256, 128, None)


def scratch(c, b, nq):
    n = ctypes.c_size_t()
    return status("jolt_cache_attend_scratch_size", c, b, nq, ctypes.byref(n)), n.value


def attend(c, b, o, q=PTR, dtype=J.JOLT_BF16, nq=4, out=PTR, at=PTR, nbytes=1 << 40):
    return status("jolt_cache_attend", c, b, o, q, dtype, nq, 512, 128, out, 512, 128, at, nbytes, None)


BAD_CACHES = [(dict(head_dim=96), "UNSUPPORTED_SHAPE"), (dict(head_dim=256), "UNSUPPORTED_SHAPE"),
              (dict(page_size=8), "UNSUPPORTED_SHAPE"), (dict(page_size=48), "UNSUPPORTED_SHAPE"),
              (dict(page_size=8192), "UNSUPPORTED_SHAPE"), (dict(bits_k=3), "UNSUPPORTED_SHAPE"),
              (dict(bits_v=0), "UNSUPPORTED_SHAPE"), (dict(bits_v=16), "UNSUPPORTED_SHAPE"),
              (dict(n_pages=1 << 24), "UNSUPPORTED_SHAPE"),
              (dict(n_heads=0), "INVALID_ARG"), (dict(n_pages=0), "INVALID_ARG"), (dict(k_codes=0), "INVALID_ARG"),
              (dict(v_scales=0), "INVALID_ARG"), (dict(k_scales=PTR + 4), "INVALID_ARG"),
              (dict(v_codes=PTR + 8), "INVALID_ARG")]
BAD_BATCHES = [(dict(n_seqs=-1), "INVALID_ARG"), (dict(n_rows=-1), "INVALID_ARG"), (dict(max_new=-1), "INVALID_ARG"),
               (dict(max_pages=-1), "INVALID_ARG"), (dict(page_table=0), "INVALID_ARG"), (dict(lens=0), "INVALID_ARG"),
               (dict(starts=0), "INVALID_ARG"), (dict(status=0), "INVALID_ARG")]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_caches_refused(kw, want):
    assert write(cache(**kw), batch()) == want
    assert read(cache(**kw), batch()) == want
    assert scratch(cache(**kw), batch(), 4)[0] == want
    assert attend(cache(**kw), batch(), options()) == want


@pytest.mark.parametrize("kw,want", BAD_BATCHES)
def test_batches_refused(kw, want):
    assert write(cache(), batch(**kw)) == want
    assert read(cache(), batch(**kw)) == want
    assert attend(cache(), batch(**kw), options()) == want


def test_rows_refused():
    for call in (write, read):
        assert call(cache(), batch(), dtype=7) == "INVALID_ARG"
        assert call(cache(), batch(), k=None) == "INVALID_ARG"
        assert call(cache(), batch(), v=None) == "INVALID_ARG"


@pytest.mark.parametrize("kw", [dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                                dict(softcap=-2.0), dict(softcap=float("nan")), dict(softcap=1e-9), dict(softcap=1e35), dict(window=-1),
                                dict(mask=PTR, mask_words=0), dict(prefix_out=PTR), dict(prefix_lse=PTR)])
def test_options_refused(kw):
    assert attend(cache(), batch(), options(**kw)) == "INVALID_ARG"


def test_attend_refused():
    assert attend(cache(), batch(max_new=33), options(mask=PTR, mask_words=1)) == "INVALID_ARG"
    for kw in (dict(q=None), dict(out=None), dict(at=None), dict(at=PTR + 16), dict(nq=3), dict(nq=0), dict(nq=-2),
               dict(dtype=J.JOLT_F32), dict(dtype=9)):
        assert attend(cache(), batch(), options(), **kw) == "INVALID_ARG", kw
    assert attend(cache(), batch(), options(), nbytes=16) == "WORKSPACE_TOO_SMALL"
    assert status("jolt_cache_attend", cache(), batch(), None, PTR, 0, 4, 512, 128, PTR, 512, 128, PTR, 1 << 40,
                  None) == "INVALID_ARG"
    assert status("jolt_cache_write", None, batch(), PTR, PTR, 0, 256, 128, 256, 128, None) == "INVALID_ARG"
    assert status("jolt_cache_read", cache(), None, 0, PTR, PTR, 256, 128, 256, 128, None) == "INVALID_ARG"
    assert status("jolt_cache_check", None, None) == "INVALID_ARG"
    assert status("jolt_attend_state", PTR, PTR, 1, 0, PTR, 4, PTR, None, PTR, 1, None) == "INVALID_ARG"


def test_nothing_to_do_launches_nothing():
    for b in (batch(n_seqs=0, page_table=0, lens=0, starts=0, status=0), batch(n_rows=0)):
        assert write(cache(), b, k=None, v=None) == "OK"
        assert read(cache(), b, k=None, v=None) == "OK"
        assert attend(cache(), b, options(), q=None, out=None, at=None, nbytes=1 << 40) == "OK"
    assert attend(cache(), batch(max_new=0), options()) == "OK"


@pytest.mark.parametrize("heads,nq", [(2, 4), (8, 32), (40, 40), (1, 33)])
@pytest.mark.parametrize("new", [1, 4, 17, 4096])
def test_scratch_size(heads, nq, new):
    st, n = scratch(cache(n_heads=heads), batch(max_new=new, n_rows=new), nq)
    assert st == "OK" and 0 < n < 1 << 30


def test_more_rows_than_an_index_holds():
    assert scratch(cache(n_heads=1), batch(max_new=1 << 30, n_rows=1), 8)[0] == "UNSUPPORTED_SHAPE"


def test_fp16_is_not_a_type_of_the_compressor():
    o = J.Options((4, 8, 16, 32), (4, 8, 16), (0, 2))
    with pytest.raises(J.JoltError) as e:
        J.sizes(J.CShape(2, 2, 64, 16, 2, J.JOLT_F16), o)
    assert e.value.name == "INVALID_ARG"


def test_struct_layouts():
    assert ctypes.sizeof(J.CCache) == 56
    assert ctypes.sizeof(J.CCacheBatch) == 48
    assert ctypes.sizeof(J.CAttendOptions) == 56
