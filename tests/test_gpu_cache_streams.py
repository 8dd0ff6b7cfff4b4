"""Calls of the paged cache that are given a stream: they run whole on it, allocations included."""
import pytest
import torch

from cache_helpers import Paged
from kv_cache_compression_group_b200 import jolt as J

pytestmark = pytest.mark.gpu


def forms(stream):
    """The forms that a stream argument may have."""
    return {"torch": stream, "handle": stream.cuda_stream,
            "object": type("Other", (), {"cuda_stream": stream.cuda_stream})()}


@pytest.mark.parametrize("form", ["torch", "handle", "object"])
def test_memory_of_a_call_is_its_streams(form, monkeypatch):
    """What attend and read allocate, and what check clears, belongs to the stream that they run on."""
    p = Paged([300, 20], [1, 1], 2, 64, 16, (4, 4))
    q = torch.randn(2, 8, 64, device="cuda").half()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = []

    def noting(f):
        def call(*args, **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return f(*args, **kw)
        return call
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    out = p.cache.attend(0, q, p.batch, stream=forms(stream)[form])
    k, v = p.cache.read(0, p.batch, 2, torch.float32, stream=forms(stream)[form])
    monkeypatch.undo()
    assert len(seen) == 4 and set(seen) == {stream.cuda_stream}      # a scratch and three results
    torch.cuda.synchronize()
    assert torch.equal(out, p.cache.attend(0, q, p.batch))
    assert torch.equal(k, p.cache.read(0, p.batch, 2, torch.float32)[0])
    owner = {s["address"]: s["stream"] for s in torch.cuda.memory_snapshot()}
    for t in (out, k, v):
        base = max(a for a in owner if a <= t.data_ptr())
        assert owner[base] == stream.cuda_stream
    p.cache.status.fill_(64)
    torch.cuda.synchronize()
    with pytest.raises(J.JoltError):
        p.cache.check(stream=forms(stream)[form])
    stream.synchronize()
    assert int(p.cache.status) == 0


@pytest.mark.parametrize("form", ["torch", "handle"])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_calls_on_the_current_and_on_a_given_stream_at_once(form, n):
    """One call queued on the current stream, the next on another without a wait between them."""
    p = Paged([5000 + n, 9000 + n, 300], [n] * 3, 2, 128, 64, (4, 4))
    q = [torch.randn(p.rows, 8, 128, device="cuda").half() for _ in range(2)]
    want = [p.cache.attend(0, x, p.batch) for x in q]
    rows = p.cache.read(0, p.batch, p.rows)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(30):
        a = [p.cache.attend(0, q[0], p.batch) for _ in range(3)]
        b = [p.cache.attend(0, q[1], p.batch, stream=forms(stream)[form]) for _ in range(3)]
        c = p.cache.read(0, p.batch, p.rows, stream=forms(stream)[form])
        a.append(p.cache.attend(0, q[0], p.batch))
        del a[0], b[0]                                   # freed while the others run
        a.append(p.cache.attend(0, q[0], p.batch))
        b.append(p.cache.attend(0, q[1], p.batch, stream=forms(stream)[form]))
        torch.cuda.synchronize()
        assert all(torch.equal(x, want[0]) for x in a) and all(torch.equal(x, want[1]) for x in b)
        assert all(torch.equal(x, y) for x, y in zip(c, rows))


def test_the_default_streams_handles():
    p = Paged([40], [1], 1, 64, 16, (4, 4))
    q = torch.randn(1, 2, 64, device="cuda").half()
    want = p.cache.attend(0, q, p.batch)
    for handle in (0, 1):
        assert torch.equal(p.cache.attend(0, q, p.batch, stream=handle), want)
    assert torch.equal(p.cache.attend(0, q, p.batch, stream=torch.cuda.default_stream()), want)
