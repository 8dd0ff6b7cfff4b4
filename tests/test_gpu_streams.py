"""Calls of the compressor's binding that are given a stream: they run whole on it, allocations included."""
import pytest
import torch

from kv_cache_compression_group_b200 import jolt as J
from kv_cache_compression_group_b200 import synth

pytestmark = pytest.mark.gpu


def test_every_call_runs_whole_on_its_stream(monkeypatch):
    w = synth.small_workload("mistral7b", n_layers=4, n_heads=2, T=256)
    K, V = (x.cuda() for x in synth.make_cache(w, 0))
    opts = J.Options((32, 64), (64, 128), (0, 2, 4), "randomized")
    comp = J.Compressor(w.n_layers, w.n_heads, w.T, w.D, w.layers_per_group, K.dtype, opts)
    budget = w.bf16_bytes() // 2
    q = torch.randn(8, 128, device="cuda", dtype=torch.float64)      # converted by the call
    dist = torch.rand(4, 3, device="cuda")
    nbytes = torch.randint(1, 100, (4, 3), device="cuda", dtype=torch.int32)
    stream = torch.cuda.Stream()

    def calls(**kw):
        """The results of all calls, one after the other."""
        blob = comp.compress(K, V, budget, 0, **kw)
        out = [*comp.decompress(blob, torch.float32, **kw)]
        U, W = comp.factor(K, V, 0, **kw)
        torch.cuda.synchronize()
        U, W = U.bfloat16(), W.bfloat16()
        choice = torch.zeros(U.shape[0], dtype=torch.int32).cuda()
        torch.cuda.synchronize()
        core, tab = comp.table(K, V, U, W, 0, **kw)
        out += [U, W, core, tab, comp.recon_operator(core, W, 0, **kw)]
        out.append(comp.encode(K, V, U, W, core, choice, tab, 0, **kw))
        att = J.Attention(comp, blob, 8, **kw)
        out += [att.attend(1, q, **kw), *att.attend_state(1, q, **kw)]
        out += J.allocate(dist, nbytes, 150, **kw)
        out += [J.frobenius(K, V, layers_per_group=w.layers_per_group, **kw),
                J.frobenius_noalloc(K, V, layers_per_group=w.layers_per_group, **kw),
                *J.quant_baseline(K, V, 4, w.layers_per_group, True, **kw)]
        assert J.read_header(blob=blob, **kw)[1] <= budget
        return out

    want = calls()
    comp.dws = None
    torch.cuda.synchronize()
    seen = []

    def noting(f):
        def call(*args, **kw):
            if kw.get("device") is not None:
                seen.append(torch.cuda.current_stream().cuda_stream)
            return f(*args, **kw)
        return call
    for handle in (stream, stream.cuda_stream):
        seen.clear()
        for name in ("empty", "zeros", "empty_like"):
            monkeypatch.setattr(torch, name, noting(getattr(torch, name)))
        got = calls(stream=handle)
        monkeypatch.undo()
        torch.cuda.synchronize()
        assert len(seen) > 15 and set(seen) == {stream.cuda_stream}
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_attention_on_two_streams_at_once():
    """Calls of one Attention that overlap have a scratch each; the query is converted on the call's stream."""
    w = synth.small_workload("mistral7b", n_layers=4, n_heads=2, T=1024)
    K, V = (x.cuda() for x in synth.make_cache(w, 0))
    comp = J.Compressor(w.n_layers, w.n_heads, w.T, w.D, w.layers_per_group, K.dtype,
                        J.Options((64, 128), (64, 128), (0, 2, 4), "randomized"))
    att = J.Attention(comp, comp.compress(K, V, w.bf16_bytes() // 2, 0), 8)
    q = [torch.randn(8, 128, device="cuda").bfloat16() for _ in range(3)]
    want = [att.attend_state(2, x) for x in q]
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [att.attend_state(2, x, stream=st) for x, st in zip(q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
