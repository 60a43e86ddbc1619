"""Attention captured through its stream= argument while another stream is current: the graph has
a workspace of its own, as it has when the captured stream is the current one."""

import pytest
import torch

from cache_cases import Case, announce

pytestmark = pytest.mark.gpu


def test_capture_by_argument(monkeypatch):
    from speculative_sampling_verification_amd import _lib as svl
    announce("attention captured on stream=, replayed beside eager calls on that stream")
    cs = [Case(s, "bf16", [9000, 300, 1200], 8, 2, 4, 128, 16) for s in (50, 51)]
    caches, qs = [c.cache(svl) for c in cs], [c.dev(c.q) for c in cs]
    want = [svl.spec_tree_attention(q, k)["out"].clone() for q, k in zip(qs, caches)]
    outs = [dict(out=torch.empty_like(q)) for q in qs]
    used = []
    call = svl._cache_call

    def spy(cache, name, fn, *args):
        used.append((args[-3], args[-2]))  # the workspace and its size
        call(cache, name, fn, *args)
    monkeypatch.setattr(svl, "_cache_call", spy)
    s, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    svl.spec_tree_attention(qs[1], caches[1], out=outs[1], stream=s)  # the stream's workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin()
    svl.spec_tree_attention(qs[0], caches[0], out=outs[0], stream=s)
    with torch.cuda.stream(s):
        graph.capture_end()
    svl.spec_tree_attention(qs[1], caches[1], out=outs[1], stream=s)
    torch.cuda.synchronize()
    eager, captured, later = used
    assert eager == later
    assert captured[0] + captured[1] <= eager[0] or eager[0] + eager[1] <= captured[0]
    for rep in range(4):
        for out in outs:
            out["out"].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        svl.spec_tree_attention(qs[1], caches[1], out=outs[1], stream=s)
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out["out"], w), rep
