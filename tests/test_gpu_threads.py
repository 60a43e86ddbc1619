"""Host threads on one stream: attention in two kernels over the stream's one workspace, with every
other thread's calls in between the calls, never inside them."""

import threading

import pytest
import torch

from cache_cases import Case, announce

pytestmark = pytest.mark.gpu


def test_threads_share_a_stream():
    import speculative_sampling_verification_amd as sv
    announce("four host threads, 150 attention calls each on one stream")
    cs = [Case(s, "bf16", [3000, 100 * s, 900], 8, 2, 4, 128, 16) for s in range(1, 5)]
    caches, qs = [c.cache(sv) for c in cs], [c.dev(c.q) for c in cs]
    want = [sv.spec_tree_attention(q, k)["out"].clone() for q, k in zip(qs, caches)]
    torch.cuda.synchronize()
    wrong, stream = [], torch.cuda.Stream()

    def work(n):
        outs = [torch.empty_like(want[n]) for _ in range(10)]
        for _ in range(15):
            for out in outs:
                sv.spec_tree_attention(qs[n], caches[n], out=dict(out=out), stream=stream)
        stream.synchronize()
        wrong.extend(n for out in outs if not torch.equal(out, want[n]))
    threads = [threading.Thread(target=work, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong
