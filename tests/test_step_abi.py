"""CPU-side refusals of the entry points around tree attention: each bad argument returns its status
before anything touches a GPU, and the binding names what is wrong with a tensor."""

import ctypes
from types import SimpleNamespace

import pytest
import torch

from test_cache_abi import BAD_CACHES, cache

INVALID, DTYPE = 1, 2
D0 = 1 << 20  # stands for device memory; never dereferenced
Q, QO, K, KO, V, F, B, P, N = (i * 64 * D0 for i in range(3, 12))  # far from each other


@pytest.fixture(scope="module")
def svl():
    from speculative_sampling_verification_amd import _lib
    return _lib


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


ROTARY = dict(q=Q, qs=None, hq=4, oq=QO, k=K, ks=None, hk=2, ok=KO, dtype=1, seqs=3, N=5, D=64,
              freq=F, rot=64, inter=0, amplitude=1.0, base=B, positions=P)


def rotary(svl, **over):
    a = dict(ROTARY)
    a.update(over)
    return svl.lib().spec_rotary(*a.values(), None)


BAD_ROTARY = [
    dict(q=None), dict(oq=None), dict(k=None), dict(ok=None), dict(hq=0), dict(hk=0), dict(hq=-1),
    dict(hq=65537), dict(q=None, oq=None, hq=0, k=None, ok=None, hk=0), dict(seqs=0), dict(N=0),
    dict(seqs=2 ** 16, N=2 ** 15), dict(D=0), dict(D=60), dict(D=520), dict(freq=None),
    dict(freq=F + 4), dict(rot=0), dict(rot=7), dict(rot=66), dict(inter=2), dict(inter=-1),
    dict(amplitude=float("nan")), dict(amplitude=float("inf")), dict(q=Q + 8), dict(oq=QO + 2),
    dict(k=K + 4), dict(ok=KO + 8), dict(base=B + 2), dict(positions=P + 1),
    dict(qs=strides(5 * 256, 256, 60)), dict(ks=strides(-640, 128, 64)),
    # what is written is apart from all else
    dict(oq=Q + 64), dict(oq=K), dict(ok=Q), dict(ok=QO), dict(oq=F - 16), dict(ok=B - 16),
    dict(oq=P), dict(ok=K + 16),
    # in place: rows that lie apart
    dict(oq=Q, qs=strides(0, 256, 64)), dict(ok=K, ks=strides(640, 0, 64)),
    dict(oq=Q, qs=strides(5 * 512, 512, 64), k=Q + 2 * 128, ks=strides(5 * 512, 512, 64)),
    dict(oq=Q, qs=strides(5 * 512, 512, 64), k=Q + 2 * 256, ks=strides(5 * 512, 1024, 64)),
    dict(oq=Q, qs=strides(5 * 320, 320, 64), k=Q + 2 * 256, ks=strides(5 * 320, 320, 64)),
]


@pytest.mark.parametrize("over", BAD_ROTARY, ids=str)
def test_rotary_arguments(svl, over):
    assert rotary(svl, **over) == INVALID


def test_rotary_dtype(svl):
    assert rotary(svl, dtype=2) == DTYPE and rotary(svl, dtype=-1) == DTYPE


def append(svl, c=None, **over):
    a = dict(q=Q, qs=None, hq=4, oq=QO, k=K, v=V, ns=None, N=5,
             cache=ctypes.byref(c if c is not None else cache(svl)), layer=1, nodes=N, freq=F,
             rot=64, inter=0, amplitude=1.0, base=B, positions=P)
    a.update(over)
    return svl.lib().spec_rotary_append(*a.values(), None)


@pytest.mark.parametrize("over,status", BAD_CACHES, ids=[str(b[0]) for b in BAD_CACHES])
def test_append_refuses_a_bad_cache(svl, over, status):
    assert append(svl, cache(svl, **over)) == status


@pytest.mark.parametrize("over", [
    dict(k=None), dict(v=None), dict(N=0), dict(N=2049), dict(layer=2), dict(layer=-1),
    dict(cache=None), dict(q=None), dict(oq=None), dict(hq=0), dict(hq=-2), dict(nodes=N + 1),
    dict(rot=0), dict(rot=66), dict(freq=None), dict(inter=3), dict(amplitude=float("nan")),
    dict(v=V + 8), dict(ns=strides(640, 128, 4)), dict(oq=K), dict(oq=V), dict(oq=N), dict(oq=P),
    # the layer's keys and values, its tables
    dict(oq=D0), dict(oq=D0 + 2 * 10 * 16 * 128), dict(k=D0 + 2 * 10 * 16 * 128),
    dict(v=D0 + 2 * 10 * 16 * 128), dict(freq=D0 + 2 * 10 * 16 * 128),
    dict(q=2 * D0 + 2 * 10 * 16 * 128)], ids=str)
def test_append_arguments(svl, over):
    assert append(svl, **over) == INVALID


def test_keys_and_values_share_no_row(svl):
    assert append(svl, cache(svl, v=D0)) == INVALID


def test_binding_names_bad_tensors(svl):
    q, f = torch.zeros((3, 4, 2, 64)), torch.zeros(32, dtype=torch.float64)
    i = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: svl.spec_rotary(None, f), lambda: svl.spec_rotary(q[0], f),
                 lambda: svl.spec_rotary(q.double(), f), lambda: svl.spec_rotary(q.long(), f),
                 lambda: svl.spec_rotary(q, f.float()), lambda: svl.spec_rotary(q, f[None]),
                 lambda: svl.spec_rotary(q, None), lambda: svl.spec_rotary(q, f[::2]),
                 lambda: svl.spec_rotary(q, f, k=q[:, :3]), lambda: svl.spec_rotary(q, f, k=q[:2]),
                 lambda: svl.spec_rotary(q, f, k=q.bfloat16()),
                 lambda: svl.spec_rotary(q, f, base=i[:2]),
                 lambda: svl.spec_rotary(q, f, base=i.long()),
                 lambda: svl.spec_rotary(q, f, positions=i),
                 lambda: svl.spec_rotary(q.transpose(2, 3), f),
                 lambda: svl.spec_rotary(q, f)):  # host memory
        with pytest.raises((TypeError, ValueError)):
            call()
    k = torch.zeros((2, 6, 4, 2, 64))
    c = svl.PagedCache(k, k.clone(), torch.zeros((3, 5), dtype=torch.int32), i)
    new = torch.zeros((3, 4, 2, 64))
    for call in (lambda: svl.spec_rotary_append(q, new, new[:, :3], c, f),
                 lambda: svl.spec_rotary_append(q[:, :3], new, new, c, f),
                 lambda: svl.spec_rotary_append(q, q[:, :, :1], q[:, :, :1], c, f),
                 lambda: svl.spec_rotary_append(q.bfloat16(), new, new, c, f),
                 lambda: svl.spec_rotary_append(q, new, new, c, f.float()),
                 lambda: svl.spec_rotary_append(q, new, new, c, f, base=i.long()),
                 lambda: svl.spec_rotary_append(q, new, new, c, f, num_nodes=i[:1]),
                 lambda: svl.spec_rotary_append(q, new, new, c, f),
                 lambda: svl.spec_rotary_append(q, new, new, c, f, stream=SimpleNamespace(
                     cuda_stream=0, device=torch.device("cuda", 1)))):
        with pytest.raises((TypeError, ValueError)):
            call()


W = 13 * 64 * D0
LSE, SEEN, KEEP, LENS, KEPT, OW = ((14 + i) * 64 * D0 for i in range(6))


def weigh(svl, c=None, **over):
    a = dict(q=Q, qs=None, N=5, hq=4, lse=LSE, cache=ctypes.byref(c if c is not None else cache(svl)),
             layer=1, seen=SEEN, nodes=N, scale=0.125, decay=1.0, w=W, length=70)
    a.update(over)
    return svl.lib().spec_cache_weigh(*a.values(), None)


def evict(svl, c=None, **over):
    a = dict(cache=ctypes.byref(c if c is not None else cache(svl)), w=W, length=70, keep=KEEP,
             max_keep=40, sinks=2, recent=3, ow=OW, lens=LENS, kept=KEPT)
    a.update(over)
    return svl.lib().spec_cache_evict(*a.values(), None)


@pytest.mark.parametrize("over,status", BAD_CACHES, ids=[str(b[0]) for b in BAD_CACHES])
def test_weigh_and_evict_refuse_a_bad_cache(svl, over, status):
    assert weigh(svl, cache(svl, **over)) == status
    assert evict(svl, cache(svl, **over)) == status


@pytest.mark.parametrize("over", [
    dict(q=None), dict(lse=None), dict(w=None), dict(cache=None), dict(layer=-1), dict(layer=2),
    dict(N=0), dict(N=2049), dict(hq=0), dict(hq=3), dict(scale=0.0), dict(scale=float("nan")),
    dict(scale=3e38), dict(decay=-0.1), dict(decay=1.1), dict(decay=float("nan")), dict(length=0),
    dict(length=2 ** 30 + 1), dict(q=Q + 4), dict(lse=LSE + 2), dict(seen=SEEN + 1),
    dict(nodes=N + 2), dict(w=W + 2), dict(qs=strides(1280, 256, 60)), dict(qs=strides(-16, 256, 64)),
    # the layer's weights (layer 1: 3 * 2 * 70 floats in) share no memory with what is read
    dict(w=Q - 4 * 3 * 2 * 70), dict(w=LSE - 4 * 3 * 2 * 70), dict(w=SEEN - 4 * 3 * 2 * 70),
    dict(w=N - 4 * 3 * 2 * 70), dict(w=D0 + 2 * 10 * 16 * 128 - 4 * 3 * 2 * 70)], ids=str)
def test_weigh_arguments(svl, over):
    assert weigh(svl, **over) == INVALID


def test_weigh_takes_the_heads_that_attention_takes(svl):
    for dim in (32, 80, 512):
        c = cache(svl, head_dim=dim, head_stride=dim, token_stride=2 * dim, page_stride=32 * dim,
                  layer_stride=320 * dim)
        assert weigh(svl, c) == INVALID


@pytest.mark.parametrize("over", [
    dict(w=None), dict(keep=None), dict(ow=None), dict(lens=None), dict(kept=None), dict(cache=None),
    dict(length=0), dict(length=2 ** 30 + 1), dict(max_keep=0), dict(max_keep=71), dict(sinks=-1),
    dict(recent=-1), dict(w=W + 1), dict(keep=KEEP + 2), dict(ow=OW + 2), dict(lens=LENS + 2),
    dict(kept=KEPT + 2), dict(ow=W + 4), dict(ow=KEPT), dict(lens=KEEP + 8), dict(lens=KEPT),
    dict(kept=KEEP - 4), dict(kept=W), dict(ow=D0), dict(kept=2 * D0 - 4), dict(keep=D0 + 4),
    dict(w=2 * D0)], ids=str)
def test_evict_arguments(svl, over):
    assert evict(svl, **over) == INVALID


def test_evict_writes_no_shared_rows_and_no_huge_arrays(svl):
    assert evict(svl, cache(svl, v=D0)) == INVALID
    huge = cache(svl, layers=8192, kv_heads=1024, seqs=8192, pages=1, page_size=1, token_stride=0,
                 page_stride=0, head_stride=64, layer_stride=65536)
    assert evict(svl, huge, length=2 ** 30, max_keep=1) == INVALID
    assert weigh(svl, huge, hq=1024, length=2 ** 30) == INVALID
    # lengths over seq_lens: spec_cache_resize stores them
    c = cache(svl, seq_lens=LENS, v=4096 * D0)
    assert evict(svl, c) == INVALID


def test_binding_names_bad_weights(svl):
    k, i = torch.zeros((2, 6, 4, 2, 64)), torch.zeros(3, dtype=torch.int32)
    c = svl.PagedCache(k, k.clone(), torch.zeros((3, 5), dtype=torch.int32), i)
    q, lse = torch.zeros((3, 4, 4, 64)), torch.zeros((3, 4, 4))
    w = torch.zeros((2, 3, 2, 20))
    for bad in (w[:1], w[..., 0], w.double(), None, w.transpose(1, 2), w[..., ::2]):
        with pytest.raises((TypeError, ValueError)):
            svl.spec_cache_weigh(q, lse, c, bad)
        with pytest.raises((TypeError, ValueError)):
            svl.spec_cache_evict(c, bad, i)
    for call in (lambda: svl.spec_cache_weigh(q, lse[:, :3], c, w),
                 lambda: svl.spec_cache_weigh(q, None, c, w),
                 lambda: svl.spec_cache_weigh(q, lse.double(), c, w),
                 lambda: svl.spec_cache_weigh(q.bfloat16(), lse, c, w),
                 lambda: svl.spec_cache_weigh(q, lse, c, w, seen=i),
                 lambda: svl.spec_cache_weigh(q, lse, c, w),
                 lambda: svl.spec_cache_evict(c, w, i.long()),
                 lambda: svl.spec_cache_evict(c, w, None),
                 lambda: svl.spec_cache_evict(c, w, i, out={"weights": w[..., :10]}),
                 lambda: svl.spec_cache_evict(c, w, i, out={"kept": i}),
                 lambda: svl.spec_cache_evict(c, w, i)):
        with pytest.raises((TypeError, ValueError)):
            call()


def logprobs(svl, **over):
    a = dict(logits=Q, dtype=1, num_rows=6, V=100000, rows=None, tokens=K, R=6, T=1.0, n=5, lp=KO,
             rank=V, ent=F, top=B, toplp=P, ws=W, ws_bytes=1 << 30)
    a.update(over)
    return svl.lib().spec_token_logprobs(*a.values(), None)


@pytest.mark.parametrize("over", [
    dict(logits=None), dict(num_rows=0), dict(V=0), dict(R=0), dict(R=5), dict(rows=N, R=0),
    dict(T=0.0), dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-39), dict(n=-1),
    dict(n=65), dict(tokens=None), dict(lp=None), dict(n=0), dict(top=None), dict(toplp=None),
    dict(n=0, top=None, toplp=None, tokens=None, lp=None, rank=None, ent=None),
    dict(tokens=None, lp=None), dict(logits=Q + 1), dict(dtype=0, logits=Q + 2), dict(tokens=K + 2),
    dict(rows=N + 1), dict(lp=KO + 2), dict(rank=V + 1), dict(ent=F + 2), dict(top=B + 2),
    dict(toplp=P + 2), dict(ws=W + 8), dict(lp=Q), dict(rank=KO + 20), dict(ent=KO), dict(top=P - 100),
    dict(toplp=Q + 6 * 100000 * 2 - 4), dict(ws=Q), dict(lp=K - 4), dict(rows=N, R=6, lp=N),
    dict(ws=KO)], ids=str)
def test_logprob_arguments(svl, over):
    assert logprobs(svl, **over) == INVALID


def test_logprob_workspace(svl):
    size = svl.lib().spec_token_logprobs_workspace_size
    assert logprobs(svl, dtype=3) == DTYPE
    need = size(6, 100000, 1, 5)
    assert need > 16 and logprobs(svl, ws_bytes=need - 1) == 3 and logprobs(svl, ws=None) == 3
    for bad in ((0, 10, 1, 0), (1, 0, 1, 0), (1, 10, 2, 0), (1, 10, 1, -1), (1, 10, 1, 65)):
        assert size(*bad) == 0
    for R, V, n in ((1, 1, 0), (2 ** 31 - 1, 2 ** 31 - 1, 64), (1, 2 ** 31 - 1, 64), (511, 128256, 20)):
        for dt in (0, 1):
            assert 16 <= size(R, V, dt, n) < 2 ** 24 + R * 64


def test_binding_names_bad_logits(svl):
    z, t = torch.zeros((3, 4, 50)), torch.zeros((3, 4), dtype=torch.int32)
    for call in (lambda: svl.spec_token_logprobs(None, t), lambda: svl.spec_token_logprobs(z[..., ::2], t),
                 lambda: svl.spec_token_logprobs(z.double(), t), lambda: svl.spec_token_logprobs(z, t[:2]),
                 lambda: svl.spec_token_logprobs(z, t.long()), lambda: svl.spec_token_logprobs(z, 3),
                 lambda: svl.spec_token_logprobs(z, want_rank=True, top_n=2),
                 lambda: svl.spec_token_logprobs(z, t, rows=t[0]),
                 lambda: svl.spec_token_logprobs(z, t, rows=[1]),
                 lambda: svl.spec_token_logprobs(z, t, out={"entropy": z[..., 0]}),
                 lambda: svl.spec_token_logprobs(z[..., :0], t),
                 lambda: svl.spec_token_logprobs(torch.tensor(1.0), None, top_n=1),
                 lambda: svl.spec_token_logprobs(z, t),  # host memory
                 lambda: svl.spec_token_logprobs(z, t, stream=SimpleNamespace(
                     cuda_stream=0, device=torch.device("cuda", 1)))):
        with pytest.raises((TypeError, ValueError)):
            call()
