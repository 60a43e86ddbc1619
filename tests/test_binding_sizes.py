"""Sizes that the C ABI's 32-bit integers do not hold are refused by the binding; ctypes would pass on
their lower halves.  Tensors without memory, as the sizes are looked at before the device."""

import pytest
import torch

BIG = 2 ** 32 + 1  # 1 to a 32-bit integer


@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    return m


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def words(*shape):
    return meta(*shape, dtype=torch.int32)


@pytest.fixture
def cache(svm):
    k = meta(2, 6, 16, 2, 64)
    return svm.PagedCache(k, meta(2, 6, 16, 2, 64), words(1, 5), words(1))


def refused(call, *args, **kw):
    with pytest.raises(ValueError, match="out of range"):
        call(*args, **kw)


@pytest.mark.parametrize("shape", [(1, BIG, 1, 64), (BIG, 1, 1, 64), (1, 1, BIG, 64),
                                   (1, 2 ** 31, 1, 64)])
def test_rotary(svm, shape):
    freq = meta(32, dtype=torch.float64)
    refused(svm.spec_rotary, meta(*shape), freq)
    if shape[0] == 1:
        q = meta(shape[0], shape[1], 1, 64)
        refused(svm.spec_rotary, q, freq, k=meta(*shape))


def test_cache_calls(svm, cache):
    freq, new = meta(32, dtype=torch.float64), meta(1, 4, 2, 64)
    q, lse, w = meta(1, 4, 4, 64), meta(1, 4, 4, dtype=torch.float32), meta(2, 1, 2, 70,
                                                                            dtype=torch.float32)
    long = meta(1, BIG, 2, 64)
    refused(svm.spec_cache_append, long, long, cache)
    refused(svm.spec_rotary_append, meta(1, BIG, 4, 64), long, long, cache, freq)
    refused(svm.spec_rotary_append, meta(1, 4, BIG, 64), new, new, cache, freq)
    refused(svm.spec_rotary_append, q, new, new, cache, freq, layer=BIG)
    refused(svm.spec_tree_attention, meta(1, BIG, 4, 64), cache)
    refused(svm.spec_cache_weigh, meta(1, BIG, 4, 64), lse, cache, w)
    refused(svm.spec_cache_weigh, q, lse, cache, w, layer=-BIG)
    refused(svm.spec_cache_weigh, q, lse, cache, meta(2, 1, 2, BIG, dtype=torch.float32))
    refused(svm.spec_cache_evict, cache, meta(2, 1, 2, BIG, dtype=torch.float32), words(1))
    for name in ("sinks", "recent", "max_keep"):
        refused(svm.spec_cache_evict, cache, w, words(1), **{name: BIG})
        refused(svm.spec_cache_evict, cache, w, words(1), **{name: -BIG})


def test_logprobs(svm):
    refused(svm.spec_token_logprobs, meta(1, BIG), words(1))
    refused(svm.spec_token_logprobs, meta(1, 2 ** 31), words(1))
    refused(svm.spec_token_logprobs, meta(BIG, 1), words(BIG))
    refused(svm.spec_token_logprobs, meta(3, 100), words(3), top_n=BIG)
    refused(svm.spec_token_logprobs, meta(3, 100), words(BIG), rows=words(BIG))
