"""spec_rotary_append of keys and values without queries, as a layer does that fills a cache whose
queries are made elsewhere."""

import numpy as np
import pytest
import torch

import oracle.decode_step_oracle as O
from cache_cases import announce, ints
from test_gpu_rotary import Books, normal, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,Hkv,D,rot,interleaved", [(1, 2, 64, 64, False), (11, 3, 96, 20, True)])
def test_keys_and_values_alone(svm, N, Hkv, D, rot, interleaved, dtype):
    announce(f"rotary_append without queries, N={N} {Hkv}x{D} rot={rot} {dtype}")
    with_q, alone = (Books(svm, dtype, N, Hkv, D) for _ in range(2))
    rng = np.random.default_rng(N)
    q, k_new, v_new = (normal(rng, (5, N, h, D), dtype) for h in (4, Hkv, Hkv))
    kw = dict(layer=1, interleaved=interleaved, amplitude=0.9, base=ints(np.arange(
        0, 50, 10, dtype=np.int32)), num_nodes=ints(rng.integers(0, N + 1, 5).astype(np.int32)))
    freq = table(O.rotary_frequencies(rot)[0])
    svm.spec_rotary_append(q, k_new, v_new, with_q.cache, freq, **kw)
    assert svm.spec_rotary_append(None, k_new, v_new, alone.cache, freq, **kw) is None
    assert torch.equal(alone.k, with_q.k) and torch.equal(alone.v, with_q.v)
    with pytest.raises(ValueError):
        svm.spec_rotary_append(None, k_new, v_new, alone.cache, freq, out=q, **kw)
