"""How near spec_token_logprobs comes to float64, held to what its order of sums can lose.

u = 2^-24 is half a step of fp32."""

import numpy as np
import pytest
import torch

import oracle.decode_step_oracle as O
from cache_cases import DTYPES, F32_HALF_STEP as u, announce, ints

pytestmark = pytest.mark.gpu

VECTOR = {"f32": 4, "bf16": 8}  # logits of 16 bytes
THREADS = 256                   # of a workgroup, each with a vector every 256


@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    return m


def device(z, dtype):
    t = torch.from_numpy(z).to(DTYPES[dtype])
    return t.cuda(), t.double().numpy()


def host(got):
    return {k: v.double().cpu().numpy() for k, v in got.items()}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [2, 300])
@pytest.mark.parametrize("tiles", [1, 3])
def test_sums_of_threads_are_joined_in_64_bits(svm, tiles, R, dtype):
    """A temperature of log2(e) makes weights powers of two.  Every thread has one of 2^-26 or none a
    tile, but for the one that has the row's maximum, of weight 1: what each thread sums is exact, and a
    tail of 2^-26 a thread is far below half a step of 1 however few threads are joined in fp32.

    The factor log2(e) / T is 1 (1 + 2^-26 in truth, u / 4): differences of 26 ln 2 < 19 in a logarithm,
    so a weight is off by 19 u at most, 2 u for the exponential; log p = -ln(1 + tail) and the
    entropy, tail (1 + 26 ln 2) nearly, by as much of themselves and u for their last rounding."""
    per = VECTOR[dtype]
    V = tiles * 4 * THREADS * per
    announce(f"logprobs: weights of powers of two, {R} rows of {V} {dtype}")
    rng = np.random.default_rng(tiles)
    z = np.full((R, V), -200.0)
    for r in range(R):
        for t in range(tiles):
            vector = 4 * THREADS * t + THREADS * rng.integers(0, 4, THREADS) + np.arange(THREADS)
            some = rng.random(THREADS) < 0.9 if r else np.ones(THREADS, bool)
            z[r, (vector * per + rng.integers(0, per, THREADS))[some]] = -26.0
        first = rng.integers(0, 64)  # a lane of the first wave, whose other weights go
        z[r].reshape(-1, THREADS, per)[:, first] = -200.0
        z[r, first * per] = 0.0
    T = float(np.float32(np.log2(np.e)))
    logits, z = device(z, dtype)
    tokens = z.argmax(1).astype(np.int32)
    ref = O.token_logprobs(z, tokens, temperature=T, top_n=1)
    got = host(svm.spec_token_logprobs(logits, ints(tokens), temperature=T, top_n=1,
                                       want_entropy=True))
    for name, want in (("logprob", ref["logprob"]), ("entropy", ref["entropy"]),
                       ("top_logprobs", ref["top_logprobs"])):
        worst = float(np.max(np.abs(got[name] - want) / np.abs(want))) / u
        assert worst <= 22, (name, worst)
