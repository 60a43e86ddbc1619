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


def within(got, want, tol, name):
    worst = float(np.max(np.abs(got - want) / tol))
    print(f"{name}: off by {float(np.max(np.abs(got - want))):.1e}, {worst:.2f} of the bound")
    return worst <= 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,tiles", [(3, 1), (3, 5), (300, 4)])
@pytest.mark.parametrize("T", [1.0, 0.3])
def test_confident_rows(svm, T, R, tiles, dtype):
    """One token, the row's last, of 2^18 to 2^23 times the weight of any other: what a thread that
    began with the others adds it to has to move up to it.

    In nats, t is the others' share, m and q the means of |x - x_max| and its square; the shift lies at
    most 2 ln 2 < 1.4 below the maximum.  The token's x is off by u (in log2 units, below 2), its weight
    by 0.7 u for that and 2 u for the exponential, and two additions behind it (its tile's sum is
    complete then) by u each; the others' sums of 32 logits a tile and `tiles` tiles by 62 u in all; and
    the factor log2(e) / T, rounded, moves ln S by u m.  So ln S is off by u (4.7 + 63 t + 2 m).  The
    mean of x: 0.7 u for the token's x, 1.4 u for its product, 1.4 u and 2.8 u for what the additions do
    to it and, through S, to the quotient, 2.7 u m for the weight, and 66 u of the others' part, 62 t u of
    the quotient, twice u q for their x: with ln S, u (11 + 240 t + 72 m + 2 q)."""
    V = tiles * 4 * THREADS * VECTOR[dtype]
    announce(f"logprobs of {R} confident rows of {V} {dtype}, T={T}")
    rng = np.random.default_rng(R + tiles)
    z = 0.5 * T * rng.standard_normal((R, V))
    above = rng.uniform(18.1, 22.9, R)
    z[:, -1] = z[:, :-1].max(1) + above * np.log(2) * T
    logits, z = device(z, dtype)
    tokens = np.full(R, V - 1, dtype=np.int32)
    ref = O.token_logprobs(z, tokens, temperature=T, top_n=1)
    t, m, q = -np.expm1(ref["logprob"]), ref["mean"], ref["square"]
    assert (t < 0.2).all()
    got = host(svm.spec_token_logprobs(logits, ints(tokens), temperature=T, top_n=1,
                                       want_entropy=True))
    own = u * (4.7 + 63 * t + 2 * m + np.abs(ref["logprob"]))
    results = [within(got["logprob"], ref["logprob"], own, "logprob"),
               within(got["top_logprobs"][:, 0], ref["top_logprobs"][:, 0], own, "first"),
               within(got["entropy"], ref["entropy"],
                      u * (11 + 240 * t + 72 * m + 2 * q + ref["entropy"]), "entropy")]
    assert all(results)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,V", [(300, 128256), (5, 128256), (300, 32000), (9, 1000)])
@pytest.mark.parametrize("T", [1.0, 0.3])
def test_rows_of_a_model(svm, T, R, V, dtype):
    """Peaked rows with noise.  A thread adds up to 32 logits a tile and then the tiles, and rescales
    what it has where the shift moves (each time by a quarter at most: 2 u in all): n additions.  With m,
    q as above, every x off by u |x|, every weight by that and 2 u: ln S is off by u (n + 5 + 2 m), the
    mean of x, of numbers of at most |x - x_max| + 1.4, by u ((m + 1.4) (2 n + 10) + 2 (q + 2)), a log
    probability by ln S's, u of the distance to the maximum and u of itself."""
    n = 32 + -(-V // (4 * THREADS * VECTOR[dtype])) + 2
    announce(f"logprobs of {R} rows of {V} {dtype}, T={T}")
    rng = np.random.default_rng(V + R)
    z = rng.standard_normal((R, V)) - 1.1 * np.log(np.arange(1, V + 1))[rng.permutation(V)]
    logits, z = device(z, dtype)
    tokens = rng.integers(0, V, R).astype(np.int32)
    ref = O.token_logprobs(z, tokens, temperature=T, top_n=5)
    got = host(svm.spec_token_logprobs(logits, ints(tokens), temperature=T, top_n=5,
                                       want_entropy=True))
    m, q = ref["mean"], ref["square"]
    ln_s = u * (n + 5 + 2 * m)
    first, each = ref["top_logprobs"], np.abs(ref["top_logprobs"])
    results = [within(got["logprob"], ref["logprob"],
                      ln_s + u * (ref["spread"] + np.abs(ref["logprob"])), "logprob"),
               within(got["top_logprobs"], first,
                      ln_s[:, None] + u * (first[:, :1] - first + each), "first"),
               within(got["entropy"], ref["entropy"],
                      ln_s + u * ((m + 1.4) * (2 * n + 10) + 2 * (q + 2) + ref["entropy"]),
                      "entropy")]
    assert all(results)
