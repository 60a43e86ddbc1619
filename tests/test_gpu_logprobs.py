"""spec_token_logprobs (through the C ABI) against the oracle: tokens and ranks exactly, log
probabilities and entropies within rounding.

With u = 2^-24, x = z / T in nats, A and B the means of |x - x_max| and its square: the factor
log2(e) / T is rounded (u of all differences), each x - k once more (the shift k lies within 24 ln 2 <
17 of x_max), the exponential is off by 2 u, a lane sums n = ceil(V / 256) + 32 terms one after the
other.  So ln S is off by u (A + 17 + 2 + n + 16), a log probability by that and u (spread + A) for the
factor and u of itself; the entropy ln S + mean by the same, with every term times |x - k| again for
the mean: u (2 (B + 17^2) + (A + 17) (2 n + 40))."""

import numpy as np
import pytest
import torch

import oracle.decode_step_oracle as O
from cache_cases import DTYPES, F32_HALF_STEP, announce, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    return m


def logits_of(rng, R, V, dtype, kind):
    z = rng.standard_normal((R, V)) * 2.0
    if kind == "peaked":
        z -= 1.1 * np.log(rng.permutation(V) + 1.0)
    elif kind == "ties":
        z = np.round(z)
    elif kind == "constant":
        z[:] = 1.25
    elif kind == "ascending":
        z = np.tile(np.linspace(-30, 30, V), (R, 1))
    elif kind == "masked":        # few tokens allowed, as under a grammar
        z[rng.random((R, V)) < 0.97] = -np.inf
        z[:, V // 2] = 0.5
    elif kind == "lowest":        # masked by the type's lowest value
        z[rng.random((R, V)) < 0.9] = float(torch.finfo(DTYPES[dtype]).min)
    elif kind == "steep":         # the maximum grows by far along the row
        z += np.linspace(0, 3000, V)
    elif kind == "large":
        z = z * 1e30
    elif kind == "zeros":
        z = np.where(rng.random((R, V)) < 0.5, 0.0, -0.0)
    return torch.from_numpy(z).float().to(DTYPES[dtype])


def check(got, ref, V, temperature):
    u = F32_HALF_STEP
    n = -(-V // 256) + 32
    host = {k: v.double().cpu().numpy() for k, v in got.items()}
    for k in ("rank", "top_tokens"):
        if k in host:
            np.testing.assert_array_equal(host[k].reshape(ref[k].shape), ref[k], err_msg=k)
    base = u * (2 * ref["mean"] + 17 + 2 + n + 16)
    spread = np.where(np.isfinite(ref["spread"]), ref["spread"], 0.0)

    def close(x, want, tol):
        # -inf in fp32 too: half a step beyond its largest number, 2^128 - 2^104
        inf = np.abs(want) >= 2.0 ** 128 - 2.0 ** 103
        np.testing.assert_array_equal(x[inf], np.where(want[inf] < 0, -np.inf, np.inf))
        bad = ~inf & ~(np.abs(np.where(inf, 0, x) - np.where(inf, 0, want)) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4], x[bad][:4], want[bad][:4],
                               np.broadcast_to(tol, x.shape)[bad][:4])
    if "logprob" in host:
        w = ref["logprob"]
        close(host["logprob"].reshape(-1), w,
              base + u * (spread + np.where(np.isinf(w), 0, np.abs(w))))
    if "top_logprobs" in host and ref["top_tokens"].shape[1]:
        w = ref["top_logprobs"]
        f = np.where(np.isinf(w), 0, np.abs(w))
        close(host["top_logprobs"].reshape(w.shape), w, base[:, None] + 2 * u * f)
    if "entropy" in host:
        close(host["entropy"].reshape(-1), ref["entropy"],
              base + u * (2 * (ref["square"] + 17 ** 2) + (ref["mean"] + 17) * (2 * n + 40)))


SIZES = [(1, 1, 1), (3, 2, 5), (5, 1000, 5), (2, 4097, 64), (7, 33, 33), (4, 32000, 20),
         (1, 128256, 20), (2, 300001, 3), (600, 515, 1), (3, 16384, 64), (1, 7, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(svm, size, dtype):
    R, V, n = size
    announce(f"logprobs {size} {dtype}")
    rng = np.random.default_rng(V)
    z = logits_of(rng, R, V, dtype, "peaked")
    tokens = rng.integers(0, V, R).astype(np.int32)
    tokens[::3] = z.float().argmax(1).numpy()[::3]
    for T in (1.0, 0.6):
        ref = O.token_logprobs(z.double().numpy(), tokens, temperature=T, top_n=n)
        got = svm.spec_token_logprobs(z.cuda(), ints(tokens), temperature=T, top_n=n,
                                      want_rank=True, want_entropy=True)
        assert set(got) == {"logprob", "rank", "entropy", "top_tokens", "top_logprobs"}
        check(got, ref, V, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["ties", "constant", "ascending", "masked", "lowest", "steep",
                                  "large", "zeros"])
@pytest.mark.parametrize("R,V", [(2, 40009), (3, 257), (700, 2050)])
def test_values(svm, kind, R, V, dtype):
    announce(f"logprobs of {kind} rows {R}x{V} {dtype}")
    rng = np.random.default_rng(V + R)
    z = logits_of(rng, R, V, dtype, kind)
    tokens = rng.integers(0, V, R).astype(np.int32)
    tokens[0], tokens[-1] = 0, V - 1
    for T, n in ((1.0, 20), (2.5, 64)):
        ref = O.token_logprobs(z.double().numpy(), tokens, temperature=T, top_n=n)
        got = svm.spec_token_logprobs(z.cuda(), ints(tokens), temperature=T, top_n=n,
                                      want_rank=True, want_entropy=True)
        check(got, ref, V, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5000, 129, 8])
def test_phases(svm, V, dtype):
    """Rows that start at every offset within 16 bytes, and end there."""
    announce(f"logprobs at every phase, V={V} {dtype}")
    rng = np.random.default_rng(V)
    per = 8 if dtype == "bf16" else 4
    for phase in range(per):
        z = logits_of(rng, 3, V, dtype, "ties")
        buf = torch.full((3 * V + 2 * per,), 1e30, dtype=z.dtype, device="cuda")
        view = buf[phase:phase + 3 * V].view(3, V)
        view.copy_(z)
        tokens = np.array([0, V - 1, V // 2], dtype=np.int32)
        ref = O.token_logprobs(z.double().numpy(), tokens, top_n=9)
        got = svm.spec_token_logprobs(view, ints(tokens), top_n=9, want_rank=True, want_entropy=True)
        check(got, ref, V, 1.0)


def test_rows_without_a_distribution(svm):
    announce("rows and tokens out of range, rows of -inf, masked tokens")
    rng = np.random.default_rng(3)
    z = logits_of(rng, 5, 3000, "f32", "peaked")
    z[1] = -torch.inf
    z[2, 17:] = -torch.inf
    z[3, :2999] = -torch.inf
    tokens = np.array([5, 100, 2999, 2999, -1, 3000, 17, 3, 0, 2 ** 31 - 1], dtype=np.int32)
    rows = np.array([0, 1, 2, 3, 4, 4, 2, -1, 5, 0], dtype=np.int32)
    ref = O.token_logprobs(z.double().numpy(), tokens, rows, top_n=20)
    got = svm.spec_token_logprobs(z.cuda(), ints(tokens), rows=ints(rows), top_n=20, want_rank=True,
                                  want_entropy=True)
    check(got, ref, 3000, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 150001])
def test_rows_of_nan_and_infinity_touch_no_other(svm, V, dtype):
    announce(f"rows with NaN and +inf beside others, V={V} {dtype}")
    rng = np.random.default_rng(V)
    z = logits_of(rng, 6, V, dtype, "peaked")
    bad, good = [0, 2, 4], [1, 3, 5]
    z[0, V // 3] = torch.nan
    z[2, [0, V - 1]] = torch.inf
    z[4] = torch.nan
    tokens = rng.integers(0, V, 6).astype(np.int32)
    got = svm.spec_token_logprobs(z.cuda(), ints(tokens), top_n=64, want_rank=True,
                                  want_entropy=True)
    ref = O.token_logprobs(z[good].double().numpy(), tokens[good], top_n=64)
    check({k: x[good] for k, x in got.items()}, ref, V, 1.0)
    top = got["top_tokens"][bad]
    assert ((top >= -1) & (top < V)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_is_not_wanted_changes_nothing(svm, dtype):
    announce(f"logprobs: subsets of the outputs, shapes, {dtype}")
    rng = np.random.default_rng(4)
    z = logits_of(rng, 6, 9001, dtype, "peaked").cuda()
    tokens = ints(rng.integers(0, 9001, 6).astype(np.int32))
    full = svm.spec_token_logprobs(z, tokens, top_n=7, want_rank=True, want_entropy=True)
    for kw in (dict(), dict(want_rank=True), dict(want_entropy=True), dict(top_n=7),
               dict(top_n=7, want_rank=True), dict(want_entropy=True, want_rank=True)):
        got = svm.spec_token_logprobs(z, tokens, **kw)
        for k, x in got.items():
            assert torch.equal(x, full[k]), (kw, k)
    for kw in (dict(top_n=7), dict(want_entropy=True), dict(top_n=7, want_entropy=True)):
        got = svm.spec_token_logprobs(z, **kw)
        assert "logprob" not in got
        for k, x in got.items():
            assert torch.equal(x, full[k]), (kw, k)
    shaped = svm.spec_token_logprobs(z.view(2, 3, -1), tokens.view(2, 3), top_n=7, want_rank=True)
    assert shaped["top_tokens"].shape == (2, 3, 7)
    assert torch.equal(shaped["top_logprobs"].view(6, 7), full["top_logprobs"])
    one = svm.spec_token_logprobs(z[0], tokens[0], top_n=7)
    assert one["logprob"].shape == () and torch.equal(one["top_tokens"], full["top_tokens"][0])
    again = svm.spec_token_logprobs(z, tokens[[4, 4, 0]], rows=ints(np.array([4, 4, 0],
                                                                            dtype=np.int32)))
    assert torch.equal(again["logprob"], full["logprob"][[4, 4, 0]])


def test_after_a_verify_step(svm):
    announce("logprobs of a verify step's tokens, -1 where none was emitted")
    rng = np.random.default_rng(5)
    B, K, V = 4, 3, 5000
    t = logits_of(rng, B * (K + 1), V, "bf16", "peaked").view(B, K + 1, V).cuda()
    d = (t[:, :K].float() + torch.from_numpy(rng.standard_normal((B, K, V))).cuda()).bfloat16()
    u = svm.spec_philox_uniform((1, 2), 0, B * K)
    drafts = svm.spec_sample(d.view(B * K, V), u).view(B, K)
    out = svm.spec_verify(t, d, drafts, svm.spec_philox_uniform((3, 4), 0, B * (K + 1)).view(B, -1))
    got = svm.spec_token_logprobs(t, out["tokens"], top_n=4, want_rank=True)
    ref = O.token_logprobs(t.view(-1, V).double().cpu().numpy(),
                           out["tokens"].view(-1).cpu().numpy(), top_n=4)
    check(got, ref, V, 1.0)
    emitted = torch.arange(K + 1, device="cuda")[None, :] <= out["num_accepted"][:, None]
    assert torch.equal(got["logprob"] > -torch.inf, emitted)
    # accepted drafts: the target's probability of them
    q = out["q_draft"][:, :K]
    accepted = torch.arange(K, device="cuda")[None, :] < out["num_accepted"][:, None]
    assert torch.allclose(got["logprob"][:, :K][accepted].exp(), q[accepted], rtol=1e-4)


def test_streams_and_graphs(svm):
    announce("logprobs on another stream; two captured graphs with workspaces of their own")
    rng = np.random.default_rng(6)
    zs = [logits_of(rng, 2, 100000, "bf16", "peaked").cuda() for _ in range(2)]
    tokens = ints(rng.integers(0, 100000, 2).astype(np.int32))
    kw = dict(top_n=20, want_rank=True, want_entropy=True)
    want = [svm.spec_token_logprobs(z, tokens, **kw) for z in zs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = svm.spec_token_logprobs(zs[0], tokens, stream=side, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[0][k]) for k in got)
    outs, graphs = [], []
    for z in zs:
        out = {k: torch.empty_like(x) for k, x in want[0].items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            svm.spec_token_logprobs(z, tokens, out=out, **kw)
        outs.append(out)
        graphs.append(graph)
    for rep in range(4):
        for out in outs:
            for x in out.values():
                x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        eager = svm.spec_token_logprobs(zs[0], tokens, **kw)
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert all(torch.equal(out[k], w[k]) for k in w), rep
        assert all(torch.equal(eager[k], want[0][k]) for k in eager)
