"""The step operators at the ends of their ranges: more rows and groups than one launch has
workgroups, offsets that pass 32 bits, extreme temperatures.

Where the same rows lie in a small array too, results are the same bit for bit."""

import numpy as np
import pytest
import torch

import oracle.decode_step_oracle as O
from cache_cases import F32_HALF_STEP, announce, ints
from test_gpu_logprobs import check, logits_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    yield m
    m.release_workspaces()
    torch.cuda.empty_cache()


def test_many_rows_of_logits(svm):
    R, V, n = 2 ** 20 + 3, 5, 2
    announce(f"logprobs of {R} rows")
    z = torch.randn((R, V), device="cuda")
    tokens = torch.randint(0, V, (R,), device="cuda", dtype=torch.int32)
    got = svm.spec_token_logprobs(z, tokens, top_n=n, want_rank=True, want_entropy=True)
    p = torch.log_softmax(z.double(), 1)
    order = torch.sort(z, dim=1, descending=True, stable=True)[1]
    assert torch.equal(got["top_tokens"], order[:, :n].int())
    at = torch.sort(order, 1)[1].gather(1, tokens.long()[:, None])[:, 0]
    assert torch.equal(got["rank"], at.int())
    # 33 terms a lane, means of |x - max| below the row's spread: as in the tests of few rows
    spread = (z.max(1)[0] - z.min(1)[0]).double()
    base = F32_HALF_STEP * (3 * spread + 17 + 2 + 33 + 16)
    w = p.gather(1, tokens.long()[:, None])[:, 0]
    assert ((got["logprob"] - w).abs() <= base + F32_HALF_STEP * w.abs()).all()
    h = -(p.exp() * p).sum(1)
    assert ((got["entropy"] - h).abs()
            <= base + F32_HALF_STEP * (2 * (spread ** 2 + 17 ** 2) + (spread + 17) * 106)).all()


def test_a_row_of_most_tokens(svm):
    V = 2 ** 31 - 1
    announce(f"logprobs of one row of {V} bf16 logits")
    z = torch.zeros((1, V), device="cuda", dtype=torch.bfloat16)
    at = {5: 4.0, V - 9: 3.0, V - 1: 2.0}
    for i, x in at.items():
        z[0, i] = x
    total = V - len(at) + sum(np.exp(x) for x in at.values())
    # a lane's 4096 tiles of 32 logits one after the other
    tol = F32_HALF_STEP * (4096 + 32 + 40 + 2 * 30)
    # V - 2 is the last of the zeros and all others lie above: V - 1 tokens come before it
    for token, rank in ((5, 0), (V - 1, 2), (V - 2, V - 1), (0, 3)):
        got = svm.spec_token_logprobs(z, ints(np.array([token], dtype=np.int32)), top_n=5,
                                      want_rank=True)
        assert got["rank"].item() == rank
        assert got["top_tokens"].tolist() == [[5, V - 9, V - 1, 0, 1]]
        want = at.get(token, 0.0) - np.log(total)
        assert abs(got["logprob"].item() - want) <= tol
    del z
    torch.cuda.empty_cache()


def test_rows_far_into_the_logits(svm):
    rows, V = 20000, 128256
    announce(f"logprobs of rows up to {rows} of {V} bf16 logits")
    z = torch.empty((rows, V), device="cuda", dtype=torch.bfloat16)
    some = torch.randn((2, V), device="cuda").bfloat16()
    z[0], z[rows - 1] = some
    at = ints(np.array([rows - 1, 0, rows - 1, rows], dtype=np.int32))
    near = ints(np.array([1, 0, 1, 2], dtype=np.int32))
    tokens = ints(np.array([9, V - 1, 100000, 3], dtype=np.int32))
    kw = dict(top_n=20, want_rank=True, want_entropy=True)
    got = svm.spec_token_logprobs(z, tokens, rows=at, **kw)
    want = svm.spec_token_logprobs(some, tokens, rows=near, **kw)
    assert all(torch.equal(got[k], want[k]) for k in want)
    del z
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("power", [-100, -13, 13, 127])
def test_temperatures(svm, power, dtype):
    T = 2.0 ** power
    announce(f"logprobs at temperature 2^{power} {dtype}")
    rng = np.random.default_rng(power + 200)
    z = logits_of(rng, 3, 3000, dtype, "peaked")
    tokens = np.array([7, int(z[1].float().argmax()), 2999], dtype=np.int32)
    ref = O.token_logprobs(z.double().numpy(), tokens, temperature=T, top_n=20)
    got = svm.spec_token_logprobs(z.cuda(), ints(tokens), temperature=T, top_n=20, want_rank=True,
                                  want_entropy=True)
    check(got, ref, 3000, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-1e29, -1e31, -3e38])
@pytest.mark.parametrize("V", [7, 300, 3000, 40009])
def test_rows_of_low_logits(svm, V, low, dtype):
    """Rows of which nothing, or little, lies above a mask's low value."""
    announce(f"logprobs of {V} logits of about {low} {dtype}")
    rng = np.random.default_rng(V)
    z = torch.full((3, V), low, dtype=torch.float64)
    z[1] *= torch.from_numpy(rng.uniform(0.5, 1.0, V))
    z[2, V // 2] = 3.0
    z = z.float().bfloat16() if dtype == "bf16" else z.float()
    tokens = np.array([V - 1, 0, V // 2], dtype=np.int32)
    for power in (0, 90):
        ref = O.token_logprobs(z.double().numpy(), tokens, temperature=2.0 ** power, top_n=9)
        got = svm.spec_token_logprobs(z.cuda(), ints(tokens), temperature=2.0 ** power, top_n=9,
                                      want_rank=True, want_entropy=True)
        check(got, ref, V, 2.0 ** power)


def test_many_tokens_turned(svm):
    B, N = 3, 700001
    announce(f"rotary of {B} x {N} tokens in place")
    x = torch.randn((B, N, 1, 4), device="cuda")
    freq = torch.tensor([1.0, 0.01], dtype=torch.float64, device="cuda")
    base = ints(np.array([0, -5, 10 ** 6], dtype=np.int32))
    t = base.double()[:, None] + torch.arange(N, device="cuda")[None, :]
    a = t[..., None] * freq
    lo, hi = x[:, :, 0, :2].double(), x[:, :, 0, 2:].double()
    want = torch.cat([lo * a.cos() - hi * a.sin(), lo * a.sin() + hi * a.cos()], 2)
    size = torch.cat([lo.abs() + hi.abs()] * 2, 2)
    svm.spec_rotary(x, freq, base=base, out={"q": x})
    tol = size * (8 * F32_HALF_STEP + 2.0 ** -50 * torch.cat([a.abs()] * 2, 2))
    assert ((x[:, :, 0].double() - want).abs() <= tol).all()


def test_many_heads_evicted(svm):
    layers, Hkv, page = 4096, 300, 2
    announce(f"evict in {layers} layers of {Hkv} heads")
    k = torch.randn((layers, 3, page, Hkv, 4), device="cuda")
    v = torch.randn_like(k)
    table = ints(np.array([[2, 0]], dtype=np.int32))
    cache = svm.PagedCache(k, v, table, ints(np.array([4], dtype=np.int32)))
    w = torch.randint(0, 5, (layers, 1, Hkv, 4), device="cuda").float()
    keep = ints(np.array([2], dtype=np.int32))
    kept = torch.sort(w, dim=3, descending=True, stable=True)[1][..., :2].sort(3)[0]

    def tokens(x):  # [layers, heads, token, 4] in order of position
        return x[:, [2, 0]].reshape(layers, 4, Hkv, 4).transpose(1, 2)
    index = kept[:, 0, :, :, None].expand(-1, -1, -1, 4)
    want = [tokens(x).gather(2, index) for x in (k, v)]
    rest = [tokens(x)[:, :, 2:].clone() for x in (k, v)]
    got = svm.spec_cache_evict(cache, w, keep)
    assert torch.equal(got["kept"][..., :2], kept.int()) and (got["kept"][..., 2:] == -1).all()
    assert torch.equal(got["weights"][..., :2], w.gather(3, kept))
    assert (got["weights"][..., 2:] == 0).all() and got["lens"].tolist() == [2]
    for x, moved, left in zip((k, v), want, rest):
        assert torch.equal(tokens(x)[:, :, :2], moved) and torch.equal(tokens(x)[:, :, 2:], left)


def test_pages_far_into_a_cache(svm):
    pages, page, Hkv, D, few = 2 ** 20 + 12, 16, 2, 64, 12  # 4 KB a page
    announce("append, weigh and evict behind the first 4 GB of keys")
    rng = np.random.default_rng(1)
    k = torch.empty((1, pages, page, Hkv, D), device="cuda", dtype=torch.bfloat16)
    far = svm.PagedCache(k, torch.empty_like(k), ints(
        (pages - 1 - rng.permutation(few)).reshape(2, 6).astype(np.int32)),
        ints(np.array([70, 41], dtype=np.int32)))
    near = svm.PagedCache(torch.randn((1, few, page, Hkv, D), device="cuda").bfloat16(),
                          torch.randn((1, few, page, Hkv, D), device="cuda").bfloat16(),
                          far.page_table - (pages - few), far.seq_lens.clone())
    for a, b in ((far.k, near.k), (far.v, near.v)):
        a[:, pages - few:] = b
    results = []
    q0, k_new, v_new = (torch.randn((2, 20, h, D), device="cuda").bfloat16() for h in (8, 2, 2))
    freq, _ = svm.rotary_frequencies(D)
    for cache in (far, near):
        q = svm.spec_rotary_append(q0, k_new, v_new, cache, freq)
        w = torch.zeros((1, 2, Hkv, 96), device="cuda")
        for n in (2, 20):  # both kernels
            att = svm.spec_tree_attention(q[:, :n].contiguous(), cache, want_lse=True)
            svm.spec_cache_weigh(q[:, :n].contiguous(), att["lse"], cache, w)
        got = svm.spec_cache_evict(cache, w, ints(np.array([33, 20], dtype=np.int32)), recent=3)
        results.append([q, w, got["kept"], got["lens"], got["weights"], cache.k[:, -few:],
                        cache.v[:, -few:]])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert results[0][1].abs().sum() > 0 and results[0][3].tolist() == [33, 20]


def test_weights_of_many_heads_and_tokens(svm):
    Hkv, D, L = 1024, 64, 2 ** 21  # 2^31 weights a layer
    announce("weigh: more than 2^31 weights a layer, in the second one")
    k = torch.randn((2, 2, 4, Hkv, D), device="cuda").bfloat16()
    cache = svm.PagedCache(k, torch.zeros_like(k), ints(np.array([[1, 0]], dtype=np.int32)),
                           ints(np.array([7], dtype=np.int32)))
    q = torch.randn((1, 20, Hkv, D), device="cuda").bfloat16()
    w = torch.zeros((2, 1, Hkv, L), device="cuda")
    near = torch.zeros((2, 1, Hkv, 8), device="cuda")
    for n in (1, 20):  # both kernels
        lse = torch.zeros((1, n, Hkv), device="cuda")
        for x in (w, near):
            svm.spec_cache_weigh(q[:, :n].contiguous(), lse, cache, x, layer=1)
    assert torch.equal(w[..., :8], near) and (near[1, ..., :7] > 0).all()
    assert (near[0] == 0).all() and (near[1, ..., 7] == 0).all()
    del w
    torch.cuda.empty_cache()


def test_threads_share_a_stream(svm):
    announce("logprobs in parts from four threads on one stream")
    from concurrent.futures import ThreadPoolExecutor
    z = torch.randn((4, 3, 70000), device="cuda")
    kw = dict(top_n=20, want_rank=True, want_entropy=True)
    tokens = ints(np.array([[1, 2, 3]] * 4, dtype=np.int32))
    want = [svm.spec_token_logprobs(z[i], tokens[i], **kw) for i in range(4)]
    torch.cuda.synchronize()

    def calls(i):
        return [svm.spec_token_logprobs(z[i], tokens[i], **kw) for _ in range(50)]
    with ThreadPoolExecutor(4) as pool:
        results = list(pool.map(calls, range(4)))
    torch.cuda.synchronize()
    for i, many in enumerate(results):
        for got in many:
            assert all(torch.equal(got[k], want[i][k]) for k in got)
