"""Attention weights and eviction: the oracle against softmax itself, brute force and planted
mistakes."""

import itertools

import numpy as np

import oracle.decode_step_oracle as O


def cache(rng, B, lens, page, Hkv, D, layers=1):
    width = max(1, max(-(-n // page) for n in lens))
    pages = B * width + 2
    table = rng.permutation(pages)[:B * width].reshape(B, width).astype(np.int32)
    k, v = (rng.standard_normal((layers, pages, page, Hkv, D)) for _ in range(2))
    return k, v, table


def test_a_step_gives_every_row_one():
    rng = np.random.default_rng(0)
    lens, N, Hkv, G, D = [9, 4, 0], 2, 2, 3, 8
    k, v, table = cache(rng, 3, lens, 4, Hkv, D)
    q = rng.standard_normal((3, N, Hkv * G, D))
    # lse over the committed tokens alone: no nodes' keys
    lse = np.zeros((3, N, Hkv * G))
    for b, n in enumerate(lens):
        for i, h in itertools.product(range(N), range(Hkv * G)):
            kk = np.array([k[0, table[b, x // 4], x % 4, h // G] for x in range(n)]).reshape(n, D)
            z = kk @ q[b, i, h] * D ** -0.5
            lse[b, i, h] = np.log(np.exp(z).sum()) if n else -np.inf
    w, given, _ = O.weigh(q, lse, k[0], table, lens, np.zeros((3, Hkv, 11)))
    np.testing.assert_allclose(w.sum(-1), np.array([[N * G] * Hkv] * 2 + [[0] * Hkv]), rtol=1e-12)
    assert (w[0, :, 9:] == 0).all() and (w[1, :, 4:] == 0).all()
    # limits, nodes, decay and replacement
    seen = np.array([[9, 5], [2, 0], [1, 1]])
    x, _, _ = O.weigh(q, lse, k[0], table, lens, np.ones((3, Hkv, 11)), seen=seen, decay=0.5)
    y, _, _ = O.weigh(q[:, :1], lse[:, :1], k[0], table, lens, np.full((3, Hkv, 11), np.nan),
                      decay=0.0)
    z, _, _ = O.weigh(q, lse, k[0], table, lens, np.zeros((3, Hkv, 11)), nodes=[1, 1, 0])
    np.testing.assert_allclose(y[0, :, :9], z[0, :, :9])
    np.testing.assert_allclose(x[0, :, 5:9], 0.5 + z[0, :, 5:9])
    np.testing.assert_allclose(x[0, :, :5], 0.5 + w[0, :, :5])
    np.testing.assert_allclose(x[1, :, :2], 0.5 + z[1, :, :2])
    assert (x[1, :, 2:4] == 0.5).all() and (x[1, :, 4:] == 1).all()
    assert np.isnan(y[0, :, 9:]).all()


def test_kept_tokens_are_the_best_subset():
    rng = np.random.default_rng(1)
    for trial in range(60):
        n, page = int(rng.integers(2, 9)), int(rng.integers(1, 4))
        want = int(rng.integers(0, n))
        sinks = int(rng.integers(0, want + 1))
        recent = int(rng.integers(0, want - sinks + 1))
        k, v, table = cache(rng, 1, [n], page, 1, 2)
        w = rng.integers(0, 4, (1, 1, 1, n)).astype(np.float64)
        before = [(k[0, table[0, x // page], x % page, 0].copy(),
                   v[0, table[0, x // page], x % page, 0].copy()) for x in range(n)]
        lens, kept, out = O.evict(k, v, table, [n], w, [want], sinks, recent)
        stay = kept[0, 0, 0, :want].tolist()
        assert lens[0] == want and (kept[0, 0, 0, want:] == -1).all()
        # the largest weight of all allowed subsets, the first of them in order of position
        fixed = set(range(sinks)) | set(range(n - recent, n))
        best = max((s for s in itertools.combinations(range(n), want) if fixed <= set(s)),
                   key=lambda s: (w[0, 0, 0, list(s)].sum(), [-x for x in s]))
        assert stay == list(best)
        for j, x in enumerate(stay):
            np.testing.assert_array_equal(k[0, table[0, j // page], j % page, 0], before[x][0])
            np.testing.assert_array_equal(v[0, table[0, j // page], j % page, 0], before[x][1])
            assert out[0, 0, 0, j] == w[0, 0, 0, x]
        assert (out[0, 0, 0, want:] == 0).all()


def test_sequences_left_alone():
    rng = np.random.default_rng(2)
    lens = [5, 5, 5, 5, 5, 9, 5]
    k, v, table = cache(rng, 7, lens, 2, 1, 2)
    table[3, 1] = -1
    held = np.array([5] * 7, dtype=np.int32)
    ref = np.zeros(k.shape[1], dtype=np.int32)
    ref[table[table >= 0]] = 1
    ref[table[6, 1]] = 2
    w = rng.random((1, 7, 1, 8))
    args = dict(sinks=1, recent=1, held=held, refcount=ref)
    for keep, want in (([-1, 6, 1, 4, 4, 4, 4], [5, 5, 5, 5, 4, 9, 5]),
                       ([5, 3, 2, 0, 8, 9, 2], [5, 3, 2, 5, 5, 9, 2])):
        kk, vv = k.copy(), v.copy()
        got, kept, out = O.evict(kk, vv, table, lens, w, keep, max_keep=8, **args)
        assert got.tolist() == want
        for b in range(7):
            if want[b] == lens[b]:
                assert (kept[:, b] == -1).all() and (out[:, b] == w[:, b]).all()
                at = [p for p in table[b] if p >= 0]
                np.testing.assert_array_equal(kk[:, at], k[:, at])


def test_nan_is_the_least():
    rng = np.random.default_rng(3)
    k, v, table = cache(rng, 1, [6], 3, 1, 2)
    w = np.array([[[[np.nan, -np.inf, 0.0, -0.0, np.nan, 5.0]]]])
    for want, stay in ((1, [5]), (2, [2, 5]), (3, [2, 3, 5]), (4, [1, 2, 3, 5]), (5, [0, 1, 2, 3, 5])):
        _, kept, _ = O.evict(k.copy(), v.copy(), table, [6], w, [want])
        assert kept[0, 0, 0, :want].tolist() == stay
