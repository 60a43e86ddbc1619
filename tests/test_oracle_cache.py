"""The paged-cache oracle pinned: attention against torch's float64 softmax over the gathered
sequence, movement and page counting against their definitions on small examples."""

import numpy as np
import pytest
import torch

import oracle.paged_cache_oracle as O
from cache_cases import Case, random_tree


@pytest.mark.parametrize("tree", [False, True])
def test_attention_is_softmax_over_the_visible_keys(tree):
    c = Case(3, "f32", [0, 7, 33], 6, 2, 3, 64, 4)
    mask = random_tree(c.rng, 3, 6)[1] if tree else None
    nodes = np.array([6, 2, 5])
    got = O.tree_attention(c.q, c.k, c.v, c.table, c.lens, mask, nodes)
    for b in range(3):
        n = c.lens[b] + nodes[b]
        rows = np.arange(n)
        k = torch.from_numpy(c.k[c.table[b, rows // 4], rows % 4]).repeat_interleave(3, 1)
        v = torch.from_numpy(c.v[c.table[b, rows // 4], rows % 4]).repeat_interleave(3, 1)
        q = torch.from_numpy(c.q[b, :nodes[b]])
        z = torch.einsum("nhd,khd->hnk", q, k) / 8.0
        see = torch.ones((nodes[b], n), dtype=torch.bool)
        see[:, c.lens[b]:] = (torch.from_numpy(mask[b, :nodes[b], :nodes[b]]) != 0 if tree
                              else torch.ones((nodes[b],) * 2, dtype=torch.bool).tril())
        z = z.masked_fill(~see, -torch.inf)
        want = torch.einsum("hnk,khd->nhd", torch.softmax(z, -1), v)
        np.testing.assert_allclose(got["out"][b, :nodes[b]], want.numpy(), rtol=1e-12, atol=1e-13)
        # m + ln(l): scores below 10 in size, so a few roundings of 10 * 2^-53 = 1.1e-15 each,
        # however near zero the sum is
        np.testing.assert_allclose(got["lse"][b, :nodes[b]],
                                   torch.logsumexp(z, -1).T.numpy(), rtol=0, atol=2e-14)
        assert (got["out"][b, nodes[b]:] == 0).all()
        assert (got["lse"][b, nodes[b]:] == -np.inf).all()


def test_commit_keeps_the_path():
    # 12 slots of one sequence hold their own position; the tree's nodes start at 5
    k = np.arange(12.0).reshape(1, 3, 4, 1, 1)
    v = -k
    table, lens = np.array([[0, 1, 2]]), np.array([5])
    parent = np.array([[-1, 0, 0, 1, 2, 2, 4]])
    assert O.commit(k, v, table, lens, np.array([6]), parent).tolist() == [9]
    assert k.ravel()[5:9].tolist() == [5, 7, 9, 11] and v.ravel()[8] == -11


def test_pool_counts_add_up():
    rng = np.random.default_rng(0)
    S, width, page, pages = 9, 6, 4, 40
    table = np.full((S, width), -1, dtype=np.int32)
    lens, held = np.zeros(S, np.int32), np.zeros(S, np.int32)
    ref = np.zeros(pages, np.int32)
    k = rng.standard_normal((2, pages, page, 1, 2))
    v = rng.standard_normal((2, pages, page, 1, 2))
    for step in range(200):
        if step % 3 == 0:
            x, d = rng.integers(0, S, 2)
            before = [k[:, table[x, i // page], i % page].copy() for i in range(lens[x])]
            if O.fork(k, v, table, lens, held, ref, np.array([x]), np.array([d]))[0]:
                assert lens[d] == lens[x]
                for i, row in enumerate(before):
                    np.testing.assert_array_equal(k[:, table[d, i // page], i % page], row)
        else:
            want = lens + rng.integers(0, 8, S)
            want[rng.random(S) < 0.2] = 0
            new = np.minimum(lens + rng.integers(0, 3, S), held * page)
            O.resize(table, lens, held, ref, np.maximum(want, 0), page, new)
        count = np.zeros(pages, np.int32)
        for b in range(S):
            assert lens[b] <= held[b] * page
            np.add.at(count, table[b, :held[b]], 1)
        np.testing.assert_array_equal(count, ref)
