"""The page pool's oracle by itself: a page that another sequence holds is never one that a
sequence will write, whatever lengths and wishes it is given."""

import numpy as np
import pytest

import oracle.paged_cache_oracle as O


def test_refused_want_keeps_a_cut_out_of_shared_pages():
    table = np.array([[0, 1, 2, 3, 4], [-1] * 5])
    lens, held = np.array([37, 0]), np.array([5, 0])
    ref = np.array([1, 1, 1, 1, 1, 0])
    k = np.zeros((1, 6, 8, 1, 1))
    assert O.fork(k, k.copy(), table, lens, held, ref, [0], [1]).tolist() == [1]
    for want in (5, 41, -1, 40):
        assert O.resize(table, lens, held, ref, np.array([want, -1]), 8,
                        np.array([20, 37])).tolist() == [0, 1]
        assert lens.tolist() == [37, 37] and held.tolist() == [5, 5]
    # 24 tokens are three pages: the shared fourth goes back, the cut stays out of the third
    assert O.resize(table, lens, held, ref, np.array([24, -1]), 8,
                    np.array([24, 37])).tolist() == [1, 1]
    assert lens.tolist() == [24, 37] and ref.tolist() == [2, 2, 2, 1, 0, 1]


@pytest.mark.parametrize("seed", range(20))
def test_pages_to_be_written_are_nobody_elses(seed):
    rng = np.random.default_rng(seed)
    S, width, page = 7, 5, 4
    pages = 30
    table = np.full((S, width), -1)
    lens, held, ref = np.zeros(S, int), np.zeros(S, int), np.zeros(pages, int)
    k = np.zeros((1, pages, page, 1, 1))
    for step in range(100):
        if step % 3 == 0:
            O.fork(k, k, table, lens, held, ref, rng.integers(0, S, 3), rng.integers(0, S, 3))
        else:
            O.resize(table, lens, held, ref, rng.integers(-1, width * page + 3, S), page,
                     rng.integers(0, width * page + 1, S))
        for b in range(S):
            assert lens[b] <= held[b] * page
            assert (ref[table[b, lens[b] // page:held[b]]] == 1).all()
