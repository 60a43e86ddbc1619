"""Who may write a page: rows of one sequence stay as they are whatever the others do, also where
reserves were refused, slots freed or tables trimmed and the batch goes on without looking."""

import numpy as np
import pytest
import torch

from cache_cases import announce, random_tree
from pool_cases import OwnedPool, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    return m


def chain_parent(S, N):
    return np.tile(np.arange(-1, N - 1, dtype=np.int32), (S, 1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("want", [8, 24])
def test_step_after_a_refused_reserve(svm, dtype, want):
    announce(f"append, attention and commit after a refused reserve, {dtype} want={want}")
    p = OwnedPool(svm, 1, 3, 6, 6, 4, 2, 2, 64, dtype)
    p.resize(i32(8, 0, 0))             # pages 0 and 1
    p.resize(i32(0, 16, 8))            # freed; 1 takes 0, 1, 2, 3 and 2 takes 4, 5
    assert p.table[0, :2].tolist() == [0, 1] and (p.ref > 0).all()
    p.lens[:] = 0, 14, 5
    p.upload()
    assert p.resize(i32(want, -1, -1)).tolist() == [0, 1, 1]
    before = [p.text(b) for b in range(3)]
    for layer in range(2):
        p.append(7, layer=layer)
        ref = p.attend(7, layer=layer)
        assert (ref["count"][0] == 0).all()  # no page: nothing is seen
    lens = p.commit(i32(6, 1, 2), chain_parent(3, 7))
    assert lens.tolist() == [0, 16, 8]
    for b in range(3):
        np.testing.assert_array_equal(p.text(b), before[b])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_with_freed_and_trimmed_slots(svm, dtype):
    announce(f"append to all slots, {dtype}: one freed, one trimmed, both without a reserve")
    p = OwnedPool(svm, 2, 4, 6, 9, 4, 2, 1, 64, dtype)
    p.resize(i32(8, 16, 0, 0))         # 0, 1 and 2, 3, 4, 5
    p.lens[:] = 0, 3, 0, 0
    p.upload()
    p.resize(i32(0, 3, 20, 8))         # 2: 0, 1, 3, 4, 5; 3: 6, 7; 8 is left
    p.lens[2:] = 17, 6
    p.upload()
    before = [p.text(b) for b in range(4)]
    for layer in range(2):
        p.append(6, layer=layer)
        p.attend(6, layer=layer)
    p.commit(i32(5, 5, 2, 1), chain_parent(4, 6))
    for b in range(4):
        np.testing.assert_array_equal(p.text(b), before[b])


def test_refused_entries_are_cleared(svm):
    announce("resize: entries that a refused sequence asked for, by values or for lack of pages")
    p = OwnedPool(svm, 3, 5, 6, 10, 4, 1, 1, 64)
    p.resize(i32(24, 8, 0, 0, 0))
    p.lens[:] = 3, 8, 0, 0, 0
    p.upload()
    p.resize(i32(4, 8, 0, 0, 0))
    # beyond the table; below the committed tokens; new lengths beyond the pages
    ok = p.resize(i32(25, 7, 12, 40, 9), i32(3, 8, 1, 0, 0))
    assert ok.tolist() == [0, 0, 0, 0, 1]
    assert p.table[0].tolist() == [0, -1, -1, -1, -1, -1] and p.table[2, :3].tolist() == [-1] * 3
    # 1, 2 and 3 of 10 pages are held: 0 takes two more, two are left, 2 asks for four and 3 for
    # six; 4 holds what it asks for
    ok = p.resize(i32(12, 8, 16, 24, 12), None)
    assert ok.tolist() == [1, 1, 0, 0, 1]
    assert (p.table[2, :4] == -1).all() and (p.table[3] == -1).all()


@pytest.mark.parametrize("seed,tight", [(s, s >= 8) for s in range(12)])
def test_committed_rows_stay(svm, seed, tight):
    rng = np.random.default_rng(100 + seed)
    S, width, page = int(rng.integers(3, 20)), int(rng.integers(2, 9)), int(rng.integers(1, 9))
    pages, dtype = int(rng.integers(4, S * width)), ["f32", "bf16"][seed % 2]
    pages = S + 2 if tight else pages
    announce(f"decoding steps over a pool of few pages, seed={seed} S={S} width={width} page={page} "
             f"pages={pages} {dtype}")
    p = OwnedPool(svm, seed, S, width, pages, page, 2, 1, 64, dtype)
    text = [p.text(b) for b in range(S)]
    refused = 0
    for step in range(12):
        # some slots freed, some trimmed to what is committed, the others left alone
        u = rng.random(S)
        p.resize(np.where(u < 0.15, 0, np.where(u < 0.6, p.lens, -1)).astype(np.int32))
        text = [t if p.held[b] else p.text(b) for b, t in enumerate(text)]
        if rng.random() < 0.5:
            F = int(rng.integers(1, S + 1))
            src, dst = (rng.integers(0, S, F).astype(np.int32) for _ in range(2))
            for x, d, ok in zip(src, dst, p.fork(src, dst)):
                if ok:
                    text[d] = text[x]
        # nodes for a part of the batch; the whole batch is fed
        N = int(rng.integers(1, 9))
        active = rng.random(S) < 0.7
        ok = p.resize(np.where(active, p.lens + N, -1).astype(np.int32))
        refused += int((ok == 0).sum())
        for layer in range(2):
            p.append(N, layer=layer)
            p.attend(N, np.where(active, N, 0).astype(np.int32), layer=layer)
        parent, _ = random_tree(rng, S, N)
        last = np.where(active, rng.integers(0, N, S), -1).astype(np.int32)
        lens = p.commit(last, parent)
        for b in range(S):
            np.testing.assert_array_equal(p.text(b), text[b], err_msg=f"step {step} sequence {b}")
        p.resize(np.full(S, -1, dtype=np.int32), lens)
        for b in range(S):
            np.testing.assert_array_equal(p.text(b, 0, text[b].shape[2]), text[b])
        text = [p.text(b) for b in range(S)]
        # no page behind the committed tokens, or begun, is another's too
        for b in range(S):
            assert (p.ref[p.table[b, p.lens[b] // page:p.held[b]]] == 1).all()
    assert refused > 0 or not tight


def test_cut_with_a_refused_want(svm):
    announce("resize: new lengths that cut into shared pages beside a want that is refused")
    p = OwnedPool(svm, 5, 6, 6, 40, 8, 1, 1, 64)
    p.resize(i32(40, 40, 40, 0, 0, 0))
    p.lens[:3] = 37, 37, 35
    p.upload()
    assert p.fork(i32(0, 1), i32(3, 4)).all()
    before = [p.text(b) for b in range(5)]
    # 0: want below the new length; 1: want beyond the table; 2: below, but all pages are its own
    ok = p.resize(i32(5, 49, 5, -1, -1, -1), i32(20, 20, 20, 37, 37, 0))
    assert ok.tolist() == [0, 0, 0, 1, 1, 1]
    assert p.lens.tolist() == [37, 37, 20, 37, 37, 0]
    p.append(6)
    for b in (0, 1, 3, 4):
        np.testing.assert_array_equal(p.text(b), before[b])
    # a cut that gives the shared pages back is taken
    assert p.resize(i32(24, 24, 20, -1, -1, -1), i32(24, 24, 20, 37, 37, 0)).all()
    p.append(6)
    for b in (3, 4):
        np.testing.assert_array_equal(p.text(b), before[b])


@pytest.mark.parametrize("seed", range(8))
def test_random_cuts_leave_shared_pages_whole(svm, seed):
    rng = np.random.default_rng(200 + seed)
    S, width, page = int(rng.integers(3, 16)), int(rng.integers(2, 9)), int(rng.integers(2, 9))
    announce(f"random cuts and forks, seed={seed} S={S} width={width} page={page}")
    p = OwnedPool(svm, seed, S, width, S * width, page, 1, 1, 64)
    for step in range(15):
        p.resize(rng.integers(-1, width * page + 2, S).astype(np.int32))
        p.lens = np.where(p.lens == 0, rng.integers(0, page * width + 1, S), p.lens)
        p.lens = np.minimum(p.lens, p.held * page).astype(np.int32)
        p.upload()
        src, dst = (rng.integers(0, S, S).astype(np.int32) for _ in range(2))
        p.fork(src, dst)
        for b in range(S):
            assert (p.ref[p.table[b, p.lens[b] // page:p.held[b]]] == 1).all()
        before = [p.text(b) for b in range(S)]
        new = rng.integers(0, p.lens + 2).astype(np.int32)
        p.resize(rng.integers(-1, width * page + 2, S).astype(np.int32), new)
        for b in range(S):
            assert (p.ref[p.table[b, p.lens[b] // page:p.held[b]]] == 1).all(), (step, b)
        p.append(int(rng.integers(1, 2 * page)))
        for b in range(S):
            n = min(int(p.lens[b]), before[b].shape[2])
            np.testing.assert_array_equal(p.text(b, 0, n), before[b][:, :, :n])
