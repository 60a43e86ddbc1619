"""spec_cache_append, _commit, _resize and _fork (through the C ABI) against the oracle: moved
rows bit for bit (NaN payloads included), lengths, tables and counts exactly."""

import numpy as np
import pytest
import torch

import oracle.paged_cache_oracle as O
from cache_cases import DTYPES, announce, ints, random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    return m


class Pool:
    """A cache and its page pool, on the device and in host arrays that the oracle changes."""

    def __init__(self, svm, seed, S, width, pages, page, layers=2, Hkv=2, D=64, dtype="bf16"):
        self.rng = np.random.default_rng(seed)
        self.svm, self.page = svm, page
        shape = (layers, pages, page, Hkv, D)
        g = torch.Generator().manual_seed(seed)
        k, v = (torch.randn(shape, generator=g).to(DTYPES[dtype]) for _ in range(2))
        self.kd, self.vd = k.cuda(), v.cuda()
        self.k, self.v = self.bits(k), self.bits(v)
        self.table = np.full((S, width), -1, dtype=np.int32)
        self.lens, self.held = (np.zeros(S, dtype=np.int32) for _ in range(2))
        self.ref = np.zeros(pages, dtype=np.int32)
        self.upload()

    @staticmethod
    def bits(t):
        return t.cpu().contiguous().view(torch.int16 if t.element_size() == 2 else
                                         torch.int32).numpy().copy()

    def upload(self):
        self.cache = self.svm.PagedCache(self.kd, self.vd, ints(self.table), ints(self.lens),
                                         seq_pages=ints(self.held), refcount=ints(self.ref))

    def resize(self, want, new_lens=None):
        got = self.svm.spec_cache_resize(self.cache, ints(want), new_lens=None if new_lens is None
                                         else ints(new_lens))
        ok = O.resize(self.table, self.lens, self.held, self.ref, want, self.page, new_lens)
        np.testing.assert_array_equal(got.cpu().numpy(), ok)
        self.same()
        return ok

    def fork(self, src, dst):
        got = self.svm.spec_cache_fork(self.cache, ints(src), ints(dst))
        ok = O.fork(self.k, self.v, self.table, self.lens, self.held, self.ref, src, dst)
        np.testing.assert_array_equal(got.cpu().numpy(), ok)
        self.same()
        return ok

    def same(self):
        torch.cuda.synchronize()
        c = self.cache
        np.testing.assert_array_equal(c.seq_lens.cpu().numpy(), self.lens)
        np.testing.assert_array_equal(c.seq_pages.cpu().numpy(), self.held)
        np.testing.assert_array_equal(c.refcount.cpu().numpy(), self.ref)
        table = c.page_table.cpu().numpy()
        for b, n in enumerate(self.held):
            if 0 <= n <= self.table.shape[1]:
                np.testing.assert_array_equal(table[b, :n], self.table[b, :n], err_msg=str(b))
        np.testing.assert_array_equal(self.bits(self.kd), self.k)
        np.testing.assert_array_equal(self.bits(self.vd), self.v)


def i32(*x):
    return np.array(x, dtype=np.int32)


# ------------------------------------------------------------------------------ append, commit
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,Hkv,D,page", [(1, 1, 1, 64, 16), (3, 7, 2, 96, 5), (5, 40, 3, 24, 16),
                                            (2, 300, 1, 128, 64), (4, 9, 8, 256, 1)])
def test_append(svm, dtype, B, N, Hkv, D, page):
    announce(f"append {dtype} B={B} N={N} Hkv={Hkv} D={D} page={page}")
    rng = np.random.default_rng(N)
    for nodes in (None, rng.integers(-2, N + 3, B).astype(np.int32)):
        width = 500 // page + 1
        p = Pool(svm, N, B, width, B * width, page, 2, Hkv, D, dtype)
        p.table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
        p.lens = rng.integers(0, 200, B).astype(np.int32)
        p.lens[0] = -3
        p.table[-1, 1] = -1  # a missing page: its rows are dropped
        p.upload()
        new = [torch.randn((B, N, Hkv, D)).to(DTYPES[dtype]) for _ in range(2)]
        svm.spec_cache_append(new[0].cuda(), new[1].cuda(), p.cache, layer=1,
                              num_nodes=None if nodes is None else ints(nodes))
        O.append(p.k[1], p.v[1], p.bits(new[0]), p.bits(new[1]), p.table, p.lens, nodes)
        p.same()


def test_append_strided(svm):
    announce("append from a fused projection, into a cache with heads before slots")
    pages, page, H, D, B, N = 20, 16, 2, 64, 3, 6
    kv = torch.zeros((2, pages, H, page, D), device="cuda").transpose(2, 3)
    table = np.arange(15, dtype=np.int32).reshape(3, 5)
    lens = i32(3, 15, 60)
    cache = svm.PagedCache(kv[0], kv[1], ints(table), ints(lens))
    qkv = torch.randn((B, N, 4 + H + H, D), device="cuda")
    svm.spec_cache_append(qkv[:, :, 4:6], qkv[:, :, 6:], cache)
    k, v = (np.zeros((pages, page, H, D)) for _ in range(2))
    O.append(k, v, qkv[:, :, 4:6].cpu().numpy(), qkv[:, :, 6:].cpu().numpy(), table, lens)
    np.testing.assert_array_equal(kv[0].cpu().numpy(), k)
    np.testing.assert_array_equal(kv[1].cpu().numpy(), v)


@pytest.mark.parametrize("dtype,N,layers,Hkv,D,page", [
    ("f32", 1, 1, 1, 64, 16), ("bf16", 8, 3, 2, 96, 3), ("bf16", 64, 5, 2, 64, 16),
    ("f32", 200, 2, 3, 32, 1), ("bf16", 33, 2, 1, 128, 64)])
def test_commit(svm, dtype, N, layers, Hkv, D, page):
    announce(f"commit {dtype} N={N} layers={layers} page={page}")
    B = 6
    width = 300 // page + 2
    p = Pool(svm, N, B, width, B * width, page, layers, Hkv, D, dtype)
    p.table = p.rng.permutation(B * width).reshape(B, width).astype(np.int32)
    p.lens = p.rng.integers(0, 90, B).astype(np.int32)
    parent, _ = random_tree(p.rng, B, N)
    for b in range(0, B, 2):  # deep trees: long paths, neighbours that move by little
        for i in range(1, N):
            parent[b, i] = max(0, i - int(p.rng.integers(1, 3)))
    last = p.rng.integers(0, N, B).astype(np.int32)
    last[0] = N - 1
    p.upload()
    before = p.lens.copy()
    got = svm.spec_cache_commit(p.cache, ints(last), parent=ints(parent))
    want = O.commit(p.k, p.v, p.table, p.lens, last, parent)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    p.same()
    np.testing.assert_array_equal(p.lens, before)
    chain = svm.spec_cache_commit(p.cache, ints(last), num_nodes=N)
    want = O.commit(p.k, p.v, p.table, p.lens, last, None, N)
    np.testing.assert_array_equal(chain.cpu().numpy(), want)
    p.same()


def test_commit_refuses_broken_paths(svm):
    announce("commit: nodes out of range, broken parents, missing pages, lengths out of range")
    B, N, page, width = 9, 12, 4, 8
    p = Pool(svm, 3, B, width, 80, page)
    p.table = p.rng.permutation(80)[:B * width].reshape(B, width).astype(np.int32)
    p.lens = i32(0, 5, 9, 3, 7, 10, -4, 31, 2 ** 31 - 1)
    parent = np.tile(i32(-1, 0, 0, 1, 2, 2, 3, 4, 5, 6, 7, 8), (B, 1))
    last = i32(-1, 12, 11, 9, 10, 8, 7, 6, 5)
    parent[2, 8] = 8          # its own parent
    parent[3, 6] = 7          # a later node
    parent[4, 2] = -7
    p.table[5, 3] = -1        # position 12 (node 2 of sequence 5) is missing
    p.upload()
    got = svm.spec_cache_commit(p.cache, ints(last), parent=ints(parent))
    want = O.commit(p.k, p.v, p.table, p.lens, last, parent)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert (want[:6] == np.maximum(p.lens[:6], 0)).all() and want[6] > 0
    p.same()


# ---------------------------------------------------------------------------------- page pool
def test_resize_rules(svm):
    announce("resize: growing, trimming, freeing, leaving alone, new lengths, bad values")
    p = Pool(svm, 1, 7, 6, 40, 8, 1)
    p.resize(i32(1, 8, 9, 48, 0, -1, 49))
    assert p.held.tolist() == [1, 1, 2, 6, 0, 0, 0]
    p.lens = i32(1, 8, 9, 40, 0, 0, 0)
    p.upload()
    ok = p.resize(i32(9, 7, 0, 40, 16, 2 ** 31 - 1, -2 ** 31))
    assert ok.tolist() == [1, 0, 1, 1, 1, 0, 1] and p.lens[2] == 0
    ok = p.resize(i32(16, 8, 3, 41, 12, 0, 1), i32(12, 8, 1, 42, -1, 0, 0))
    assert ok.tolist() == [1, 1, 0, 0, 0, 1, 1]


def test_resize_exhaustion(svm):
    announce("resize: too few free pages: served in order, the rest keep what they hold")
    p = Pool(svm, 2, 6, 10, 12, 4, 1)
    ok = p.resize(i32(16, 20, 16, 4, -1, 0))  # 4 + 5 + 4 of 12: the third does not fit
    assert ok.tolist() == [1, 1, 0, 0, 1, 1] and (p.ref != 0).sum() == 9
    # pages given back in the call serve it
    ok = p.resize(i32(0, 20, 16, 12, -1, 4))
    assert ok.tolist() == [1, 1, 1, 1, 1, 0]
    assert (p.ref == 0).sum() == 0
    ok = p.resize(i32(0, 0, 0, 0, 0, 0))
    assert (p.ref == 0).all() and (p.held == 0).all()


def test_fork_rules(svm):
    announce("fork: sharing, copies, chains of sharing, empty sources, refused forks")
    p = Pool(svm, 3, 12, 5, 30, 8, 3)
    p.resize(i32(20, 16, 3, 40, 0, 0, 0, 0, 0, 0, 0, 0))
    p.lens[:4] = 19, 16, 3, 40
    p.upload()
    ok = p.fork(i32(0, 0, 1, 2, 3), i32(4, 5, 6, 7, 8))
    assert ok.all() and p.ref[p.table[0, 0]] == 3 and p.table[4, 2] != p.table[5, 2]
    # same slot twice, a held slot, itself, out of range, a slot that is a source, empty source
    ok = p.fork(i32(1, 2, 0, 9, -1, 12, 0, 10, 3), i32(9, 9, 1, 9, 10, 10, 12, 11, -5))
    assert ok.tolist() == [0] * 7 + [1, 0]
    ok = p.fork(i32(1, 2, 4), i32(9, 9, 10))
    assert ok.tolist() == [1, 0, 1]
    # shared pages go back when the last holder does
    p.resize(i32(0, -1, -1, -1, -1, -1, -1, -1, -1, -1, -1, -1))
    p.resize(i32(-1, -1, -1, -1, 0, 0, -1, -1, -1, -1, 0, -1))
    assert p.fork(i32(), i32()).tolist() == []


def test_fork_exhaustion(svm):
    announce("fork: too few free pages: forks without a begun page still succeed")
    p = Pool(svm, 4, 8, 4, 6, 4, 1)
    p.resize(i32(9, 4, 0, 0, 0, 0, 0, 0))
    p.lens[:2] = 9, 4
    p.upload()
    ok = p.fork(i32(0, 0, 1, 0, 1), i32(2, 3, 4, 5, 6))
    assert ok.tolist() == [1, 1, 1, 0, 1]


@pytest.mark.parametrize("seed", range(6))
def test_random_pool_operations(svm, seed):
    rng = np.random.default_rng(seed)
    S, width, page = int(rng.integers(2, 60)), int(rng.integers(1, 12)), int(rng.integers(1, 20))
    pages = int(rng.integers(1, S * width + 40))
    announce(f"random pool operations seed={seed} S={S} width={width} page={page} pages={pages}")
    p = Pool(svm, seed, S, width, pages, page, 2, 1, 64)
    for step in range(25):
        if rng.random() < 0.4:
            F = int(rng.integers(1, S + 1))
            p.fork(rng.integers(-1, S + 1, F).astype(np.int32),
                   rng.integers(-1, S + 1, F).astype(np.int32))
            continue
        new = None
        if rng.random() < 0.6:
            new = np.minimum(p.lens + rng.integers(0, page + 2, S),
                             p.held * page + (rng.random(S) < 0.1)).astype(np.int32)
        base = p.lens if new is None else new
        want = base + rng.integers(-1, 3 * page, S)
        want = np.where(rng.random(S) < 0.2, 0, np.where(rng.random(S) < 0.2, -1, want))
        p.resize(want.astype(np.int32), new)


@pytest.mark.parametrize("S,pages,page", [(1024, 100003, 16), (8192, 20000, 4)])
def test_large_pools(svm, S, pages, page):
    announce(f"a pool of {pages} pages and {S} sequences (several rounds of the scan)")
    rng = np.random.default_rng(S)
    p = Pool(svm, 5, S, 8, pages, page, 1, 1, 8)
    p.ref[:] = rng.integers(0, 3, pages) * (rng.random(pages) < 0.7)
    taken = p.ref.copy()
    p.upload()
    p.resize(rng.integers(0, 4 * page, S).astype(np.int32))
    p.lens = np.minimum(rng.integers(0, 4 * page, S), p.held * page).astype(np.int32)
    p.upload()
    p.resize(np.where(rng.random(S) < 0.5, 0, p.lens + 2 * page).astype(np.int32))
    free = np.flatnonzero(p.held == 0)[:500]
    src = rng.choice(np.flatnonzero(p.held > 0), len(free)).astype(np.int32)
    p.fork(src, free.astype(np.int32))
    p.resize(np.zeros(S, dtype=np.int32))
    np.testing.assert_array_equal(p.ref, taken)


def test_unaligned_counts(svm):
    announce("resize over a count array that does not start on 16 bytes")
    ref = torch.zeros(1 + 50, dtype=torch.int32, device="cuda")[1:]
    ref[::2] = 1
    k = torch.zeros((1, 50, 4, 1, 64), device="cuda")
    held = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.full((3, 5), -1, dtype=torch.int32, device="cuda")
    cache = svm.PagedCache(k, k.clone(), table, torch.zeros_like(held), seq_pages=held,
                           refcount=ref)
    assert svm.spec_cache_resize(cache, ints(i32(20, 3, 8))).tolist() == [1, 1, 1]
    assert table[0].tolist() == [1, 3, 5, 7, 9] and table[2, :2].tolist() == [13, 15]


def test_taking_back_committed_tokens(svm):
    announce("resize: new lengths below the old ones, in own pages and in shared ones")
    p = Pool(svm, 5, 8, 6, 40, 8, 1)
    p.resize(i32(40, 40, 30, 0, 0, 0, 0, 0))
    p.lens[:3] = 37, 35, 30
    p.upload()
    assert p.fork(i32(0, 0, 2), i32(3, 4, 5)).all()
    # 0: into a page that 3 and 4 hold; 1: its own; 2: into its begun page, its own; 3: to a page's
    # end, the shared pages behind it given back; 4: the same, but kept
    ok = p.resize(i32(40, 40, 30, 16, 24, -1, -1, -1), i32(20, 3, 27, 16, 16, 30, 0, 0))
    assert ok.tolist() == [0, 1, 1, 1, 0, 1, 1, 1]
    assert p.lens.tolist() == [37, 3, 27, 16, 37, 30, 0, 0]
    # left alone otherwise, or freed whatever is shared; page 2 of 0 is 4's too, page 4 its own
    ok = p.resize(i32(-1, 0, -1, 0, 0, 2 ** 31 - 1, -1, -1), i32(33, 3, 5, 1, 2, 3, 0, 0))
    assert ok.tolist() == [1, 1, 0, 1, 1, 0, 1, 1]
    # the other holders gone: now 0 may
    assert p.lens.tolist() == [33, 0, 27, 0, 0, 30, 0, 0]
    assert p.resize(i32(40, 0, -1, 0, 0, 0, 0, 0), i32(20, 0, 30, 0, 0, 30, 0, 0)).all()
    assert p.lens.tolist() == [20, 0, 30, 0, 0, 0, 0, 0]


def test_seq_lens_as_the_wanted_ones(svm):
    announce("resize: want is seq_lens itself, with and without new lengths")
    p = Pool(svm, 7, 4, 6, 20, 8, 1)
    p.resize(i32(40, 17, 8, 0))
    p.lens = i32(9, 17, 0, 0)
    p.upload()
    want = p.lens.copy()
    ok = svm.spec_cache_resize(p.cache, p.cache.seq_lens)
    assert ok.tolist() == O.resize(p.table, p.lens, p.held, p.ref, want, 8).tolist() == [1] * 4
    p.same()
    want, new = p.lens.copy(), i32(3, 18, 0, 0)
    ok = svm.spec_cache_resize(p.cache, p.cache.seq_lens, new_lens=ints(new))
    assert ok.tolist() == O.resize(p.table, p.lens, p.held, p.ref, want, 8, new).tolist()
    p.same()


def test_fork_of_a_page_for_several_workgroups(svm):
    announce("fork: a begun page of 3000 rows, copied by many workgroups")
    p = Pool(svm, 6, 4, 2, 6, 3000, 2, 2, 256, "f32")
    p.resize(i32(2900, 3001, 0, 0))
    p.lens[:2] = 2899, 3001
    p.upload()
    assert p.fork(i32(0, 1), i32(2, 3)).all()


def test_graph_replays(svm):
    announce("a reserve, fork, commit and free sequence captured once and replayed")
    p = Pool(svm, 9, 6, 8, 60, 4, 2)
    p.resize(i32(10, 6, 12, 0, 0, 0))
    p.lens[:3] = 9, 4, 11
    p.upload()
    c = p.cache
    want, src, dst, last = ints(i32(20, 12, 20, -1, -1, -1)), ints(i32(0, 0, 2)), \
        ints(i32(3, 4, 5)), ints(i32(3, 2, 4, 0, 0, 0))
    parent = ints(np.tile(i32(-1, 0, 0, 1, 2), (6, 1)))
    free, trim = ints(i32(-1, -1, -1, 0, 0, 0)), c.seq_lens.clone()
    outs = [torch.zeros(6, dtype=torch.int32, device="cuda") for _ in range(4)]
    okf = torch.zeros(3, dtype=torch.int32, device="cuda")

    def call():
        svm.spec_cache_resize(c, want, out=outs[0])
        svm.spec_cache_commit(c, last, parent=parent, out=outs[1])
        svm.spec_cache_fork(c, src, dst, out=okf)
        svm.spec_cache_resize(c, free, out=outs[2])
        svm.spec_cache_resize(c, trim, out=outs[3])

    state = [p.kd, p.vd, c.page_table, c.seq_lens, c.seq_pages, c.refcount]
    start = [t.clone() for t in state]
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rep in range(4):
        for t, s in zip(state, start):
            t.copy_(s)
        last[:3] = torch.tensor([rep, 4 - rep, (rep * 2) % 5], dtype=torch.int32)
        want[:3] = torch.tensor([16 + 3 * rep, 12 + rep, 20], dtype=torch.int32)
        (torch.randn(256, 256, device="cuda") @ torch.randn(256, 256, device="cuda")).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in state + outs + [okf]]
        for t, s in zip(state, start):
            t.copy_(s)
        call()
        torch.cuda.synchronize()
        for g, w in zip(got, state + outs + [okf]):
            assert torch.equal(g, w), rep
