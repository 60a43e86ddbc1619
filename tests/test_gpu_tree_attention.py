"""spec_tree_attention (through the C ABI) against the float64 oracle: types, head layouts,
lengths, page sizes, masks, garbage behind every boundary, strides, streams and graphs."""

import numpy as np
import pytest
import torch

import oracle.paged_cache_oracle as O
from cache_cases import Case, DTYPES, announce, check_attention, ints, random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    return m


def run(svm, c, mask=None, nodes=None, scale=None, want_lse=True, cache=None, q=None, **kw):
    got = svm.spec_tree_attention(
        c.dev(c.q) if q is None else q, c.cache(svm) if cache is None else cache,
        mask=None if mask is None else ints(mask), num_nodes=None if nodes is None else ints(nodes),
        scale=scale, want_lse=want_lse, **kw)
    torch.cuda.synchronize()
    return got


def check(svm, c, mask=None, nodes=None, scale=None, **kw):
    got = run(svm, c, mask, nodes, scale, **kw)
    ref = O.tree_attention(c.q, c.k, c.v, c.table, c.lens, mask, nodes, scale)
    check_attention(got, ref, c.dtype, c.D)
    return got, ref


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("N,G,Hkv,page", [(1, 1, 2, 16), (1, 8, 1, 7), (5, 3, 2, 16),
                                          (13, 4, 2, 1), (20, 8, 1, 100)])
def test_shapes(svm, dtype, D, N, G, Hkv, page):
    announce(f"tree attention {dtype} D={D} N={N} G={G} Hkv={Hkv} page={page}")
    c = Case(D + N, dtype, [0, 1, 63, 200, 129], N, Hkv, G, D, page)
    _, mask = random_tree(c.rng, 5, N)
    check(svm, c, mask)
    check(svm, c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,G", [(7, 5), (33, 2), (64, 3), (64, 4), (150, 1), (70, 8)])
def test_row_tiles_and_ragged_nodes(svm, dtype, N, G):
    announce(f"tree attention {dtype} N={N} G={G}: several row tiles, ragged node counts")
    c = Case(N, dtype, [40, 0, 131, 5, 77], N, 2, G, 64, 16)
    _, mask = random_tree(c.rng, 5, N)
    nodes = np.array([N, 1, 0, N // 2, N - 1], dtype=np.int32)
    check(svm, c, mask, nodes)
    check(svm, c, None, nodes)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [96, 128, 256])
@pytest.mark.parametrize("N,G", [(33, 3), (70, 4), (9, 7)])
def test_row_tiles_of_wide_heads(svm, dtype, D, N, G):
    announce(f"tree attention {dtype} D={D} N={N} G={G}: several row tiles over longer contexts")
    c = Case(N + D, dtype, [700, 0, 131, 65, 1023], N, 2, G, D, 16)
    _, mask = random_tree(c.rng, 5, N)
    mask[2, N // 2:] = 0
    nodes = np.array([N, N, N // 2 + 3, 1, N - 1], dtype=np.int32)
    c.v[c.table[0, 702 // 16], 702 % 16, 1, ::5] = np.inf  # node 2 of sequence 0
    check(svm, c, mask, nodes)


@pytest.mark.parametrize("dtype,D,N,G", [("bf16", 128, 600, 2), ("bf16", 64, 300, 5), ("f32", 64, 500, 1),
                                         ("bf16", 256, 300, 1), ("f32", 128, 257, 1), ("bf16", 96, 400, 1)])
def test_long_chains(svm, dtype, D, N, G):
    announce(f"pieces of prompts as chains, {dtype} D={D} N={N} G={G}: tiles that some rows see")
    c = Case(N + D, dtype, [0, 100, 700], N, 1, G, D, 16)
    nodes = np.array([N, N // 2, N - 1], dtype=np.int32)
    c.v[c.table[0, 130 // 16], 130 % 16, 0, ::7] = -np.inf   # node 130 of sequence 0
    c.v[c.table[1, 141 // 16], 141 % 16, 0, 3] = np.nan      # node 41 of sequence 1
    c.k[c.table[2, 900 // 16], 900 % 16, 0, 5] = np.nan      # node 200 of sequence 2
    check(svm, c, None, nodes)
    tril = np.tril(np.ones((N, N), dtype=np.uint8))[None].repeat(3, 0)
    check(svm, c, tril, nodes)  # the same rows, no tile left out


@pytest.mark.parametrize("length", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_lengths_at_tile_edges(svm, length):
    announce(f"tree attention at a tile edge: {length} committed tokens")
    for dtype in ("f32", "bf16"):
        for N in (1, 9):
            check(svm, Case(length, dtype, [length], N, 1, 2, 64, 16))


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128), ("bf16", 256)])
def test_rows_without_keys(svm, dtype, D):
    announce(f"tree attention {dtype} D={D}: masks that leave rows empty")
    c = Case(3, dtype, [0, 0, 5], 40, 1, 2, D, 16)
    _, mask = random_tree(c.rng, 3, 40)
    mask[0] = 0               # no row of sequence 0 sees anything
    mask[1, ::2] = 0          # every other row of sequence 1
    got, ref = check(svm, c, mask)
    assert (ref["count"] == 0).sum() == 60
    assert torch.isinf(got["lse"][0]).all() and (got["out"][0] == 0).all()
    # any nonzero byte shows a node, and a mask need not be a tree's
    wild = (c.rng.integers(0, 3, (3, 40, 40)) * 127).astype(np.uint8)
    check(svm, c, wild)


@pytest.mark.parametrize("dtype,D,G", [("f32", 64, 2), ("f32", 256, 1), ("bf16", 64, 4),
                                       ("bf16", 128, 9), ("bf16", 256, 2)])
def test_hidden_non_finite_values(svm, dtype, D, G):
    announce(f"tree attention {dtype} D={D}: NaN and infinities in hidden nodes")
    N = 24
    c = Case(11, dtype, [70, 3], N, 2, G, D, 16)
    _, mask = random_tree(c.rng, 2, N)
    for b, node, what in ((0, 5, np.nan), (0, 9, np.inf), (1, 2, -np.inf), (1, 7, np.nan)):
        page, slot = O.positions(c.table[b], 16, c.pages, c.lens[b] + node,
                                 c.lens[b] + node + 1)[0][1:]
        c.v[page, slot, 0, ::3] = what
        c.k[page, slot, 1, 2] = what
    got, ref = check(svm, c, mask)
    assert np.isnan(ref["out"]).any() and np.isinf(ref["out"]).any()
    assert np.isfinite(ref["out"]).mean() > 0.3


def test_values_behind_the_table(svm):
    announce("tree attention: bad pages, lengths out of range, a table too short")
    for dtype in ("f32", "bf16"):
        c = Case(5, dtype, [100, 60, 30, 90], 6, 2, 2, 64, 16)
        cache_rows = c.table.copy()
        c.table[0, 2] = -1              # a missing page in the middle
        c.table[0, 4] = c.pages         # one past the last
        c.table[1, 0] = -2 ** 31
        c.table[1, 1] = 2 ** 31 - 1
        c.table[2, :] = -5              # no page at all
        check(svm, c)
        c.table = cache_rows
        c.lens = np.array([-7, 2 ** 31 - 1, -2 ** 31, c.width * 16 - 3], dtype=np.int32)
        c.table = np.where(c.table < 0, cache_rows[0, 0], c.table)
        c.k = np.nan_to_num(c.k)        # the whole table counts as committed now
        c.v = np.nan_to_num(c.v)
        check(svm, c)
        nodes = np.array([-3, 2, 10 ** 9, 6], dtype=np.int32)
        check(svm, c, None, nodes)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_layouts(svm, dtype):
    announce(f"tree attention {dtype}: heads before slots, keys and values interleaved, layers, "
             "queries inside a fused projection")
    c = Case(21, dtype, [50, 130, 7], 10, 2, 3, 64, 16)
    _, mask = random_tree(c.rng, 3, 10)
    ref = O.tree_attention(c.q, c.k, c.v, c.table, c.lens, mask)
    k, v = c.dev(c.k), c.dev(c.v)
    # [pages, heads, slots, D]
    kh = k.transpose(1, 2).contiguous().transpose(1, 2)
    vh = v.transpose(1, 2).contiguous().transpose(1, 2)
    # [layers, pages, 2, slots, heads, D], the values behind the keys of each page; layer 1 of 3
    both = torch.full((3, c.pages, 2, 16, 2, 64), float("nan"), dtype=DTYPES[dtype],
                      device="cuda")
    both[1, :, 0], both[1, :, 1] = k, v
    # [pages, slots, heads, D + 32]: padded rows
    wide = torch.zeros((2, c.pages, 16, 2, 96), dtype=DTYPES[dtype], device="cuda")
    wide[0, ..., :64], wide[1, ..., :64] = k, v
    qkv = torch.randn((3, 10, 6 + 2 + 2, 64), device="cuda").to(DTYPES[dtype])
    qkv[:, :, :6] = c.dev(c.q)
    qt = c.dev(c.q).permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3)
    t, n = ints(c.table), ints(c.lens)
    for cache, layer in ((svm.PagedCache(kh, vh, t, n), 0),
                         (svm.PagedCache(both[:, :, 0], both[:, :, 1], t, n), 1),
                         (svm.PagedCache(wide[0, ..., :64], wide[1, ..., :64], t, n), 0)):
        for q in (c.dev(c.q), qkv[:, :, :6], qt):
            check_attention(run(svm, c, mask, cache=cache, q=q, layer=layer), ref, dtype, 64)


def test_many_sequences(svm):
    announce("tree attention: 700 short sequences, more than one prefix-sum chunk a thread")
    rng = np.random.default_rng(1)
    c = Case(8, "bf16", rng.integers(0, 40, 700).tolist(), 2, 1, 2, 64, 8)
    check(svm, c, None, rng.integers(0, 3, 700).astype(np.int32))


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 64), ("bf16", 96), ("bf16", 128),
                                     ("f32", 96), ("f32", 128), ("f32", 256), ("bf16", 256)])
def test_long_and_ragged(svm, dtype, D):
    announce(f"tree attention {dtype} D={D}: one long sequence and a ragged batch (parts joined)")
    for lens, N, G in (([9000], 3, 2), ([5000, 0, 1, 700, 64], 12, 4), ([2500, 2501], 40, 4)):
        c = Case(sum(lens), dtype, lens, N, 1, G, D, 16)
        _, mask = random_tree(c.rng, len(lens), N)
        a, _ = check(svm, c, mask)
        b = run(svm, c, mask)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_scale_and_outputs(svm):
    announce("tree attention: scale, preallocated outputs, no lse")
    c = Case(2, "bf16", [300, 20], 4, 2, 2, 128, 32)
    check(svm, c, scale=1.0)    # scores of several hundred: weights of one and zero
    check(svm, c, scale=1e-6)   # all weights alike
    out = {"out": torch.full((2, 4, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")}
    got = run(svm, c, want_lse=False, out=out)
    assert got["out"] is out["out"] and "lse" not in got
    ref = O.tree_attention(c.q, c.k, c.v, c.table, c.lens)
    check_attention(got, ref, "bf16", 128)


def test_offsets_beyond_32_bits(svm):
    announce("tree attention, append and commit: rows more than 2^32 bytes into the cache")
    D, Hkv, page = 128, 8, 64
    pages = (2 ** 32 + 2 ** 28) // (2 * page * Hkv * D * 2)  # 4.25 GiB of keys and values
    big = torch.empty((pages, 2, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    c = Case(4, "bf16", [150, 100], 5, Hkv, 1, D, page)
    place = torch.arange(c.pages, device="cuda") * ((pages - 1) // (c.pages - 1))
    big[place, 0], big[place, 1] = c.dev(c.k), c.dev(c.v)
    table = np.where(c.table >= 0, place.cpu().numpy()[np.maximum(c.table, 0)], -1)
    cache = svm.PagedCache(big[:, 0], big[:, 1], ints(table.astype(np.int32)), ints(c.lens))
    got = run(svm, c, cache=cache)
    ref = O.tree_attention(c.q, c.k, c.v, c.table, c.lens)
    check_attention(got, ref, "bf16", D)
    new = torch.randn((2, 5, Hkv, D), device="cuda").to(torch.bfloat16)
    svm.spec_cache_append(new, -new, cache)
    parent = torch.tensor([[-1, 0, 0, 1, 2]] * 2, dtype=torch.int32, device="cuda")
    last = torch.tensor([4, 3], dtype=torch.int32, device="cuda")
    lens = svm.spec_cache_commit(cache, last, parent=parent)
    assert lens.tolist() == [153, 103]
    for b, path in ((0, [0, 2, 4]), (1, [0, 1, 3])):
        for d, node in enumerate(path):
            x = int(c.lens[b]) + d
            row = big[int(table[b, x // page]), :, x % page]
            assert torch.equal(row[0], new[b, node]) and torch.equal(row[1], -new[b, node])


def test_graph_replays(svm):
    announce("tree attention captured once, replayed with other lengths, masks and values")
    B, N = 6, 16
    c = Case(30, "bf16", [700] * B, N, 2, 4, 128, 16)
    cache = c.cache(svm)
    static = dict(q=c.dev(c.q), mask=ints(random_tree(c.rng, B, N)[1]),
                  nodes=ints(np.full(B, N, dtype=np.int32)))

    def call(out=None):
        return svm.spec_tree_attention(static["q"], cache, mask=static["mask"],
                                       num_nodes=static["nodes"], want_lse=True, out=out)
    out = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for rep in range(4):
        c.lens = c.rng.integers(0, 701, B).astype(np.int32)
        mask = random_tree(c.rng, B, N)[1]
        nodes = c.rng.integers(0, N + 1, B).astype(np.int32)
        c.q = c.rounded(c.rng.standard_normal(c.q.shape))
        cache.seq_lens.copy_(ints(c.lens))
        static["mask"].copy_(ints(mask))
        static["nodes"].copy_(ints(nodes))
        static["q"].copy_(c.dev(c.q))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        (torch.randn(512, 512, device="cuda") @ torch.randn(512, 512, device="cuda")).sum().item()
        eager = call()
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k], eager[k]), (rep, k)
        ref = O.tree_attention(c.q, c.k, c.v, c.table, c.lens, mask, nodes)
        check_attention(got, ref, "bf16", 128)


@pytest.mark.parametrize("dtype,N,Hkv,G,D,lens", [
    ("bf16", 5, 1, 1, 128, [14304, 9]), ("f32", 25, 1, 4, 64, [12775]), ("bf16", 1, 2, 7, 256, [9000]),
    ("bf16", 3, 3, 5, 96, [17000]), ("f32", 2, 1, 5, 128, [6001, 0, 4000]), ("f32", 9, 2, 1, 256, [5000])])
def test_groups_of_many_parts(svm, dtype, N, Hkv, G, D, lens):
    announce(f"few rows over long contexts, {dtype} N={N} Hkv={Hkv} G={G} D={D} lens={lens}")
    c = Case(N + D, dtype, lens, N, Hkv, G, D, 24)
    mask = random_tree(c.rng, len(lens), N)[1]
    nodes = np.full(len(lens), N, dtype=np.int32)
    nodes[-1] = N - N // 3
    got = svm.spec_tree_attention(c.dev(c.q), c.cache(svm), mask=ints(mask), num_nodes=ints(nodes),
                                  want_lse=True)
    ref = O.tree_attention(c.q, c.k, c.v, c.table, c.lens, mask, nodes)
    check_attention(got, ref, dtype, D)


def test_two_graphs_at_once(svm):
    announce("two graphs captured one after the other, replayed side by side on two streams")
    cs = [Case(s, "bf16", [20000, 9000, 14000], 8, 2, 4, 128, 16) for s in (42, 43)]
    caches = [c.cache(svm) for c in cs]
    qs = [c.dev(c.q) for c in cs]
    want = [svm.spec_tree_attention(q, k)["out"].clone() for q, k in zip(qs, caches)]
    outs = [dict(out=torch.empty_like(q)) for q in qs]
    torch.cuda.synchronize()
    graphs = []
    for q, k, out in zip(qs, caches, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(8):
                svm.spec_tree_attention(q, k, out=out)
    streams = [torch.cuda.Stream() for _ in graphs]
    for rep in range(5):
        for out in outs:
            out["out"].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out["out"], w), rep


def test_two_streams_at_once(svm):
    announce("tree attention on two streams at once, and on a stream= argument")
    cs = [Case(s, "bf16", [3000, 100, 900], 8, 2, 4, 128, 16) for s in (40, 41)]
    caches = [c.cache(svm) for c in cs]
    qs = [c.dev(c.q) for c in cs]
    want = [svm.spec_tree_attention(q, k)["out"].clone() for q, k in zip(qs, caches)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for q, k, s in zip(qs, caches, streams):
            with torch.cuda.stream(s):
                got.append(svm.spec_tree_attention(q, k)["out"])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    got = [svm.spec_tree_attention(q, k, stream=s)["out"]
           for q, k, s in zip(qs, caches, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
