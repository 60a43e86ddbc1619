"""spec_tree_attention where a worker's part of a group runs over many key tiles, as in every long
batch: each tile shape, cut by the lengths into parts with 0, 1, 2 and 3 fixed pieces a group,
against float64.  How many tiles a worker gets is worked out from the workspace and asserted."""

import numpy as np
import pytest
import torch

import attention_reference as R
from cache_cases import announce, check_attention

pytestmark = pytest.mark.gpu

BN = 64  # keys of a tile

@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    return m


def workers_of(svm, dtype, seqs, N, Hkv, G, D, MT, page, width):
    """Workers that share the tiles, from the size of the workspace that holds two parts (MT rows
    of D sums, a maximum and a total, fp32) and a note of 16 bytes of each."""
    t = torch.empty((1, page, Hkv, D), dtype=R.DTYPES[dtype], device="cuda")
    cache = svm.PagedCache(t, t, torch.zeros((seqs, width), dtype=torch.int32, device="cuda"),
                           torch.zeros(seqs, dtype=torch.int32, device="cuda"))
    size = cache._attention_workspace(N, Hkv * G)
    w = round(size / (2 * MT * (4 * D + 8) + 16))
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    assert size == up(2 * w * MT * D * 4) + up(2 * w * MT * 8) + up(16 * w), (size, w)
    return w


def pieces(lens, nodes, N, Hkv, G, MT):
    tiles = np.maximum(1, -(-(np.asarray(lens) + nodes) // BN))
    live = -(-np.asarray(nodes) * G // MT)
    return int((Hkv * (live * tiles + (-(-N * G // MT) - live))).sum())


def check_parts(svm, dtype, D, MT, N, Hkv, G, each, tree, page=16, B=4, seed=0, dead=False):
    """B ragged sequences that give each worker about `each` tiles."""
    width = (1 << 21 if B <= 16 else 1 << 14) // page  # keys that the table has room for
    W = workers_of(svm, dtype, B, N, Hkv, G, D, MT, page, width)
    nodes = np.array([N - (3 * b) % (N // 4 + 1) for b in range(B)], dtype=np.int32)
    if dead:
        nodes[1] = 0
    share = np.array([0.41, 0.02, 0.34, 0.23]) if B == 4 else np.linspace(0.5, 1.5, B) / B
    tokens = (each + 0.5) * W * BN / (Hkv * (share * -(-nodes * G // MT)).sum())
    lens = np.maximum(1, (tokens * share).astype(int) - N)
    per = pieces(lens, nodes, N, Hkv, G, MT) // W
    announce(f"{dtype} D={D} rows {N * G} (tiles of {MT}) kv heads {Hkv} lens "
             f"{lens.min()}..{lens.max()} {'tree' if tree else 'chain'}: {per} tiles a worker of {W}")
    lo, hi = next(r for r in ((24, 10 ** 9), (16, 23), (8, 15), (1, 7)) if each >= r[0])
    assert lo <= per <= hi
    c = R.Batch(seed + D + N + each, dtype, lens, N, Hkv, G, D, page, width)
    # pages that are missing, one of them where a tile of the longest sequence begins
    c.table[0, 1280 // page] = -1
    c.table[0, int(lens[0]) // (2 * page)] = c.pages
    c.table[2, int(lens[2]) // page - 1] = -7
    if N > 1:  # values and a key that some rows must not meet
        for b, node, what in ((0, N - 2, np.inf), (2, N // 2, np.nan), (3, N - 1, -np.inf)):
            at = int(c.slots(b, int(lens[b]) + node, int(lens[b]) + node + 1))
            assert at >= 0
            c.v.view(-1, Hkv, D)[at, 0, ::5] = what
        at = int(c.slots(3, int(lens[3]) + N // 2, int(lens[3]) + N // 2 + 1))
        c.k.view(-1, Hkv, D)[at, Hkv - 1, 7] = np.nan
    mask = R.tree_masks(c.rng, B, N) if tree else None
    got = svm.spec_tree_attention(c.q, c.cache(svm), mask=mask,
                                  num_nodes=torch.from_numpy(nodes).cuda(), want_lse=True)
    torch.cuda.synchronize()
    ref = R.attention(c, mask, nodes)
    check_attention(got, ref, dtype, D)
    assert np.isfinite(ref["out"]).mean() > 0.4
    again = svm.spec_tree_attention(c.q, c.cache(svm), mask=mask,
                                    num_nodes=torch.from_numpy(nodes).cuda(), want_lse=True)
    for key in got:  # the same bits (NaN too)
        assert torch.equal(got[key].view(torch.uint8), again[key].view(torch.uint8))


# dtype, columns, rows of a tile, nodes, kv heads, query heads a kv head: every tile shape
SHAPES = [("bf16", 64, 32, 6, 2, 5), ("bf16", 64, 64, 16, 2, 4), ("bf16", 64, 128, 40, 2, 3),
          ("bf16", 64, 256, 41, 2, 4), ("bf16", 96, 64, 1, 2, 8), ("bf16", 96, 128, 25, 2, 4),
          ("bf16", 128, 64, 1, 4, 4), ("bf16", 128, 128, 16, 2, 8), ("bf16", 128, 256, 64, 2, 4),
          ("bf16", 256, 32, 1, 2, 8), ("bf16", 256, 64, 12, 2, 4), ("bf16", 256, 128, 24, 2, 4),
          ("f32", 64, 32, 5, 3, 2), ("f32", 64, 64, 12, 2, 4), ("f32", 64, 128, 30, 2, 3),
          ("f32", 96, 32, 1, 2, 5), ("f32", 96, 64, 20, 2, 3), ("f32", 96, 128, 24, 2, 4),
          ("f32", 128, 32, 8, 2, 4), ("f32", 128, 64, 15, 2, 4), ("f32", 128, 128, 50, 2, 2),
          ("f32", 256, 64, 9, 2, 2)]


@pytest.mark.parametrize("dtype,D,MT,N,Hkv,G", SHAPES)
@pytest.mark.parametrize("each,tree", [(27, True), (9, False)])
def test_many_tiles_a_part(svm, dtype, D, MT, N, Hkv, G, each, tree):
    check_parts(svm, dtype, D, MT, N, Hkv, G, each, tree)


@pytest.mark.parametrize("dtype,D,MT,N,Hkv,G", SHAPES)
def test_parts_of_some_tiles(svm, dtype, D, MT, N, Hkv, G):
    check_parts(svm, dtype, D, MT, N, Hkv, G, 18, True, page=24, dead=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("each", [3, 5, 12, 18, 40])
@pytest.mark.parametrize("tree", [True, False])
def test_four_tiles_in_flight(svm, D, each, tree):
    check_parts(svm, "bf16", D, 256, 50, 2, 4, each, tree, page=64, seed=1)


@pytest.mark.parametrize("dtype,D,MT,N,G", [("bf16", 128, 256, 700, 2), ("bf16", 64, 256, 400, 3),
                                            ("bf16", 96, 128, 500, 1), ("bf16", 256, 128, 300, 2),
                                            ("f32", 64, 128, 300, 2), ("f32", 128, 128, 260, 1),
                                            ("f32", 256, 64, 200, 1)])
@pytest.mark.parametrize("each,tree", [(26, False), (10, False), (26, True)])
def test_many_rows_tiles(svm, dtype, D, MT, N, G, each, tree):
    check_parts(svm, dtype, D, MT, N, 2, G, each, tree, B=16, seed=2, dead=True)


@pytest.mark.parametrize("dtype,D,MT", [("bf16", 128, 64), ("f32", 64, 32)])
def test_more_sequences_than_lds_keeps(svm, dtype, D, MT):
    check_parts(svm, dtype, D, MT, 2, 2, 2, 28, True, B=600, seed=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_comparison_notices_a_tile(svm, dtype):
    announce(f"{dtype}: outputs over all keys do not pass for those with 64 keys fewer")
    c = R.Batch(9, dtype, [20000, 9000], 64, 2, 2, 128, 16, 1 << 12)
    got = svm.spec_tree_attention(c.q, c.cache(svm), want_lse=True)
    check_attention(got, R.attention(c), dtype, 128)
    for b, tile in ((0, 0), (0, 77), (0, 150), (0, 311), (1, 5), (1, 139)):
        table = c.table.copy()
        c.table[b, 4 * tile:4 * tile + 4] = -1
        with pytest.raises(AssertionError):
            check_attention(got, R.attention(c), dtype, 128)
        c.table = table
