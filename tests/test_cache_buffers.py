"""CPU-side refusals of calls whose buffers share memory: what attention writes lies apart from all
that it reads, and a commit's lengths apart from the cache's books.  And of scales too large."""

import ctypes

import pytest

INVALID, WS = 1, 3
MB = 1 << 20
SEQS, N, HEADS, KV, D, PAGES, PAGE, LAYERS, WIDTH = 3, 4, 4, 2, 64, 10, 16, 2, 5
ROW = D * 2                                     # bytes, bf16
LAYER = PAGES * PAGE * KV * ROW
OUT, LSE = SEQS * N * HEADS * ROW, SEQS * N * HEADS * 4
AT = dict(k=64 * MB, v=128 * MB, table=1 * MB, lens=2 * MB, held=3 * MB, ref=4 * MB, q=5 * MB,
          mask=6 * MB, nodes=7 * MB, out=8 * MB, lse=9 * MB, ws=512 * MB)
SIZE = dict(k=LAYER, v=LAYER, table=4 * SEQS * WIDTH, lens=4 * SEQS, held=4 * SEQS, ref=4 * PAGES,
            q=OUT, mask=SEQS * N * N, nodes=4 * SEQS, out=OUT, lse=LSE)


@pytest.fixture(scope="module")
def svl():
    from speculative_sampling_verification_amd import _lib
    return _lib


def cache(svl, at):
    return svl.SVCache(at["k"], at["v"], 1, LAYERS, PAGES, PAGE, KV, D, PAGES * PAGE * KV * D,
                       PAGE * KV * D, KV * D, D, SEQS, WIDTH, at["table"], at["lens"], at["held"],
                       at["ref"])


def attend(svl, layer=0, strides=None, heads=HEADS, ws_bytes=None, scale=0.125, **moved):
    at = {**AT, **moved}
    c = cache(svl, at)
    need = svl.lib().spec_tree_attention_workspace_size(ctypes.byref(c), N, heads)
    assert need > 0
    s = None if strides is None else (ctypes.c_int64 * 3)(*strides)
    return svl.lib().spec_tree_attention(at["q"], s, N, heads, ctypes.byref(c), layer, at["mask"],
                                         at["nodes"], scale, at["out"], at["lse"], at["ws"],
                                         need if ws_bytes is None else ws_bytes, None), need


@pytest.mark.parametrize("name", [n for n in SIZE if n != "out"])
def test_out_apart_from_everything(svl, name):
    for where in (AT[name], AT[name] + SIZE[name] // 16 * 16 - 16, AT[name] - OUT + 16):
        assert attend(svl, out=where // 16 * 16)[0] == INVALID, where


@pytest.mark.parametrize("name", [n for n in SIZE if n != "lse"])
def test_lse_apart_from_everything(svl, name):
    for where in (AT[name], AT[name] + SIZE[name] // 4 * 4 - 4, AT[name] - LSE + 4):
        assert attend(svl, lse=where)[0] == INVALID, where


@pytest.mark.parametrize("name", list(SIZE))
def test_workspace_apart_from_everything(svl, name):
    need = attend(svl, ws_bytes=0)[1]
    for where in (AT[name] // 16 * 16, (AT[name] - need + 16) // 16 * 16):
        if where > 0:  # the workspace is larger than the low addresses here
            assert attend(svl, ws=where)[0] == INVALID, where


def test_the_layer_of_the_call_counts(svl):
    # the second layer's keys, and the gap behind a query's heads in a fused projection
    assert attend(svl, layer=1, out=AT["k"] + 2 * LAYER - 16)[0] == INVALID
    wide = (N * 2 * HEADS * D, 2 * HEADS * D, D)
    assert attend(svl, strides=wide, out=AT["q"] + 2 * OUT - HEADS * ROW - 16)[0] == INVALID
    assert attend(svl, strides=(0, 0, 0), out=AT["q"] + ROW - 16)[0] == INVALID
    # extents that no memory has
    huge = 2 ** 63 // 8 - 8
    assert attend(svl, strides=(huge, huge, huge))[0] == INVALID
    assert attend(svl, strides=(huge, huge, huge), ws_bytes=0)[0] == WS


def test_committed_lengths_apart_from_the_books(svl):
    c = cache(svl, AT)
    for name in ("lens", "table", "held", "ref"):
        for off in (0, SIZE[name] - 4, 4 - 4 * SEQS):
            assert svl.lib().spec_cache_commit(ctypes.byref(c), AT["q"], AT["mask"], N,
                                               AT[name] + off, None) == INVALID, (name, off)


def test_scales_whose_multiple_overflows(svl):
    # scores are multiplied by scale * log2(e) = 1.4427 scale: 3.4028e38 / 1.4427 = 2.3587e38
    for scale in (2.36e38, 3.4e38):
        assert attend(svl, scale=scale, ws_bytes=0)[0] == INVALID
    for scale in (2.358e38, 1e-38):
        assert attend(svl, scale=scale, ws_bytes=0)[0] == WS
