"""CPU-side refusals of the paged-cache entry points: each bad argument returns its status before
anything touches a GPU, and the binding names what is wrong with a tensor."""

import ctypes
from types import SimpleNamespace

import pytest
import torch

INVALID, DTYPE, WS = 1, 2, 3
DUMMY = 1 << 20  # stands for device memory; never dereferenced


@pytest.fixture(scope="module")
def svl():
    from speculative_sampling_verification_amd import _lib
    return _lib


def cache(svl, **over):
    a = dict(k=DUMMY, v=2 * DUMMY, dtype=1, layers=2, pages=10, page_size=16, kv_heads=2,
             head_dim=64, layer_stride=10 * 16 * 128, page_stride=16 * 128, token_stride=128,
             head_stride=64, seqs=3, table_width=5, page_table=DUMMY, seq_lens=DUMMY,
             seq_pages=DUMMY, refcount=DUMMY)
    a.update(over)
    return svl.SVCache(*a.values())


def attend(svl, c, q=DUMMY, strides=None, N=4, heads=4, layer=0, scale=0.125, out=DUMMY, ws=DUMMY,
           ws_bytes=0):
    s = None if strides is None else (ctypes.c_int64 * 3)(*strides)
    return svl.lib().spec_tree_attention(q, s, N, heads, ctypes.byref(c), layer, None, None, scale,
                                         out, None, ws, ws_bytes, None)


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(page_table=None), INVALID),
    (dict(seq_lens=None), INVALID), (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE),
    (dict(layers=0), INVALID), (dict(pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(kv_heads=0), INVALID), (dict(kv_heads=1025), INVALID), (dict(head_dim=0), INVALID),
    (dict(head_dim=60), INVALID), (dict(head_dim=520), INVALID), (dict(seqs=0), INVALID),
    (dict(seqs=8193), INVALID), (dict(table_width=0), INVALID),
    (dict(table_width=2 ** 30), INVALID), (dict(table_width=2 ** 18, page_size=2 ** 13), INVALID),
    (dict(k=DUMMY + 8), INVALID), (dict(v=DUMMY + 2), INVALID), (dict(seq_lens=DUMMY + 2), INVALID),
    # rows that overlap, start off 16 bytes, or run backwards
    (dict(token_stride=64), INVALID), (dict(head_stride=32), INVALID),
    (dict(page_stride=15 * 128), INVALID), (dict(layer_stride=0), INVALID),
    (dict(token_stride=132), INVALID), (dict(head_stride=-64), INVALID),
    (dict(layer_stride=2 ** 62), INVALID),
]


@pytest.mark.parametrize("over,status", BAD_CACHES, ids=[str(b[0]) for b in BAD_CACHES])
def test_every_entry_point_refuses_a_bad_cache(svl, over, status):
    L, c = svl.lib(), cache(svl, **over)
    r = ctypes.byref(c)
    assert attend(svl, c, ws_bytes=1 << 40) == status
    assert L.spec_tree_attention_workspace_size(r, 4, 4) == 0
    assert L.spec_cache_append(DUMMY, DUMMY, None, 4, r, 0, None, None) == status
    assert L.spec_cache_commit(r, DUMMY, DUMMY, 4, 3 * DUMMY, None) == status
    assert L.spec_cache_resize(r, DUMMY, None, DUMMY, None) == status
    assert L.spec_cache_fork(r, DUMMY, DUMMY, 2, DUMMY, None) == status


def test_layouts_whose_rows_lie_apart_are_taken(svl):
    # heads before slots; one page, layer or head whose stride does not matter
    for over in (dict(head_stride=16 * 64, token_stride=64),
                 dict(pages=1, page_stride=0), dict(layers=1, layer_stride=0),
                 dict(kv_heads=1, head_stride=0, token_stride=64),
                 dict(layer_stride=128 * 16, page_stride=2 * 128 * 16)):
        assert attend(svl, cache(svl, **over), heads=2 * cache(svl, **over).kv_heads) == WS


def test_attention_arguments(svl):
    c = cache(svl)
    assert attend(svl, c) == WS
    need = svl.lib().spec_tree_attention_workspace_size(ctypes.byref(c), 4, 4)
    assert need > 0 and attend(svl, c, ws_bytes=need - 1) == WS
    assert attend(svl, c, ws=None, ws_bytes=need) == WS
    assert attend(svl, c, ws=DUMMY + 4, ws_bytes=need) == INVALID
    for bad in (dict(q=None), dict(out=None), dict(N=0), dict(N=2049), dict(heads=0),
                dict(heads=3), dict(layer=-1), dict(layer=2), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(q=DUMMY + 4),
                dict(out=DUMMY + 2), dict(strides=(256, 64, 4)), dict(strides=(-256, 64, 64))):
        assert attend(svl, c, ws_bytes=1 << 40, **bad) == INVALID, bad
    # head sizes that the cache holds but attention does not take
    for dim in (32, 80, 512):
        d = cache(svl, head_dim=dim, head_stride=dim, token_stride=2 * dim, page_stride=32 * dim,
                  layer_stride=320 * dim)
        assert attend(svl, d, ws_bytes=1 << 40) == INVALID
        assert svl.lib().spec_tree_attention_workspace_size(ctypes.byref(d), 4, 4) == 0
    assert svl.lib().spec_tree_attention_workspace_size(None, 4, 4) == 0


def test_move_and_pool_arguments(svl):
    L, c = svl.lib(), cache(svl)
    r = ctypes.byref(c)
    for a in ((None, DUMMY, None, 4, r, 0, None), (DUMMY, None, None, 4, r, 0, None),
              (DUMMY, DUMMY, None, 0, r, 0, None), (DUMMY, DUMMY, None, 2049, r, 0, None),
              (DUMMY, DUMMY, None, 4, r, 2, None), (DUMMY + 8, DUMMY, None, 4, r, 0, None),
              (DUMMY, DUMMY, (ctypes.c_int64 * 3)(256, 128, 4), 4, r, 0, None),
              (DUMMY, DUMMY, None, 4, None, 0, None)):
        assert L.spec_cache_append(*a, None) == INVALID, a
    for a in ((None, DUMMY, DUMMY, 4, 3 * DUMMY), (r, None, DUMMY, 4, 3 * DUMMY),
              (r, DUMMY, DUMMY, 0, 3 * DUMMY), (r, DUMMY, DUMMY, 2049, 3 * DUMMY),
              (r, DUMMY, DUMMY, 4, None),
              # new lengths over the old ones, wholly or in part
              (r, DUMMY, DUMMY, 4, DUMMY), (r, DUMMY, DUMMY, 4, DUMMY + 8),
              (r, DUMMY, DUMMY, 4, DUMMY - 8)):
        assert L.spec_cache_commit(*a, None) == INVALID, a
    for a in ((r, None, None, DUMMY), (r, DUMMY, None, None), (None, DUMMY, None, DUMMY),
              (r, DUMMY + 2, None, DUMMY)):
        assert L.spec_cache_resize(*a, None) == INVALID, a
    for a in ((r, None, DUMMY, 2, DUMMY), (r, DUMMY, None, 2, DUMMY), (r, DUMMY, DUMMY, 2, None),
              (r, DUMMY, DUMMY, -1, DUMMY), (r, DUMMY, DUMMY, 4, DUMMY)):
        assert L.spec_cache_fork(*a, None) == INVALID, a
    assert L.spec_cache_fork(r, None, None, 0, None, None) == 0  # nothing to do
    for over in (dict(seq_pages=None), dict(refcount=None)):
        p = cache(svl, **over)
        assert L.spec_cache_resize(ctypes.byref(p), DUMMY, None, DUMMY, None) == INVALID
        assert L.spec_cache_fork(ctypes.byref(p), DUMMY, DUMMY, 2, DUMMY, None) == INVALID
    same = cache(svl, v=DUMMY)  # keys and values in one place: nothing is written there
    assert L.spec_cache_append(DUMMY, DUMMY, None, 4, ctypes.byref(same), 0, None, None) == INVALID
    assert L.spec_cache_commit(ctypes.byref(same), DUMMY, DUMMY, 4, 3 * DUMMY, None) == INVALID
    assert L.spec_cache_fork(ctypes.byref(same), DUMMY, DUMMY, 2, DUMMY, None) == INVALID


def test_arrays_of_a_call_share_no_memory(svl):
    L, c = svl.lib(), cache(svl, seq_lens=16 * DUMMY, seq_pages=17 * DUMMY, refcount=18 * DUMMY,
                            page_table=19 * DUMMY)
    r, a, b, o = ctypes.byref(c), 24 * DUMMY, 25 * DUMMY, 26 * DUMMY
    for out in (a, a + 8, a - 8, b, b + 44, 16 * DUMMY + 8, 19 * DUMMY + 56):
        assert L.spec_cache_commit(r, a, b, 4, out, None) == INVALID, out
    state = (16 * DUMMY + 8, 17 * DUMMY - 8, 18 * DUMMY + 36, 19 * DUMMY + 56)
    for x in state:
        for args in ((x, None, o), (a, x, o), (a, b, x)):
            assert L.spec_cache_resize(r, *args, None) == INVALID, (x, args)
        for args in ((x, b, o), (a, x, o), (a, b, x)):
            assert L.spec_cache_fork(r, args[0], args[1], 3, args[2], None) == INVALID, (x, args)
    # seq_lens itself may be wanted, not returned to
    assert L.spec_cache_resize(r, 16 * DUMMY, None, 16 * DUMMY, None) == INVALID
    for x in (a + 8, b - 8):
        assert L.spec_cache_resize(r, a, b, x, None) == INVALID
        assert L.spec_cache_fork(r, a, b, 3, x, None) == INVALID
    assert attend(svl, c, q=a, out=a, ws=o, ws_bytes=1 << 40) == INVALID
    assert attend(svl, cache(svl, layers=8193), ws_bytes=1 << 40) == INVALID


def test_keys_and_values_share_no_row(svl):
    L = svl.lib()
    row, page = 128, 16 * 128  # a token's elements, a page's
    # k and v as neighbouring halves of a row, a token, a page, a layer: taken (the refusal is
    # that of the new rows' address)
    for over in (dict(head_stride=128, token_stride=256, page_stride=2 * page, v=DUMMY + 128),
                 dict(token_stride=2 * row, page_stride=2 * page, v=DUMMY + 2 * row),
                 dict(page_stride=2 * page, v=DUMMY + 2 * page),
                 dict(layer_stride=20 * page, v=DUMMY + 2 * 10 * page)):
        over.setdefault("layer_stride", 20 * page)
        for c in (cache(svl, **over), cache(svl, **{**over, "k": over["v"], "v": DUMMY})):
            assert L.spec_cache_append(DUMMY, DUMMY, None, 0, ctypes.byref(c), 0, None, None) \
                == INVALID
            assert L.spec_cache_fork(ctypes.byref(c), None, None, 0, None, None) == 0
    for v in (DUMMY + 16, DUMMY + 2 * row, DUMMY + 2 * page, DUMMY + 2 * 10 * page,
              DUMMY + 2 * 20 * page - 16):
        c = cache(svl, v=v)
        assert L.spec_cache_append(3 * DUMMY, 4 * DUMMY, None, 4, ctypes.byref(c), 0, None,
                                   None) == INVALID
        assert L.spec_cache_commit(ctypes.byref(c), DUMMY, DUMMY, 4, 3 * DUMMY, None) == INVALID
        assert L.spec_cache_fork(ctypes.byref(c), None, None, 0, None, None) == INVALID
    assert L.spec_cache_fork(ctypes.byref(cache(svl, v=DUMMY + 2 * 20 * page)), None, None, 0, None,
                             None) == 0


def test_binding_names_bad_tensors(svl):
    k = torch.zeros((2, 6, 4, 2, 64))
    table, lens = torch.zeros((3, 5), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    c = svl.PagedCache(k, k.clone(), table, lens)
    for bad in ((k, k[:, :, :, :, :32], table, lens), (k, k.bfloat16(), table, lens),
                (k[0, 0], k[0, 0], table, lens), (k, k, table.long(), lens), (k, k, table[0], lens),
                (k, k, table, lens[:2]), (k.double(), k.double(), table, lens),
                (k.transpose(3, 4), k.transpose(3, 4), table, lens),
                (k, k.transpose(2, 3).contiguous().transpose(2, 3), table, lens)):
        with pytest.raises((TypeError, ValueError)):
            svl.PagedCache(*bad)
    with pytest.raises((TypeError, ValueError)):
        svl.PagedCache(k, k, table, lens, refcount=torch.zeros(5, dtype=torch.int32))
    with pytest.raises((TypeError, ValueError)):
        svl.PagedCache(k, k, table, lens, seq_pages=lens.long())
    q = torch.zeros((3, 4, 4, 64))
    for bad in (q.bfloat16(), q[:2], q[..., :32], q[0], None):
        with pytest.raises((TypeError, ValueError)):
            svl.spec_tree_attention(bad, c)
    new = torch.zeros((3, 4, 2, 64))
    for pair in ((new, new[:, :3]), (new, q), (new.bfloat16(), new.bfloat16()),
                 (new, new.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            svl.spec_cache_append(*pair, c)
    i = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: svl.spec_cache_commit(c, i.long()), lambda: svl.spec_cache_commit(c, None),
                 lambda: svl.spec_cache_commit(c, i, parent=i),
                 lambda: svl.spec_cache_resize(c, i[:2]), lambda: svl.spec_cache_resize(c, 5),
                 lambda: svl.spec_cache_fork(c, i, i[:2]), lambda: svl.spec_cache_fork(c, i[None], i)):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_binding_refuses_other_devices(svl):
    """Every argument agrees, but the cache is in host memory: nothing may be launched on it."""
    k = torch.zeros((2, 6, 4, 2, 64))
    table, i = torch.zeros((3, 5), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    c = svl.PagedCache(k, k.clone(), table, i, seq_pages=i.clone(), refcount=torch.zeros(6, dtype=torch.int32))
    q, new, x, o = torch.zeros((3, 4, 4, 64)), torch.zeros((3, 4, 2, 64)), i.clone(), i.clone()
    other = SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    same = SimpleNamespace(cuda_stream=0, device=torch.device("cpu"))
    for stream in (None, other, same):
        for call in (lambda: svl.spec_tree_attention(q, c, out={"out": torch.empty_like(q)}, stream=stream),
                     lambda: svl.spec_cache_append(new, new.clone(), c, stream=stream),
                     lambda: svl.spec_cache_commit(c, x, num_nodes=4, out=o, stream=stream),
                     lambda: svl.spec_cache_resize(c, x, out=o, stream=stream),
                     lambda: svl.spec_cache_fork(c, x, x.clone(), out=o, stream=stream)):
            with pytest.raises(ValueError):
                call()
    for call in (lambda: svl.spec_cache_fork(c, [0], x), lambda: svl.spec_cache_commit(c, x, parent=[0])):
        with pytest.raises(TypeError):
            call()
