"""spec_cache_weigh over longer contexts and many rows, every tile shape, against the definition in
float64 on the device.  Every row has a key of its own among the committed tokens that carries most
of its weight, so that a key or a row left out, or taken twice, shows.  Error bound as for the short
cases: (scale sum |q k| (D + 8) + 4 |lse| + 4) u of every row's weight and (rows + 8) u of the sum,
u = 2^-24."""

import numpy as np
import pytest
import torch

from attention_reference import Batch
from cache_cases import F32_HALF_STEP, announce

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    return m


def reference(c, lse, seen, nodes, L):
    """(given, tolerance) [B, Hkv, L] float64."""
    B, N, Hq, D = c.q.shape
    G, scale, u = c.G, D ** -0.5, F32_HALF_STEP
    given = torch.zeros((B, c.Hkv, L), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(given)
    kf = c.k.reshape(-1, c.Hkv, D)
    for b in range(B):
        n, length = int(nodes[b]), min(int(c.lens[b]), L)
        at = c.slots(b, 0, length)
        there = at >= 0
        x = torch.arange(len(at), device="cuda")
        limit = torch.full((n,), length, device="cuda") if seen is None else seen[b, :n].long()
        see = (x[None, :] < limit[:, None]).repeat_interleave(G, 0) & there
        for h in range(c.Hkv):
            hq = slice(h * G, (h + 1) * G)
            q = c.q[b, :n, hq].double().reshape(n * G, D)
            s = lse[b, :n, hq].double().reshape(n * G, 1)
            kk = torch.where(there[:, None], kf[at.clamp(min=0), h].double(), 0.0).t().contiguous()
            w = torch.where(see & (s > -torch.inf), torch.exp(scale * (q @ kk) - s), 0.0)
            reach = scale * (q.abs() @ kk.abs())
            doubt = w * (reach * (D + 8) + 4 * torch.where(s > -torch.inf, s.abs(), 0.0) + 4)
            given[b, h, :length] = w.sum(0)
            tol[b, h, :length] = doubt.sum(0) * u * 1.01 + (n * G + 10) * u * w.sum(0)
    return given, tol


CASES = [  # dtype, lens, N, Hkv, G, D, page
    ("bf16", [5000, 70, 0, 1023], 1, 2, 4, 128, 16), ("bf16", [9001], 3, 1, 5, 64, 24),
    ("bf16", [3000, 511], 2, 3, 8, 96, 100), ("bf16", [2500, 64], 5, 2, 3, 256, 8),
    ("f32", [2500, 65], 4, 2, 4, 64, 16), ("f32", [1500], 1, 1, 16, 96, 5),
    ("f32", [1400, 31], 3, 2, 2, 128, 64), ("f32", [900, 17], 2, 1, 7, 256, 16),
    # more than 16 rows, up to 256, more
    ("bf16", [4100, 129, 0], 17, 2, 1, 128, 16), ("bf16", [2100, 255], 64, 1, 4, 128, 32),
    ("bf16", [1900, 600], 65, 2, 4, 128, 16), ("bf16", [2000], 100, 1, 3, 64, 16),
    ("bf16", [2000], 33, 1, 8, 64, 16), ("bf16", [1800, 90], 50, 1, 6, 96, 16),
    ("bf16", [1700], 10, 2, 5, 96, 8), ("bf16", [1300, 257], 70, 2, 5, 256, 16),
    ("f32", [1600, 40], 9, 2, 3, 64, 16), ("f32", [1500], 90, 1, 4, 64, 16),
    ("f32", [1200, 127], 45, 1, 7, 96, 16), ("f32", [1000], 32, 2, 2, 128, 16),
    ("f32", [700, 128], 33, 1, 5, 256, 16), ("bf16", [1500] * 9, 200, 1, 8, 128, 64)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_long(svm, case):
    dtype, lens, N, Hkv, G, D, page = case
    announce(f"weigh long {case}")
    width = -(-(max(lens) + N) // page)
    c = Batch(N + D, dtype, lens, N, Hkv, G, D, page, width)
    if max(lens) > 1000:  # a page that does not exist
        c.table[0, 900 // page] = c.pages
    B, L = len(lens), max(lens)
    cache = c.cache(svm)
    chain = svm.spec_tree_attention(c.q, cache, want_lse=True)["lse"]
    lse = torch.nan_to_num(chain, nan=0.0, neginf=-torch.inf)
    lse[0, N // 2] = -torch.inf
    full = np.full(B, N, dtype=np.int32)
    some = c.rng.integers(0, N + 1, B).astype(np.int32)
    # the last N committed tokens as the nodes; nodes that do not count; all at once
    own = torch.from_numpy(np.array(lens)[:, None] - N + 1 + np.arange(N)[None, :]).cuda()
    own[:, ::7] = 0
    for seen, nodes, decay in ((None, full, 1.0), (own.int(), some, 0.25)):
        start = torch.rand((1, B, Hkv, L), device="cuda")
        w = start.clone()
        svm.spec_cache_weigh(c.q, lse, cache, w, seen=seen, decay=decay,
                             num_nodes=torch.from_numpy(nodes).cuda())
        given, tol = reference(c, lse, seen, nodes, L)
        at = torch.arange(L, device="cuda")
        live = at[None, :] < torch.from_numpy(np.array(lens)).cuda()[:, None]
        want = torch.where(live[:, None], decay * start[0].double() + given, start[0].double())
        off = (w[0].double() - want).abs()
        assert (off <= tol + 2 * F32_HALF_STEP * want.abs() + 1e-30).all(), off.max()


def test_strided_queries(svm):
    announce("weigh: queries as a part of one product, sequences behind nodes")
    c = Batch(3, "bf16", [800, 300], 40, 2, 2, 64, 16, 60)
    cache = c.cache(svm)
    lse = svm.spec_tree_attention(c.q, cache, want_lse=True)["lse"]
    want = torch.zeros((1, 2, 2, 800), device="cuda")
    svm.spec_cache_weigh(c.q, lse, cache, want)
    part = torch.zeros((2, 40, 6, 64), dtype=torch.bfloat16, device="cuda")
    part[:, :, 1:5] = c.q
    behind = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    for q in (part[:, :, 1:5], behind):
        for n in (40, 7):  # both kernels
            w, ref = torch.zeros_like(want), torch.zeros_like(want)
            svm.spec_cache_weigh(q[:, :n], lse[:, :n].contiguous(), cache, w)
            svm.spec_cache_weigh(c.q[:, :n].contiguous(), lse[:, :n].contiguous(), cache, ref)
            assert torch.equal(w, ref) and (n < 40 or torch.equal(w, want))


def test_many_sequences(svm):
    announce("weigh: more sequences than a workgroup's threads, most of them short")
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 40, 700)
    lens[[3, 400]] = 900
    for N in (2, 20):
        c = Batch(N, "bf16", lens.tolist(), N, 1, 1, 64, 16, 60)
        cache = c.cache(svm)
        lse = svm.spec_tree_attention(c.q, cache, want_lse=True)["lse"]
        w = torch.zeros((1, 700, 1, 900), device="cuda")
        svm.spec_cache_weigh(c.q, lse, cache, w)
        given, tol = reference(c, lse, None, np.full(700, N), 900)
        assert ((w[0].double() - given).abs() <= tol + 1e-30).all()
