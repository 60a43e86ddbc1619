"""Inputs and error bounds shared by the tests of the paged-cache operators."""

import numpy as np
import torch

import oracle.paged_cache_oracle as O

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
F32_HALF_STEP = 2.0 ** -24
BF16_HALF_STEP = 2.0 ** -8


def announce(msg):
    print(f"\n[case] {msg}", flush=True)


def random_tree(rng, B, N):
    """Parents [B, N] (-1 for the root) and ancestor masks [B, N, N] of random trees."""
    parent = np.full((B, N), -1, dtype=np.int32)
    mask = np.zeros((B, N, N), dtype=np.uint8)
    for b in range(B):
        for i in range(N):
            if i:
                parent[b, i] = rng.integers(0, i)
                mask[b, i] = mask[b, parent[b, i]]
            mask[b, i, i] = 1
    return parent, mask


class Case:
    """A one-layer cache in host arrays (float64 values that the dtype holds exactly)."""

    def __init__(self, seed, dtype, lens, N, Hkv, G, D, page_size, spare=2, width=None,
                 garbage=float("nan")):
        rng = np.random.default_rng(seed)
        self.rng, self.dtype, self.D = rng, dtype, D
        self.lens = np.array(lens, dtype=np.int32)
        B = len(lens)
        held = [-(-(max(0, n) + N) // page_size) for n in lens]
        self.width = width or max(held)
        self.pages = sum(held) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((B, self.width), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(held):
            n = min(n, self.width)
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.pages, page_size, Hkv, D)
        # every slot that holds no key or value of a sequence is garbage
        self.k, self.v = np.full(shape, garbage), np.full(shape, garbage)
        for b in range(B):
            for _, p, s in O.positions(self.table[b], page_size, self.pages, 0,
                                       max(0, int(lens[b])) + N):
                self.k[p, s] = self.rounded(rng.standard_normal((Hkv, D)))
                self.v[p, s] = self.rounded(rng.standard_normal((Hkv, D)))
        self.q = self.rounded(1.5 * rng.standard_normal((B, N, Hkv * G, D)))

    def rounded(self, x):
        return torch.from_numpy(np.asarray(x)).to(DTYPES[self.dtype]).double().numpy()

    def dev(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(DTYPES[self.dtype]).cuda()

    def cache(self, sv, **kw):
        return sv.PagedCache(self.dev(self.k), self.dev(self.v), ints(self.table),
                             ints(self.lens), **kw)


def ints(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def check_attention(got, ref, dtype, D, nodes=None):
    """out and lse against the oracle, element by element.

    With u = 2^-24, a score is a product sum of D terms and a scaling: off by at most
    e = (D + 4) u reach (reach = scale * sum |q k|, rounded inputs being exact), the exponential
    by 2 steps on top, so a weight by (2 e + 8 u) relative to the row's largest reach; sums over
    n keys add (n + 8) u, merged partial sums included.  Hence |out - exact| <= absolute *
    (2 e + (2 n + 24) u) with absolute = sum weight |v|; bf16 rounds each weight (half a step,
    2^-8 of absolute) and the result (2^-8 of its size).  The logarithm of the sum is off by
    e + (n + 24) u, and its own rounding adds 4 u (1 + |lse| + reach)."""
    out = got["out"].double().cpu().numpy()
    u = F32_HALF_STEP
    n = ref["count"][:, :, None].astype(np.float64)
    e = (D + 4) * u * ref["reach"]
    rel = 2 * e + (2 * n + 24) * u
    tol = ref["absolute"] * rel[..., None] + 1e-30
    if dtype == "bf16":
        tol = tol + (ref["absolute"] + np.abs(ref["out"])) * BF16_HALF_STEP * 1.01
    fine = np.isfinite(ref["out"])
    np.testing.assert_array_equal(np.isfinite(out), fine)
    np.testing.assert_array_equal(np.isnan(out), np.isnan(ref["out"]))
    both = ~fine & ~np.isnan(out)
    np.testing.assert_array_equal(out[both], ref["out"][both])
    with np.errstate(invalid="ignore"):
        bad = fine & (np.abs(np.where(fine, out - ref["out"], 0.0)) > tol)
    assert not bad.any(), (np.argwhere(bad)[:4], out[bad][:4], ref["out"][bad][:4], tol[bad][:4])
    empty = ref["count"] == 0
    assert (out[empty] == 0).all()
    if "lse" in got:
        lse = got["lse"].double().cpu().numpy()
        has = np.isfinite(ref["lse"])
        same = ~has & ~np.isnan(ref["lse"])
        np.testing.assert_array_equal(lse[same], ref["lse"][same])
        np.testing.assert_array_equal(np.isnan(lse), np.isnan(ref["lse"]))
        t = e + (n + 24) * u + 4 * u * (1 + np.abs(np.where(has, ref["lse"], 0)) + ref["reach"])
        with np.errstate(invalid="ignore"):
            bad = has & (np.abs(np.where(has, lse - ref["lse"], 0.0)) > t)
        assert not bad.any(), (np.argwhere(bad)[:4], lse[bad][:4], ref["lse"][bad][:4])
