"""spec_tree_attention over long batches: inputs made on the device, and the definition in float64
there, one sequence and kv head at a time."""

import numpy as np
import torch

from cache_cases import DTYPES


class Batch:
    """A one-layer cache of B sequences of `lens` committed tokens and N nodes, and queries.

    Every row (node, query head) has a key of its own somewhere among the committed tokens that
    carries most of its weight, so that a key left out, or taken twice, shows in some row however
    long the sequence is.  Slots that hold no key or value are NaN."""

    def __init__(self, seed, dtype, lens, N, Hkv, G, D, page, width):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.rng = rng = np.random.default_rng(seed)
        self.dtype, self.N, self.Hkv, self.G, self.D, self.page = dtype, N, Hkv, G, D, page
        self.lens, self.width = np.array(lens, dtype=np.int32), width
        B = len(lens)
        held = [-(-(n + N) // page) for n in lens]
        self.pages = sum(held) + 2
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((B, width), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n
        normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.q = (1.5 * normal(B, N, Hkv * G, D)).to(DTYPES[dtype])
        k, v = (torch.full((self.pages * page, Hkv, D), float("nan"), dtype=DTYPES[dtype],
                           device="cuda") for _ in range(2))
        for b in range(B):
            at = self.slots(b, 0, lens[b] + N)
            k[at], v[at] = (normal(len(at), Hkv, D).to(k.dtype) for _ in range(2))
            if lens[b] < N * G:
                continue
            # scores of 12 or so among thousands of order 1
            for h in range(Hkv):
                rows = self.q[b, :, h * G:(h + 1) * G].reshape(N * G, D)
                where = torch.from_numpy(rng.permutation(int(lens[b]))[:N * G]).cuda()
                size = rows.double().square().sum(1, keepdim=True) * D ** -0.5
                k[at[where], h] = (rows.double() * (12.0 / size)).to(k.dtype)
        self.k, self.v = (x.view(self.pages, page, Hkv, D) for x in (k, v))

    def slots(self, b, first, last):
        """Rows of the flat cache of positions first .. last - 1; -1 where there is no page."""
        x = np.arange(first, min(last, self.width * self.page))
        p = self.table[b, x // self.page].astype(np.int64)
        s = np.where((p >= 0) & (p < self.pages), p * self.page + x % self.page, -1)
        return torch.from_numpy(s).cuda()

    def cache(self, sv):
        return sv.PagedCache(self.k, self.v, torch.from_numpy(self.table).cuda(),
                             torch.from_numpy(self.lens).cuda())


def tree_masks(rng, B, N):
    """Ancestor masks [B, N, N] uint8 of random trees, on the device."""
    parent = torch.from_numpy((rng.random((B, N)) * np.arange(N)).astype(np.int64)).cuda()
    mask = torch.eye(N, dtype=torch.bool, device="cuda").repeat(B, 1, 1)
    rows = torch.arange(B, device="cuda")
    for i in range(1, N):
        mask[:, i] |= mask[rows, parent[:, i]]
    return mask.to(torch.uint8)


def attention(c, mask=None, nodes=None):
    """out, lse and what error bounds are made of (absolute, reach, count), as numpy arrays."""
    B, N, Hq, D = c.q.shape
    G, scale = c.G, D ** -0.5
    f64 = dict(dtype=torch.float64, device="cuda")
    out, absolute = (torch.zeros((B, N, Hq, D), **f64) for _ in range(2))
    lse, reach = torch.full((B, N, Hq), -torch.inf, **f64), torch.zeros((B, N, Hq), **f64)
    count = torch.zeros((B, N), dtype=torch.int64, device="cuda")
    kf, vf = (x.reshape(-1, c.Hkv, D) for x in (c.k, c.v))
    for b in range(B):
        n = N if nodes is None else int(nodes[b])
        length = int(c.lens[b])
        at = c.slots(b, 0, length + n)
        there = at >= 0
        if n == 0 or not there.any():
            continue
        x = torch.arange(len(at), device="cuda")[there] - length
        at = at[there]
        if mask is None:
            sees = x[None, :] <= torch.arange(n, device="cuda")[:, None]
        else:
            sees = (x < 0)[None, :] | (mask[b, :n][:, x.clamp(min=0)] != 0)
        count[b, :n] = sees.sum(1)
        for h in range(c.Hkv):
            kk, vv = kf[at, h].double(), vf[at, h].double()
            hq = slice(h * G, (h + 1) * G)
            q = c.q[b, :n, hq].double().reshape(n * G, D)
            see = sees.repeat_interleave(G, 0)
            z = scale * (q @ kk.t().contiguous())
            z = torch.where(see, z, torch.full_like(z, -torch.inf))
            r = scale * (q.abs() @ kk.abs().t().contiguous())
            top = z.amax(1, keepdim=True)
            w = torch.where(see, torch.exp(z - torch.where(top == -torch.inf, 0.0, top)), 0.0)
            total = w.sum(1, keepdim=True)
            fine = torch.isfinite(vv)
            v0 = torch.where(fine, vv, 0.0)
            o = w @ v0
            for t in torch.nonzero(~fine.all(1)).flatten().tolist():
                add = w[:, t, None] * torch.where(fine[t], 0.0, vv[t])[None, :]
                o += torch.where(see[:, t, None] & ~fine[t], add, 0.0)
            some = total != 0  # NaN is not zero
            o = torch.where(some, o / total, 0.0)
            a = torch.where(some, (w @ v0.abs()) / total, 0.0)
            out[b, :n, hq], absolute[b, :n, hq] = o.view(n, G, D), a.view(n, G, D)
            lse[b, :n, hq] = torch.where(some, top + total.log(), -torch.inf).view(n, G)
            r = torch.where(see, r, torch.full_like(r, -torch.inf)).amax(1)
            reach[b, :n, hq] = torch.where(some.squeeze(1), r, 0.0).view(n, G)
    return {k: v.cpu().numpy() for k, v in dict(out=out, lse=lse, absolute=absolute, reach=reach,
                                                count=count).items()}
