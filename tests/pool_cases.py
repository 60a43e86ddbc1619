"""A page pool on the device beside the oracle's, as tests of who may write a page use it."""

import numpy as np
import torch

import oracle.paged_cache_oracle as O
from cache_cases import DTYPES, check_attention, ints, random_tree
from test_gpu_cache import Pool


def i32(*x):
    return np.array(x, dtype=np.int32)


class OwnedPool(Pool):
    """Calls on the pool's cache, each compared with the oracle where a page is held.  (A page that
    nobody holds may be written by several sequences whose stale entries name it.)"""

    def same(self):
        torch.cuda.synchronize()
        c = self.cache
        np.testing.assert_array_equal(c.seq_lens.cpu().numpy(), self.lens)
        np.testing.assert_array_equal(c.seq_pages.cpu().numpy(), self.held)
        np.testing.assert_array_equal(c.refcount.cpu().numpy(), self.ref)
        np.testing.assert_array_equal(c.page_table.cpu().numpy(), self.table)
        owned = self.ref > 0
        for host, dev in ((self.k, self.kd), (self.v, self.vd)):
            got = self.bits(dev)
            np.testing.assert_array_equal(got[:, owned], host[:, owned])
            host[:, ~owned] = got[:, ~owned]

    def append(self, N, nodes=None, layer=0):
        dtype = self.kd.dtype
        new = [torch.from_numpy(self.rng.standard_normal((len(self.lens), N) + self.kd.shape[3:]))
               .to(dtype) for _ in range(2)]
        self.svm.spec_cache_append(new[0].cuda(), new[1].cuda(), self.cache, layer=layer,
                                   num_nodes=None if nodes is None else ints(nodes))
        O.append(self.k[layer], self.v[layer], self.bits(new[0]), self.bits(new[1]), self.table,
                 self.lens, nodes, self.held, self.ref)
        self.same()

    def attend(self, N, nodes=None, layer=0, G=2):
        name = next(n for n, t in DTYPES.items() if t == self.kd.dtype)
        Hkv, D = self.kd.shape[3:]
        q = torch.from_numpy(self.rng.standard_normal((len(self.lens), N, Hkv * G, D)))
        q = q.to(self.kd.dtype)
        mask = random_tree(self.rng, len(self.lens), N)[1]
        got = self.svm.spec_tree_attention(q.cuda(), self.cache, layer=layer, mask=ints(mask),
                                           num_nodes=None if nodes is None else ints(nodes),
                                           want_lse=True)
        torch.cuda.synchronize()
        ref = O.tree_attention(q.double().numpy(), self.kd[layer].double().cpu().numpy(),
                               self.vd[layer].double().cpu().numpy(), self.table, self.lens, mask,
                               nodes, held=self.held, refcount=self.ref)
        check_attention(got, ref, name, D)
        return ref

    def commit(self, last, parent):
        got = self.svm.spec_cache_commit(self.cache, ints(last), parent=ints(parent))
        want = O.commit(self.k, self.v, self.table, self.lens, last, parent, held=self.held,
                        refcount=self.ref)
        np.testing.assert_array_equal(got.cpu().numpy(), want)
        self.same()
        return want

    def text(self, b, first=0, last=None):
        """The committed rows of a sequence in every layer, by the pages it holds."""
        last = int(self.lens[b]) if last is None else last
        x = np.arange(first, last)
        at = self.table[b, x // self.page], x % self.page
        return np.stack([self.k[:, at[0], at[1]], self.v[:, at[0], at[1]]])
