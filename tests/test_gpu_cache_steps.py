"""The cache operators together, as a speculative decoding loop uses them: a small two-layer
model decodes greedily through spec_build_tree, spec_cache_resize, spec_cache_append,
spec_tree_attention, spec_verify_tree and spec_cache_commit, and has to emit what the same model
emits token by token in float64 on the CPU."""

import numpy as np
import pytest
import torch

from cache_cases import announce

pytestmark = pytest.mark.gpu

V, E, HQ, HKV, D, LAYERS, PAGE = 61, 128, 4, 2, 64, 2, 8


@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    return m


class Model:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
        self.emb, self.pos = r(V, E), 0.3 * r(400, E)
        self.wq = [r(E, HQ * D) * E ** -0.5 for _ in range(LAYERS)]
        self.wk = [r(E, HKV * D) * E ** -0.5 for _ in range(LAYERS)]
        self.wv = [r(E, HKV * D) * E ** -0.5 for _ in range(LAYERS)]
        self.wo = [2 * r(HQ * D, E) * (HQ * D) ** -0.5 for _ in range(LAYERS)]
        self.head = r(E, V)

    def to(self, dtype, device):
        m = object.__new__(Model)
        for k, v in self.__dict__.items():
            m.__dict__[k] = [x.to(device, dtype) for x in v] if isinstance(v, list) else \
                v.to(device, dtype)
        return m

    def norm(self, x):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)

    def logits(self, tokens):
        """Next-token logits after each prefix of a list of tokens (dense, causal)."""
        n = len(tokens)
        x = self.emb[tokens] + self.pos[:n]
        see = torch.ones((n, n), dtype=torch.bool).tril()
        for layer in range(LAYERS):
            y = self.norm(x)
            q = (y @ self.wq[layer]).view(n, HQ, D).transpose(0, 1)
            k = (y @ self.wk[layer]).view(n, HKV, D).repeat_interleave(HQ // HKV, 1)
            v = (y @ self.wv[layer]).view(n, HKV, D).repeat_interleave(HQ // HKV, 1)
            z = (q @ k.permute(1, 2, 0)) * D ** -0.5
            p = torch.softmax(z.masked_fill(~see, -torch.inf), -1)
            x = x + (p @ v.transpose(0, 1)).transpose(0, 1).reshape(n, -1) @ self.wo[layer]
        return self.norm(x) @ self.head

    def continue_greedily(self, prompt, count):
        """count tokens, and the smallest lead of a chosen logit over the next one."""
        tokens, lead = list(prompt), np.inf
        for _ in range(count):
            top = torch.topk(self.logits(tokens)[-1], 2)
            lead = min(lead, float(top.values[0] - top.values[1]))
            tokens.append(int(top.indices[0]))
        return tokens[len(prompt):], lead


def forward(svm, m, cache, tokens, pos, mask, nodes):
    """Logits [B, N, V] of drafted nodes through the cache's layers."""
    B, N = tokens.shape
    x = m.emb[tokens.clamp(min=0).long()] + m.pos[pos.clamp(min=0).long()]
    for layer in range(LAYERS):
        y = m.norm(x)
        qkv = torch.cat([y @ m.wq[layer], y @ m.wk[layer], y @ m.wv[layer]], -1)
        qkv = qkv.view(B, N, HQ + 2 * HKV, D)
        svm.spec_cache_append(qkv[:, :, HQ:HQ + HKV], qkv[:, :, HQ + HKV:], cache, layer=layer,
                              num_nodes=nodes)
        o = svm.spec_tree_attention(qkv[:, :, :HQ], cache, layer=layer, mask=mask,
                                    num_nodes=nodes)["out"]
        x = x + o.reshape(B, N, -1) @ m.wo[layer]
    return m.norm(x) @ m.head


@pytest.mark.parametrize("seed", [0, 1])
def test_tree_decoding_equals_token_by_token(svm, seed):
    announce(f"tree decoding through a paged cache, seed={seed}")
    rng = np.random.default_rng(seed)
    model = Model(seed)
    gpu = model.to(torch.float32, "cuda")
    S, live, count, M, L, N = 5, 3, 24, 6, 5, 16
    prompts = [rng.integers(0, V, n).tolist() for n in (1, 19, 8)]
    answer, leads = zip(*(model.continue_greedily(p, count) for p in prompts))
    # fp32 logits here are off by less than 1e-3 (sums of 128 products of size 10 in 24 bits, a
    # few layers deep): a lead beyond that decides alike
    assert min(leads) > 2e-3
    pages = 80
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.full((LAYERS, pages, 2, PAGE, HKV, D), float("nan"), device="cuda")
    cache = svm.PagedCache(k[:, :, 0], k[:, :, 1], torch.full((S, 12), -1, dtype=torch.int32,
                                                              device="cuda"),
                           i32([0] * S), seq_pages=i32([0] * S), refcount=i32([0] * pages))
    # the prompts but their last tokens, as ragged chains
    width = max(len(p) for p in prompts)
    assert svm.spec_cache_resize(cache, i32([len(p) for p in prompts] + [-1, -1])).tolist() == [1] * S
    head = torch.zeros((S, width), dtype=torch.int32, device="cuda")
    for b, p in enumerate(prompts):
        head[b, :len(p) - 1] = i32(p[:-1])
    fed = i32([len(p) - 1 for p in prompts] + [0, 0])
    pos = torch.arange(width, device="cuda").expand(S, -1)
    forward(svm, gpu, cache, head, pos, None, fed)
    new = svm.spec_cache_commit(cache, fed - 1, num_nodes=width)
    assert svm.spec_cache_resize(cache, new, new_lens=new).tolist() == [1] * S
    assert cache.seq_lens.tolist() == fed.tolist()

    texts = [list(p) for p in prompts] + [None, None]
    goal = [p + list(a) for p, a in zip(prompts, answer)]
    alive = list(range(live))
    for step in range(40):
        if step == 2:  # sequence 1 goes on as 3 and 4 too
            ok = svm.spec_cache_fork(cache, i32([1, 1]), i32([3, 4]))
            assert ok.tolist() == [1, 1]
            texts[3], texts[4] = list(texts[1]), list(texts[1])
            goal += [goal[1], goal[1]]
            alive = list(range(S))
        # candidates that follow the true text for a while
        cands = rng.integers(0, V, (S, M, L)).astype(np.int32)
        for b in alive:
            rest = (goal[b][len(texts[b]):] + [0] * L)[:L]
            for c in range(M):
                n = rng.integers(0, L + 1)
                cands[b, c, :n] = rest[:n]
        tree = svm.spec_build_tree(i32(cands), N)
        root = i32([t[-1] if t else 0 for t in texts])
        tokens = tree["tokens"].clone()
        tokens[:, 0] = root
        used = torch.zeros(S, dtype=torch.bool, device="cuda")
        used[alive] = True
        nodes = torch.where(used, tree["num_nodes"], torch.zeros_like(tree["num_nodes"]))
        want = torch.where(used, cache.seq_lens + N, torch.full_like(nodes, -1))
        assert svm.spec_cache_resize(cache, want).tolist() == [1] * S
        logits = forward(svm, gpu, cache, tokens, cache.seq_lens[:, None] + tree["depth"],
                         tree["mask"], nodes)
        logits = torch.nan_to_num(logits).contiguous()
        seen = svm.spec_verify_tree(logits, tree["parent"], tokens, L)
        last = torch.where(used, seen["last_node"], torch.full_like(nodes, -1))
        new = svm.spec_cache_commit(cache, last, parent=tree["parent"])
        assert svm.spec_cache_resize(cache, torch.where(used, new, want), new_lens=new).tolist() \
            == [1] * S
        out, n = seen["tokens"].tolist(), seen["num_accepted"].tolist()
        for b in alive:
            texts[b] += out[b][:n[b] + 1]
        if all(len(texts[b]) >= len(goal[b]) for b in alive):
            break
    for b in alive:
        assert texts[b][:len(goal[b])] == goal[b], b
        assert int(cache.seq_lens[b]) == len(texts[b]) - 1
    # the pool's books: every page is held as often as tables name it
    held = cache.seq_pages.tolist()
    names = np.concatenate([cache.page_table[b, :held[b]].cpu().numpy() for b in range(S)])
    np.testing.assert_array_equal(np.bincount(names, minlength=pages), cache.refcount.cpu().numpy())
    assert svm.spec_cache_resize(cache, i32([0] * S)).tolist() == [1] * S
    assert cache.refcount.abs().sum().item() == 0
