"""Trees decoded at a budget of tokens, as a serving loop does it: rotary positions, tree attention,
verification, commit, the weights of what the accepted nodes alone gave, eviction; against the same
model in float64 on the CPU, token by token."""

import copy

import numpy as np
import pytest
import torch

from cache_cases import announce
from test_gpu_decode_steps import HKV, LAYERS, PAGE, V, Model, Text, forward, i32, new_cache

pytestmark = pytest.mark.gpu

S, M, L, STEPS = 3, 5, 4, 12
N = 1 + M * L                       # every prefix of the candidates has a node
TOP, KEEP, SINKS, RECENT = 24, 16, 2, 4


@pytest.fixture(scope="module")
def svm():
    import speculative_sampling_verification_amd as m
    return m


def clear(logp):
    """The first token, far from the second: fp32 logits here are off by less than 1e-3."""
    order = np.argsort(-logp)
    assert logp[order[0]] - logp[order[1]] > 2e-3
    return int(order[0])


def plan(seed):
    """Steps of each sequence in float64: candidates, the tokens accepted and emitted, whether it was cut
    before, and what it holds behind."""
    rng = np.random.default_rng(seed)
    model = Model(seed)
    prompts = [rng.integers(0, V, n).tolist() for n in (21, 3, 14)]
    texts, steps = [], [[] for _ in range(S)]
    for b, prompt in enumerate(prompts):
        t = Text(model)
        for token in prompt[:-1]:
            t.feed(token, weigh_own=True)
        texts.append(t)
        root = prompt[-1]
        for _ in range(STEPS):
            cut = len(t.w[0][0]) >= TOP
            if cut:  # weights are sums of a few tens of numbers of at most 1, off by less than 1e-4
                assert t.evict(KEEP, SINKS, RECENT) > 2e-4
            trial, truth = copy.deepcopy(t), []
            logp = trial.feed(root, weigh_own=True)
            for _ in range(L + 1):
                truth.append(clear(logp))
                logp = trial.feed(truth[-1], weigh_own=True)
            cands = rng.integers(0, V, (M, L)).astype(np.int32)
            for c in range(M):
                n = rng.integers(0, L + 1)
                cands[c, :n] = truth[:n]
            right = int(max((np.cumprod(c == truth[:L])).sum() for c in cands))
            for token in [root] + truth[:right]:
                t.feed(token, weigh_own=True)
            steps[b].append(dict(cut=cut, cands=cands, out=truth[:right + 1], root=root,
                                 count=t.count, length=len(t.w[0][0]), w=copy.deepcopy(t.w)))
            root = truth[right]
    return model, prompts, steps


def path_of(tree, last):
    """Of each sequence's last accepted node, itself and its ancestors (none for -1)."""
    rows = torch.arange(last.numel(), device="cuda")
    return (tree["mask"][rows, last.clamp(min=0).long()] != 0) & (last >= 0)[:, None]


@pytest.mark.parametrize("seed", [1, 2])
def test_trees_at_a_budget(svm, seed):
    announce(f"trees at a budget of {KEEP} tokens, seed={seed}")
    model, prompts, steps = plan(seed)
    gpu = model.gpu()
    cache = new_cache(svm, S, 8, 30)
    weights = torch.zeros((LAYERS, S, HKV, 64), device="cuda")
    fed = i32([len(p) - 1 for p in prompts])
    width = int(fed.max())
    assert svm.spec_cache_resize(cache, fed + 0).tolist() == [1] * S
    head = torch.zeros((S, width), dtype=torch.int32, device="cuda")
    for b, p in enumerate(prompts):
        head[b, :len(p) - 1] = i32(p[:-1])
    _, given = forward(svm, gpu, cache, head, None, None, None, fed)
    lens = svm.spec_cache_commit(cache, fed - 1, num_nodes=width)
    assert svm.spec_cache_resize(cache, lens, new_lens=lens).tolist() == [1] * S
    upto = torch.arange(1, width + 1, dtype=torch.int32, device="cuda").repeat(S, 1)
    for layer, (q, lse) in enumerate(given):
        svm.spec_cache_weigh(q, lse, cache, weights, layer=layer, seen=upto, num_nodes=fed)
    position = fed.clone()
    for step in range(STEPS):
        want = [steps[b][step] for b in range(S)]
        budget = torch.where(cache.seq_lens >= TOP, KEEP, -1).to(torch.int32)
        assert (budget > 0).tolist() == [w["cut"] for w in want]
        kept = svm.spec_cache_evict(cache, weights, budget, sinks=SINKS, recent=RECENT,
                                    max_keep=KEEP, out={"weights": weights})
        assert svm.spec_cache_resize(cache, kept["lens"], new_lens=kept["lens"]).tolist() == [1] * S
        tree = svm.spec_build_tree(i32(np.stack([w["cands"] for w in want])), N)
        tokens = tree["tokens"].clone()
        tokens[:, 0] = i32([w["root"] for w in want])
        held = cache.seq_lens.clone()
        assert svm.spec_cache_resize(cache, held + N).tolist() == [1] * S
        logits, given = forward(svm, gpu, cache, tokens, position, tree["depth"], tree["mask"],
                                tree["num_nodes"])
        logits = torch.nan_to_num(logits).contiguous()  # slots without a node
        seen = svm.spec_verify_tree(logits, tree["parent"], tokens, L)
        lens = svm.spec_cache_commit(cache, seen["last_node"], parent=tree["parent"])
        assert svm.spec_cache_resize(cache, lens, new_lens=lens).tolist() == [1] * S
        position += lens - held
        # an accepted node counts up to its own position, the others not at all
        upto = torch.where(path_of(tree, seen["last_node"]), held[:, None] + tree["depth"] + 1, 0)
        for layer, (q, lse) in enumerate(given):
            svm.spec_cache_weigh(q, lse, cache, weights, layer=layer, seen=upto.int(),
                                 num_nodes=tree["num_nodes"])
        for b, w in enumerate(want):
            n = int(seen["num_accepted"][b]) + 1
            assert seen["tokens"][b, :n].tolist() == w["out"], (step, b)
            assert position[b] == w["count"] and cache.seq_lens[b] == w["length"]
            there = np.array(w["w"])
            np.testing.assert_allclose(weights[:, b, :, :w["length"]].cpu().numpy(), there,
                                       atol=1e-4, err_msg=f"step {step}, sequence {b}")
            assert (weights[:, b, :, w["length"]:] == 0).all()
    assert cache.seq_pages.tolist() == [-(-n // PAGE) for n in cache.seq_lens.tolist()]
