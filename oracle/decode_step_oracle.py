"""What a decoding step does around verification, in float64 and index order: rotary positions,
attention weights of the committed tokens, eviction, token log probabilities.

Plain numpy, written from the formulas; it shares no code with the HIP path.
"""

import numpy as np

from .paged_cache_oracle import positions as cache_positions


# --------------------------------------------------------------------------------------- rotary
def rotary_frequencies(rot_dim, theta=10000.0, scaling=None, factor=1.0, original_length=0.0,
                       beta_fast=32.0, beta_slow=1.0):
    """Frequencies of the pairs and the amplitude that goes with them."""
    half = rot_dim // 2
    out = []
    for p in range(half):
        f = theta ** (-2.0 * p / rot_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "ntk" and rot_dim > 2:
            f = (theta * factor ** (rot_dim / (rot_dim - 2.0))) ** (-2.0 * p / rot_dim)
        elif scaling == "yarn":
            r = original_length / (2 * np.pi / f)  # original context over wavelength
            gamma = 0.0 if r < beta_slow else 1.0 if r > beta_fast else \
                (r - beta_slow) / (beta_fast - beta_slow)
            f = (1 - gamma) * f / factor + gamma * f
        out.append(f)
    return np.array(out), 0.1 * np.log(factor) + 1 if scaling == "yarn" else 1.0


def rotary(x, position, freq, interleaved=False, amplitude=1.0):
    """x [B, N, H, D] turned; position [B, N]."""
    half = len(freq)
    out = np.array(x, dtype=np.float64)
    for p in range(half):
        c0, c1 = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        a = position.astype(np.float64) * freq[p]
        cos, sin = np.cos(a)[:, :, None], np.sin(a)[:, :, None]
        u, v = x[..., c0].astype(np.float64), x[..., c1].astype(np.float64)
        out[..., c0] = amplitude * (u * cos - v * sin)
        out[..., c1] = amplitude * (u * sin + v * cos)
    return out


# ------------------------------------------------------------------------------------- eviction
def _books(held, refcount, b):
    return None if held is None or refcount is None else (int(held[b]), refcount)


def _length(lens, b, cap):
    return min(max(int(lens[b]), 0), cap)


def weigh(q, lse, k, table, lens, weights, seen=None, nodes=None, scale=None, decay=1.0, held=None,
          refcount=None):
    """weights [B, Hkv, L] of one layer after a step whose nodes' queries are q [B, N, Hq, D]; k
    [pages, page_size, Hkv, D].  Also returns what error bounds are made of, each [B, Hkv, L]: given
    (what the step adds) and doubt = sum over rows of weight * (scale * sum |q k| * (D + 8)
    + 4 |lse| + 4)."""
    B, N, Hq, D = q.shape
    pages, page_size, Hkv, _ = k.shape
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    out = np.array(weights, dtype=np.float64)
    L = out.shape[2]
    given, doubt = np.zeros_like(out), np.zeros_like(out)
    for b in range(B):
        length = min(_length(lens, b, table.shape[1] * page_size), L)
        n = N if nodes is None else min(max(int(nodes[b]), 0), N)
        for x, page, slot in cache_positions(table[b], page_size, pages, 0, length,
                                             _books(held, refcount, b)):
            for i in range(n):
                if seen is not None and x >= int(seen[b, i]):
                    continue
                for h in range(Hq):
                    if lse[b, i, h] == -np.inf:
                        continue
                    kk = k[page, slot, h // G]
                    w = np.exp(scale * (q[b, i, h] @ kk) - lse[b, i, h])
                    given[b, h // G, x] += w
                    doubt[b, h // G, x] += w * (scale * (np.abs(q[b, i, h]) @ np.abs(kk)) * (D + 8)
                                                + 4 * abs(lse[b, i, h]) + 4)
        if decay == 0:
            out[b, :, :length] = given[b, :, :length]
        else:
            out[b, :, :length] = decay * out[b, :, :length] + given[b, :, :length]
    return out, given, doubt


def evict(k, v, table, lens, weights, keep, sinks=0, recent=0, max_keep=None, held=None,
          refcount=None):
    """Changes k, v [layers, pages, page_size, Hkv, D]; returns (lens, kept, weights) as
    spec_cache_evict does."""
    layers, pages, page_size, Hkv, _ = k.shape
    B, L = weights.shape[1], weights.shape[3]
    max_keep = L if max_keep is None else max_keep
    out = np.array(weights)
    kept = np.full((layers, B, Hkv, max_keep), -1, dtype=np.int32)
    new_lens = np.zeros(B, dtype=np.int32)
    for b in range(B):
        n, want = _length(lens, b, table.shape[1] * page_size), int(keep[b])
        new_lens[b] = n
        where = cache_positions(table[b], page_size, pages, 0, n, _books(held, refcount, b))
        if want < 0 or want > max_keep or want < sinks + recent or n <= want or n > L:
            continue
        if len(where) < n:
            continue
        if refcount is not None and any(refcount[page] > 1 for x, page, _ in where
                                        if x // page_size * page_size < want
                                        and (x // page_size + 1) * page_size > sinks):
            continue
        new_lens[b] = want
        for layer in range(layers):
            for h in range(Hkv):
                w = weights[layer, b, h]
                middle = list(range(sinks, n - recent))
                # largest first, NaN behind all, ties by position (Python's sort is stable)
                middle.sort(key=lambda x: np.inf if np.isnan(w[x]) else -float(w[x]))
                nans = [x for x in middle if np.isnan(w[x])]
                middle = [x for x in middle if not np.isnan(w[x])] + nans
                stay = list(range(sinks)) + sorted(middle[:want - sinks - recent]) + \
                    list(range(n - recent, n))
                kept[layer, b, h, :want] = stay
                out[layer, b, h, :n] = 0
                out[layer, b, h, :want] = w[stay]
                for t in (k, v):
                    rows = [t[layer, where[x][1], where[x][2], h].copy() for x in stay]
                    for j, row in enumerate(rows):
                        t[layer, where[j][1], where[j][2], h] = row
    return new_lens, kept, out


# --------------------------------------------------------------------- token log probabilities
def token_logprobs(logits, tokens=None, rows=None, temperature=1.0, top_n=0):
    """logits [num_rows, V] float64, tokens [R], rows [R]: a dict as spec_token_logprobs returns it,
    everything wanted, and what error bounds are made of, [R] each: spread = |x_t - x_max|, mean and
    square = the means of |x - x_max| and its square under the distribution (x = logits / T)."""
    num_rows, V = logits.shape
    R = num_rows if rows is None else len(rows)
    out = dict(logprob=np.full(R, -np.inf), rank=np.full(R, -1, dtype=np.int64),
               entropy=np.zeros(R), top_tokens=np.full((R, top_n), -1, dtype=np.int64),
               top_logprobs=np.full((R, top_n), -np.inf), spread=np.zeros(R), mean=np.zeros(R),
               square=np.zeros(R))
    for r in range(R):
        row = r if rows is None else int(rows[r])
        if not 0 <= row < num_rows:
            continue
        z = np.asarray(logits[row], dtype=np.float64)
        t = -1 if tokens is None else int(tokens[r])
        if 0 <= t < V:
            out["rank"][r] = (z > z[t]).sum() + (z[:t] == z[t]).sum()
        some = np.flatnonzero(z > -np.inf)
        if len(some) == 0:
            continue
        x = (z - z.max()) / temperature
        e = np.exp(x)
        log_total = np.log(e.sum())
        p = e / e.sum()
        far = np.where(p > 0, -x, 0.0)
        if 0 <= t < V:
            out["logprob"][r] = x[t] - log_total
            out["spread"][r] = -x[t] if z[t] > -np.inf else 0.0
        out["entropy"][r] = log_total + (p * far).sum()
        out["mean"][r], out["square"][r] = (p * far).sum(), (p * far ** 2).sum()
        first = some[np.lexsort((some, -z[some]))][:top_n]
        out["top_tokens"][r, :len(first)] = first
        out["top_logprobs"][r, :len(first)] = x[first] - log_total
    return out
