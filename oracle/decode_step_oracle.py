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
