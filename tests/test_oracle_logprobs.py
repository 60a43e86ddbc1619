"""Token log probabilities: the oracle against definitions and closed forms."""

import numpy as np

import oracle.decode_step_oracle as O


def test_definition():
    rng = np.random.default_rng(0)
    z = rng.standard_normal((4, 9))
    got = O.token_logprobs(z, tokens=[0, 3, 8, 9], temperature=0.7, top_n=9)
    for r in range(4):
        p = np.exp(z[r] / 0.7) / np.exp(z[r] / 0.7).sum()
        np.testing.assert_allclose(np.exp(got["top_logprobs"][r]).sum(), 1.0, rtol=1e-12)
        np.testing.assert_allclose(got["entropy"][r], -(p * np.log(p)).sum(), rtol=1e-12)
        np.testing.assert_array_equal(z[r][got["top_tokens"][r]], np.sort(z[r])[::-1])
        t = [0, 3, 8, 9][r]
        if t == 9:
            assert got["logprob"][r] == -np.inf and got["rank"][r] == -1
        else:
            np.testing.assert_allclose(np.exp(got["logprob"][r]), p[t], rtol=1e-12)
            assert got["top_tokens"][r, got["rank"][r]] == t


def test_ties_and_masks():
    z = np.array([[1.0, 2.0, 2.0, -np.inf, 2.0], [-np.inf] * 5, [0.0, -0.0, 0.0, 0.0, 0.0]])
    got = O.token_logprobs(z, tokens=[4, 2, 1], top_n=5)
    assert got["top_tokens"].tolist() == [[1, 2, 4, 0, -1], [-1] * 5, [0, 1, 2, 3, 4]]
    assert got["rank"].tolist() == [2, 2, 1]
    assert got["logprob"][1] == -np.inf and got["entropy"][1] == 0
    np.testing.assert_allclose(got["entropy"][2], np.log(5), rtol=1e-12)
    np.testing.assert_allclose(got["top_logprobs"][2], -np.log(5))


def test_rows():
    rng = np.random.default_rng(1)
    z = rng.standard_normal((3, 6))
    rows, tokens = [2, 2, 0, -1, 3], [1, 5, 0, 0, 0]
    got = O.token_logprobs(z, tokens, rows, top_n=2)
    one = O.token_logprobs(z[rows[:3]], tokens[:3], top_n=2)
    for k in got:
        np.testing.assert_array_equal(got[k][:3], one[k])
    assert (got["logprob"][3:] == -np.inf).all() and (got["rank"][3:] == -1).all()
    assert (got["top_tokens"][3:] == -1).all() and (got["entropy"][3:] == 0).all()
