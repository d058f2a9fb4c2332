"""Pins of the sampling oracle: small rows whose cuts and draws are worked out by hand."""
import numpy as np
import pytest

from oracle import sample_oracle as Q

LOG = np.log


def test_temperature_only_is_softmax():
    z = np.array([0.5, -1.0, 2.0, 0.0])
    p = Q.probs(z, temperature=0.5)
    np.testing.assert_allclose(p, np.exp(2 * z) / np.exp(2 * z).sum(), rtol=1e-14)


def test_cuts_by_hand():
    z = LOG(np.array([0.1, 0.4, 0.2, 0.3]))
    np.testing.assert_allclose(Q.probs(z, top_k=2), [0, 4 / 7, 0, 3 / 7])
    # before 0.4: 0, before 0.3: 0.4, before 0.2: 0.7, before 0.1: 0.9
    np.testing.assert_allclose(Q.probs(z, top_p=0.69), [0, 4 / 7, 0, 3 / 7])
    np.testing.assert_allclose(Q.probs(z, top_p=0.71), [0, 4 / 9, 2 / 9, 3 / 9])
    # top-p counts within the top-k: before 0.3 of 0.7 lies 0.571
    np.testing.assert_allclose(Q.probs(z, top_k=2, top_p=0.55), [0, 1, 0, 0])
    np.testing.assert_allclose(Q.probs(z, min_p=0.6), [0, 4 / 7, 0, 3 / 7])
    np.testing.assert_allclose(Q.probs(z, temperature=0.0), [0, 1, 0, 0])


def test_ties_go_to_the_lower_index_and_one_token_always_stays():
    z = np.zeros(8)
    np.testing.assert_allclose(Q.probs(z, top_k=3), [1 / 3] * 3 + [0] * 5)
    np.testing.assert_allclose(Q.probs(z, top_p=0.5), [0.25] * 4 + [0] * 4)
    np.testing.assert_allclose(Q.probs(z, top_p=0.0), [1] + [0] * 7)
    np.testing.assert_allclose(Q.probs(z, min_p=2.0), [1 / 8] * 8)


def test_masked_values():
    z = np.array([np.nan, -np.inf, 1.0, np.inf, np.inf])
    np.testing.assert_allclose(Q.probs(z), [0, 0, 0, 0.5, 0.5])
    assert not Q.probs(np.full(4, -np.inf)).any()
    assert Q.token(np.array([np.nan, -np.inf]), 0.3)[:2] == (-1, 0.0)


@pytest.mark.parametrize("u,want", [(0.0, 0), (0.09, 0), (0.11, 1), (0.49, 1), (0.51, 2), (0.999, 3), (1.0, 3), (-1.0, 0), (np.nan, 0)])
def test_token_is_the_first_whose_sum_passes_u(u, want):
    z = LOG(np.array([0.1, 0.4, 0.2, 0.3]))
    i, p, _ = Q.token(z, u)
    assert i == want and abs(p - [0.1, 0.4, 0.2, 0.3][want]) < 1e-12
