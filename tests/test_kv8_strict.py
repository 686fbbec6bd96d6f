"""The attention tests' comparison itself, without a GPU: it passes what is right and nothing else."""

import numpy as np
import pytest

import kv8_helpers as K8
import kv8_strict


@pytest.fixture(scope="module")
def case():
    rng = np.random.default_rng(0)
    cache = K8.Cache(rng, [40, 7], 1, 64, 16)
    qs = K8.Queries(rng, 2, 5, 2, 1, 64, n_nodes=[5, 3])
    answers = [K8.exact(cache, qs, b) for b in range(2)]
    return cache, qs, np.stack([a[0] for a in answers]), np.stack([a[1] for a in answers]), answers


def test_right_answers_pass(case):
    cache, qs, out, lse, answers = case
    kv8_strict.check(cache, qs, out, lse)
    kv8_strict.check(cache, qs, out + 0.9 * np.stack([a[2] for a in answers]), lse)


@pytest.mark.parametrize("wrong", [np.nan, np.inf, -np.inf, 1e9])
@pytest.mark.parametrize("which", ["out", "lse"])
@pytest.mark.parametrize("at", [(0, 4, 1), (1, 2, 0), (1, 4, 1)])
def test_wrong_answers_fail(case, which, wrong, at):
    """Also in a padded node's row, which has to be zeros."""
    cache, qs, out, lse, _ = case
    out, lse = out.copy(), lse.copy()
    if which == "out":
        out[at + (63,)] = wrong
    else:
        lse[at] = wrong
    with pytest.raises(AssertionError):
        kv8_strict.check(cache, qs, out, lse)
