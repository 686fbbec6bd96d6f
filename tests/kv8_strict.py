"""The comparison of the 8-bit cache's attention tests (kv8_helpers.check) in a form that no NaN passes: what is
not at most its bound off fails, and so does anything that is no finite number."""

import numpy as np

import kv8_helpers as K8


def within(got, want, bound):
    """Where `got` is at most `bound` from `want`; a NaN on any side is nowhere."""
    return np.isfinite(got) & (np.abs(got - want) <= bound)


def check(cache, qs, out, lse, scale=0.0, requests=None):
    for b in range(len(cache.lens)) if requests is None else requests:
        O, LSE, E, EL = K8.exact(cache, qs, b, scale)
        n = int(qs.n_nodes[b])
        assert (out[b, n:] == 0).all() and (lse[b, n:] == 0).all(), b
        bad = ~within(out[b], O, E)
        assert not bad.any(), (b, int(bad.sum()), np.nanmax(np.abs(out[b] - O)), np.argwhere(bad)[:3].tolist())
        bad = ~within(lse[b], LSE, EL)
        assert not bad.any(), (b, int(bad.sum()), np.nanmax(np.abs(lse[b] - LSE)), np.argwhere(bad)[:3].tolist())
