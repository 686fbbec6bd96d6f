"""The 8-bit cache's attention tests once more, with a comparison that no NaN passes (kv8_strict.check in the place
of kv8_helpers.check, whose `error > bound` is false for a NaN)."""

import pytest

import kv8_helpers as K8
import kv8_strict
from test_gpu_kv8_attention import (  # noqa: F401  (collected here)
    test_any_scale_and_softmax_scale, test_bad_requests_are_zeroed_alone, test_blocks_beyond_two_gigabytes,
    test_entries_behind_the_prefix_are_not_read, test_long_prefix_and_chain, test_one_long_request_among_many,
    test_sharp_and_flat_rows, test_single_tokens, test_trees, test_values_far_from_one)
from test_gpu_kv8_together import test_decoding_rounds  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    monkeypatch.setattr(K8, "check", kv8_strict.check)
