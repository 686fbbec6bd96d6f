"""The order of tensor instructions in the tensor-core attention over the 8-bit cache, without a GPU.

A tile's weights lie over its scores, and the next scores of that buffer over them.  Tensor instructions keep the order they
are issued in only where they have one accumulator and one shape, which the output's and the scores' are not.  So between
them stands a commit of the one and a wait for it."""

import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_speculative_decoding_split_gb300", "csrc",
                      "attention_kv8_tc.cu")


def _code():
    return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", open(SOURCE).read()))


def test_the_next_scores_wait_for_the_product_that_reads_the_weights():
    code = _code()
    step = code[code.index("auto step = [&]"):code.index("auto run = [&]")]
    steps = ["wait(&pfull[g][t & 1], (t >> 1) & 1)", "issue_pv(pv_tree, t, g);", "if (t + C::kNB < T) {", "if (leader) umma_commit(&s_pread[g]);",
             "if (!wait(&s_pread[g], t & 1)) return false;", "issue_s(s_tree, t + C::kNB, g);"]
    at = [step.index(x) for x in steps]
    assert at == sorted(at) and step.count("issue_s(") == 1 and step.count("issue_pv(") == 1
    assert "mbar_init(&s_pread[g], 1);" in code and code.count("&s_pread[g]") == 3


@pytest.mark.parametrize("groups,buffers", [(1, 2), (2, 1)])
@pytest.mark.parametrize("waits", [True, False])
def test_the_steps_with_instructions_in_any_allowed_order(groups, buffers, waits):
    """The issuer's steps over tensor cores that keep each accumulator's order and no other; the softmax answers scores with
    weights.  With the waits no scores come over weights that are still to be read; without them some do."""
    found = 0
    for seed in range(60):
        rng, T = random.Random(seed), 7
        columns = {(g, b): None for g in range(groups) for b in range(buffers)}
        queue = []  # (accumulator, what it does); a commit is a count of what is ahead of it

        def run_one():
            nonlocal found
            allowed = [i for i, op in enumerate(queue) if all(x[0] != op[0] for x in queue[:i])]
            acc, kind, t, g = queue.pop(rng.choice(allowed))
            at = (g, t % buffers)
            if kind == "S":
                found += columns[at] is not None and columns[at] != ("read", t - buffers)
                columns[at] = ("weights", t)
            else:
                found += columns[at] != ("weights", t)
                columns[at] = ("read", t)

        def issue(kind, t, g):
            queue.append((("O", g) if kind == "PV" else ("S", g, t % buffers), kind, t, g))

        def until(kind, t, g):
            while any(x[1:] == (kind, t, g) for x in queue):
                run_one()

        for t in range(buffers):
            for g in range(groups):
                issue("S", t, g)
        for t in range(T):
            for g in range(groups):
                until("S", t, g)  # the weights are there
                issue("PV", t, g)
                if t + buffers < T:
                    if waits:
                        until("PV", t, g)
                    issue("S", t + buffers, g)
        while queue:
            run_one()
    assert (found == 0) == waits
