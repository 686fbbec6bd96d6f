"""The way of the two softmax warps that share rows of the tensor-core attention kernel over the 8-bit cache
(csrc/attention_kv8_tc.cu), without a GPU.

Their barriers have no limit, while each warp's waits for scores and for the output's products may give up at any
time.  So whatever the waits answer, the two have to meet at the same barriers.  The walk below is the kernel's, with
the waits' answers and the softmax's own questions (does a reference have to move?) left open; the test goes through
all of them."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "tree_speculative_decoding_split_gb300", "csrc", "attention_kv8_tc.cu")


def walk(T, Tt, ends_inside, one_buffer):
    """One warp: yields ("wait", name), ("ask", name) for an open answer and ("barrier", name, predicate) for the OR;
    returns whether all its waits were kept."""
    kept = True

    def wait(name):
        nonlocal kept
        if not (yield "wait", name):
            kept = False

    def move(t):
        yield "barrier", "move, scores exchanged", False
        yield "barrier", "move, both have read", False
        if t > 0 and not one_buffer:
            yield from wait("products")

    for t in range(T):
        yield from wait("scores")
        if t < Tt:
            ask = yield "ask", "tree tile"
            if (yield "barrier", "tree tile", ask):
                yield from move(t)
            continue
        slow = t == Tt or (t == T - 1 and ends_inside)
        if not slow:
            ask = yield "ask", "prefix tile"
            slow = yield "barrier", "prefix tile", ask
        if slow:
            yield from move(t)
    return kept


def walk_alone(T, Tt, one_buffer):
    """The same where a warp whose wait gives up leaves by itself."""
    for t in range(T):
        if not (yield "wait", "scores"):
            return False
        ask = yield "ask", "tile"
        if (yield "barrier", "tile", ask):
            yield "barrier", "move, scores exchanged", False
            yield "barrier", "move, both have read", False
            if t > 0 and not one_buffer and not (yield "wait", "products"):
                return False
    return True


def run(make, script):
    """Both warps with the open answers of `script` (further ones True for waits, False for questions).  Returns
    (the answers given, each warp's end or None when one stands at a barrier that the other never comes to)."""
    given, ends = [], [None, None]
    warps = [make(), make()]
    at = [None, None]

    def answer(kind):
        bit = script[len(given)] if len(given) < len(script) else False
        given.append(bit)
        return bit if kind == "ask" else not bit  # (a wait is kept unless its bit is set)

    def go(i, value):
        try:
            event = warps[i].send(value)
            while event[0] != "barrier":
                event = warps[i].send(answer(event[0]))
            at[i] = event
        except StopIteration as stop:
            at[i], ends[i] = None, stop.value

    go(0, None)
    go(1, None)
    while at[0] and at[1]:
        if at[0][1] != at[1][1]:
            return given, None
        both = at[0][2] or at[1][2]
        go(0, both)
        go(1, both)
    return given, (ends if not at[0] and not at[1] else None)


def every(make):
    """Ends for all answers (each run's script, and every later answer turned over in turn)."""
    todo = [[]]
    while todo:
        script = todo.pop()
        given, ends = run(make, script)
        yield given, ends
        for i in range(len(script), len(given)):
            todo.append(given[:i] + [True])


@pytest.mark.parametrize("one_buffer", [False, True])
@pytest.mark.parametrize("ends_inside", [False, True])
@pytest.mark.parametrize("T,Tt", [(1, 1), (1, 0), (2, 1), (2, 2), (2, 0), (3, 1)])
def test_the_pair_stays_together(T, Tt, ends_inside, one_buffer):
    ends = [e for _, e in every(lambda: walk(T, Tt, ends_inside, one_buffer))]
    assert None not in ends and [True, True] in ends and [False, True] in ends and [False, False] in ends


def test_the_search_finds_a_warp_left_alone():
    assert any(ends is None for _, ends in every(lambda: walk_alone(2, 1, False)))


def test_the_kernel_takes_these_steps():
    """The pair's barriers in the order in which the source has them, and no way out between them."""
    code = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    body = code[code.index("auto move_references ="): code.index("const bool fin =")]
    steps = re.findall(r"bar_or\(pair|named_bar_sync\(pair|[^ ]* = move_references\(|move_references\(top|"
                       r"\breturn;|\breturn (?:true|false)|\bbreak\b|\bcontinue\b|\bgoto\b", body)
    assert steps == ["named_bar_sync(pair", "named_bar_sync(pair",  # move_references
                     "bar_or(pair", "move_references(top",          # tree tile
                     "bar_or(pair", "asked = move_references("]     # prefix tile
