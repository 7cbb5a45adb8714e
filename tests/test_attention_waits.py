"""How the attention kernels' named barriers stand to their bounded waits, read
from the sources (a wait that runs out cannot be had on purpose on a GPU).

A wait that runs out in one warp must not keep it from a named barrier that
other warps still come to: those have no limit.  So no loop around a named
barrier may end on the outcome of a wait (`ok`), and no branch around one may
depend on it."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "recommender_sparse_embeddings_gb300", "csrc")


def closing(text, at):
    """Position of the brace that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return i
    raise ValueError("unbalanced braces")


def conditions_around(text, at):
    """Heads of the loops and branches that enclose position `at`."""
    found, i, depth = [], at, 0
    while i > 0:
        i -= 1
        if text[i] == "}":
            depth += 1
        elif text[i] == "{":
            if depth:
                depth -= 1
                continue
            head = text[max(text.rfind(c, 0, i) for c in ";{}") + 1:i].strip()
            for_head = re.search(r"for \([^{}]*$", text[max(0, i - 400):i])
            if for_head and text[:i].rstrip().endswith(")"):
                head = for_head.group(0)
            if head.endswith("do"):
                end = closing(text, i)
                head = text[end + 1:text.index(";", end)].strip()
            found.append(head)
    return found


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.startswith("attention")))
def test_named_barriers_are_met_whatever_a_wait_said(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    text = re.sub(r'"(\\.|[^"\\])*"', lambda m: m.group(0).replace("{", "(").replace("}", ")"), text)
    at = [m.start() for m in re.finditer(r"bar(?:rier)?(?:\.cta)?\.(?:sync|red)", text)]
    if name in ("attention_fwd.cu", "attention_bwd.cu"):
        assert len(at) >= 2
    for i in at:
        for head in conditions_around(text, i):
            assert not re.search(r"\bok\b", head), (name, head)
