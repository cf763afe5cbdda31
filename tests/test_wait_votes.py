"""Bounded waits of whole warps, read from the source (no GPU).

Each lane of a warp polls a barrier, the clock and the abort flag by itself, so a wait that
runs out can tell some lanes of a warp that it succeeded and others that it did not.  Code
that goes on with warp-wide operations must take the answer of the whole warp."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_indexer_sum_b200", "csrc")


def _body(name, function):
    """The text of `function` in csrc/`name`, without comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index("void %s(" % function)
    at = text.index("{", at)
    depth, end = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
        if depth == 0:
            return text[at:end]


VOTE = r"__(?:all|any)_sync\(\s*0xffffffffu,"


def _unvoted_branches(body):
    """Branches of the body on the answer of a wait (`wait(..)`, or `ok`, which holds the last
    ones' answers) that no vote of the warp came before."""
    bad = []
    for m in re.finditer(r"\b(?:if|while)\s*\(", body):
        depth, end = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(body[end], 0)
            end += 1
        cond = body[m.end():end - 1]
        if re.search(r"(?<![\w.])wait\(", cond):
            voted = re.search(VOTE, cond)
        elif re.search(r"\bok\b", cond):
            last = [a for a in re.finditer(r"\bok = ([^;]*);", body[:m.start()])][-1]
            voted = re.search(VOTE, cond) or re.match(VOTE, last.group(1))
        else:
            continue
        if not voted:
            bad.append(re.sub(r"\s+", " ", cond))
    return bad


@pytest.mark.parametrize("name,function", [("attn_packed.cuh", "packed_consumer")])
def test_a_warp_branches_on_the_answer_of_all_its_lanes(name, function):
    body = _body(name, function)
    assert len(re.findall(r"(?<![\w.])wait\(", body)) >= 3
    assert _unvoted_branches(body) == []

