"""A tcgen05 commit tracks the products of the thread that issues it, and which lane elect.sync chooses is not said:
in the products' source every product and commit stands inside a branch of an elected lane."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "blockwise_fp8_zero_gb300", "csrc")


def enclosing(text, at):
    """What stands before each brace that is open at `at`, innermost last."""
    heads = []
    for m in re.finditer(r"[{}]", text[:at]):
        if m.group() == "{":
            start = max(text.rfind(c, 0, m.start()) for c in ";{}")
            heads.append(text[start + 1:m.start()])
        else:
            heads.pop()
    return heads


@pytest.mark.parametrize("call", ["umma_e4m3_pair(", "umma_e4m3(", "umma_commit_pair(", "umma_commit_one("])
def test_products_and_commits_are_the_elected_lane_s(call):
    with open(os.path.join(CSRC, "matmul.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    places = [m.start() for m in re.finditer(r"(?<!\w)" + re.escape(call), text)]
    assert places
    for at in places:
        assert any("elect_one()" in head for head in enclosing(text, at)), text[at - 200:at + 40]
