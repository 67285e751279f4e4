"""The documented speculative step gives every call the status words that its check reads."""

import re

import pytest


@pytest.mark.parametrize("where", ["module", "README"])
def test_every_documented_call_reports(splitkv, where):
    import os
    from conftest import ROOT
    from context_block_sparse_b200 import draft_tree
    text = draft_tree.__doc__
    if where == "README":
        with open(os.path.join(ROOT, "README.md")) as f:
            text = f.read()
    for call in ("verify_draft", "commit_draft"):
        used = re.findall(rf"{call}\(((?:[^()]|\([^()]*\))*)\)", text)
        assert used and all("status=tree.status" in a for a in used), call
    assert "tree.check()" in text
