"""The merge's table of units that a run's end cuts (`cuts`): one thread of a CTA makes
every store to it, so that a run's "nothing cut" and the cut that it does leave have an
order.  Nothing else orders them: the thread that finds the cut may store it before the
CTA's first wait."""
import os
import re

import pytest

from exact_attention_48_gb300 import build as fa_build


@pytest.mark.parametrize("name", ["fa_tree.cu", "fa_tree_fp8_tc.cu", "fa_tree_fp8_rows.cu"])
def test_one_thread_stores_the_cuts(name):
    with open(os.path.join(fa_build.CSRC, name), encoding="utf-8") as f:
        text = f.read()
    stores = [m.start() for m in re.finditer(r"p\.cuts\[[^;]*?\]\s*=\s", text, re.S)]
    assert len(stores) == 2
    threads = set()
    for at in stores:
        condition = text[text.rindex("if (", 0, at):at]
        assert ";" not in condition, condition            # the store's own condition
        threads.add(re.search(r"threadIdx\.x == ([^&)]+?)\s*(?:&&|\))", condition).group(1).strip())
    assert len(threads) == 1, threads
