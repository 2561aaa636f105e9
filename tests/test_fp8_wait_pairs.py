"""The sites of every wait of the kernels on an 8-bit cache, those for two barriers at once
(mbar_wait_both) among them: each barrier has its site beside it, and no site stands for
both a buffer to be filled and one to be free."""
import collections
import os
import re

import pytest

from exact_attention_48_gb300 import build as fa_build

KERNELS = ("fa_tree_fp8_tc.cu", "fa_tree_fp8_rows.cu")


def arguments(text, at):
    """The arguments of the call whose opening bracket is at text[at]."""
    out, depth, start = [], 0, at + 1
    for i in range(at, len(text)):
        depth += (text[i] in "([") - (text[i] in ")]")
        if depth == 0 or (depth == 1 and text[i] == ","):
            out.append(" ".join(text[start:i].split()))
            start = i + 1
        if depth == 0:
            return out
    raise ValueError("no closing bracket")


def waits(name):
    """(barrier, site) of every wait of a file."""
    with open(os.path.join(fa_build.CSRC, name), encoding="utf-8") as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = []
    for m in re.finditer(r"\bmbar_wait(_both)?\(", text):
        a = arguments(text, m.end() - 1)
        if m.group(1):
            assert len(a) == 7 and a[6] == "ctl", a
            found += [(a[0], a[2]), (a[3], a[5])]
        else:
            assert len(a) == 4 and a[2] == "ctl", a
            found.append((a[0], a[3]))
    assert all(site.startswith("kSite") for _, site in found)
    return [(re.match(r"&?(\w+)", bar).group(1), site) for bar, site in found]


def test_every_wait_is_looked_at():
    for name in KERNELS:
        with open(os.path.join(fa_build.CSRC, name), encoding="utf-8") as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        both = text.count("mbar_wait_both(")
        assert both >= 2 and len(waits(name)) == text.count("mbar_wait(") + 2 * both


# what a wait for the barrier waits for; K's slot and S (or V's slot and O) are told free by the product that read them
SITES = {
    "k_full": {"kSiteKFull"}, "v_full": {"kSiteVFull"}, "q_full": {"kSiteQFull"}, "q_empty": {"kSiteQEmpty"},
    "s_free": {"kSiteSFree"}, "p_ready": {"kSitePReady"}, "o_empty": {"kSiteDqEmpty"}, "mask_full": {"kSiteMaskFull"},
    "mask_empty": {"kSiteMaskEmpty"}, "l_full": {"kSiteLseFull"}, "l_empty": {"kSiteLseEmpty"},
    "s_full": {"kSiteSFull", "kSiteKEmpty"}, "pv_done": {"kSitePvDone", "kSiteVEmpty", "kSiteSFree"},
}


@pytest.mark.parametrize("name", KERNELS)
def test_each_barrier_reports_its_own_site(name):
    for bar, site in waits(name):
        assert site in SITES[bar], f"{bar} reports {site}"


def test_no_site_is_both_filled_and_free():
    kinds = collections.defaultdict(set)
    for name in KERNELS:
        for bar, site in waits(name):
            kinds[site].add("free" if re.search("free|empty", bar) else "full" if bar in ("k_full", "v_full", "q_full", "mask_full",
                                                                                          "l_full") else "other")
    assert len(kinds) > 10 and not [s for s, k in kinds.items() if {"free", "full"} <= k]
