"""The sites that bounded waits of the cache operators report
(fa_debug_last_wait_site): a wait for a buffer to be free never reports the
site of a wait for one to be filled, or a timeout would name the wrong side."""
import collections
import os
import re

from exact_attention_48_gb300 import build as fa_build


def test_free_and_full_waits_have_their_own_sites():
    sites = collections.defaultdict(lambda: collections.defaultdict(list))
    for name in ("fa_tree.cu", "fa_key_weights.cu"):
        with open(os.path.join(fa_build.CSRC, name), encoding="utf-8") as f:
            for bar, site in re.findall(r"mbar_wait\(\s*&?(?:a\.)?(\w+)[^;]*?\b(kSite\w+)\)", f.read()):
                kind = "free" if re.search("free|empty", bar) else "full" if "full" in bar else "other"
                sites[site][kind].append((name, bar))
    assert sum(len(x) for kinds in sites.values() for x in kinds.values()) > 20
    for site, kinds in sites.items():
        assert not (kinds["free"] and kinds["full"]), f"{site}: {kinds['free']} and {kinds['full']}"
