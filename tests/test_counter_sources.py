"""The sources whose change makes the benchmark's counter records void: those of
the kernels that the counters measure, and no others."""
import os
import re

import bench_counters

CSRC = os.path.join(bench_counters.ROOT, "histogram_gradient_boosted_amd", "csrc")


def included(name, found):
    """Every file of csrc that `name` includes, itself among them."""
    path = os.path.join(CSRC, name)
    if name in found or not os.path.exists(path):
        return found
    found.add(name)
    with open(path, encoding="utf-8") as f:
        for other in re.findall(r'^#include "(.*)"', f.read(), re.M):
            included(other, found)
    return found


def test_the_tree_path_s_sources_and_no_others():
    names = {os.path.basename(p) for p in bench_counters.source_files()}
    want = included("hgb.hip", set()) | {"lds_rate.hip", "hgb.h"}
    assert names == want
    assert not any("vector" in n for n in names)


def test_comments_do_not_change_the_hash():
    text = "int a; // one\n/* two\nlines */ int  b;\n"
    assert bench_counters._code_only(text) == "int a; int b;"
