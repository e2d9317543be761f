"""The traffic figures of bench.py retire with any code of the step kernel that changes."""

import os
import re

import bench

CSRC = os.path.join(os.path.dirname(os.path.abspath(bench.__file__)), "query_aware_sparse_page_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return f.read()


def test_hash_covers_what_the_step_kernel_is_built_from():
    seen, todo = set(), ["spg_fused.cu"]
    while todo:
        f = todo.pop()
        if f not in seen and os.path.exists(os.path.join(CSRC, f)):
            seen.add(f)
            todo += re.findall(r'#include "([^"]+)"', _code(f))
    # and the file that makes its tensor maps
    makers = {f for f in os.listdir(CSRC) if re.search(r"^bool make_kv_tmap\([^;]*\{", _code(f), re.M)}
    assert makers and seen | makers == set(bench.STEP_SOURCES)
