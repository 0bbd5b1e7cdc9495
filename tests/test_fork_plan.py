"""How many blocks a fork of many takes (no GPU needed)."""
import os
import shutil

import pytest

from test_sanitizers import HERE, ROOT, _build_and_run


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_comparisons_go_with_the_copies(tmp_path):
    csrc = os.path.join(ROOT, "paged_split_kv_attn_gb300", "csrc")
    out = _build_and_run(tmp_path, "g++", [os.path.join(HERE, "fork_plan_driver.cpp"), os.path.join(csrc, "pskv_plan.cpp")],
                         [csrc, os.path.join(ROOT, "include")], "fork_plan_driver", ["-std=c++17"])
    assert "fork plan driver ok" in out
