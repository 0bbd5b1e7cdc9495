"""sample_tokens' search for a border, on the host: its guesses, its result and how many passes it takes (no GPU needed)."""
import os
import re
import shutil

import pytest

from test_sanitizers import HERE, ROOT, _build_and_run


@pytest.fixture(scope="module")
def passes(tmp_path_factory):
    """Passes -> rows, of 8,000 peaked, flat, tied and masked rows; the driver checks each one's border."""
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    csrc = os.path.join(ROOT, "paged_split_kv_attn_gb300", "csrc")
    out = _build_and_run(tmp_path_factory.mktemp("search"), "g++", [os.path.join(HERE, "sample_search_driver.cpp")], [csrc],
                         "sample_search_driver", ["-std=c++17"])
    assert "sample search driver ok" in out
    return {int(p): int(n) for p, n in re.findall(r"(\d+) passes: (\d+) rows", out)}


def test_guesses_go_on_from_where_the_exact_sum_ends_and_borders_are_right(passes):
    assert sum(passes.values()) == 8000


def test_most_searches_are_short(passes):
    assert max(passes) <= 48
    assert sum(n for p, n in passes.items() if p <= 5) >= 0.97 * 8000
