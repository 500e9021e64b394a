"""Host build of the planning of attention over shared prefixes and selected blocks under AddressSanitizer and
UndefinedBehaviorSanitizer (no GPU needed): tests/sanitize/prefix_plan_check.cpp drives
ultra_bit_weight_uint32_amd/csrc/cache_plan.h over random and edge shapes."""
import os

import pytest

from test_sanitizers import HERE, SAN, _build_and_run, _have


@pytest.mark.skipif(not _have("g++"), reason="g++ not found")
def test_prefix_plan_under_sanitizers(tmp_path):
    src = os.path.join(HERE, "sanitize", "prefix_plan_check.cpp")
    _build_and_run(tmp_path, ["g++", "-std=c++17", "-Wall", "-Wextra"] + SAN + [src], tmp_path / "prefix_plan_check")
