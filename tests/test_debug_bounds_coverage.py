"""CPU: the kernels that the bounds-checking build is run for do check their indices. A kernel without a check
would pass those runs whatever it did."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differential_attention_v2_b200", "csrc")


def _function(file, name):
    """The text of a function at the top level of a source file."""
    for chunk in re.split(r"^}\s*$", open(os.path.join(CSRC, file)).read(), flags=re.M):
        head = re.search(rf"\b{name}\([^;{{}}]*\)\s*\{{\n", chunk)
        if head:
            return chunk[head.start():]
    raise AssertionError(f"{name} is not in {file}")


KERNELS = {
    "rope.cu": ["rope_kernel", "walk", "cache_row"],
    "cache_pages.cu": ["extend_kernel", "fork_kernel", "trim_kernel", "free_kernel", "compact_kernel", "copy_kernel"],
    "backward_sm100.cu": ["preprocess_sink_kernel", "dkdv_cta", "dq_cta", "sum_parts_kernel"],
    "decode_sink_sm100.cu": ["decode_sink_kernel"],
    "prefill_sm100.cu": ["diffattn_prefill_sm100"],
}


@pytest.mark.parametrize("file", KERNELS)
def test_every_kernel_checks_its_indices(file):
    for kernel in KERNELS[file]:
        body = _function(file, kernel)
        assert "checked(" in body, kernel
        if kernel.endswith("_kernel") or "_sm100" in kernel:
            assert re.search(r"\berr\b", body), f"{kernel} has no error word to report to"


def test_launches_hand_over_the_error_word():
    """The word that each check reports to is the device's in that build."""
    for op in ("extend", "fork", "trim", "free", "compact", "copy_pages"):
        body = _function("cache_pages.cu", f"launch_cache_{op}")
        assert "bounds_error_word(&err)" in body and re.search(r"\berr\);", body), op
    api = open(os.path.join(CSRC, "api_cache.cu")).read()
    assert api.count("bounds_error_word(&p.err)") == api.count("launch_rope(p,") == 2
