"""Refusals of the step calls before anything is launched, at the borders of what they take (no GPU)."""
import pytest

import pagedattention_kv_cache_paged_gb300 as pa
from test_tree_host import TREE, call, lib  # noqa: F401  (lib: the fixture)


@pytest.mark.parametrize("scale,refused", [(2.36e38, True), (2.9e38, True), (3.0e38, True), (3.4e38, True), (2.35e38, False),
                                           (1e-45, False), (1e-30, False), (-0.0, True)])
def test_scales_that_pass_the_largest_number_in_the_log2_domain(lib, scale, refused):  # noqa: F811
    # with an empty batch the call ends before its pointers are looked at
    status = call(lib, "paged_attention_tree", list(TREE), TREE, scale=scale, batch=0)
    assert status == (pa.PA_EINVAL if refused else pa.PA_OK)
