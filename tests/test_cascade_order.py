"""What orders the cascade kernel's warps, read from its source as the prefill's is.  No GPU."""
import os

import pytest

from paged_kv_cache_75_gb300 import build as pkg_build
from test_prefill_order import (test_a_warp_leaves_its_waits_together, test_an_elected_thread_meets_no_collective,  # noqa: F401
                                test_tensor_memory_is_read_behind_a_fence, without_comments)


@pytest.fixture(scope="module")
def kernel():
    with open(os.path.join(pkg_build.CSRC, "cascade.cu")) as f:
        text = without_comments(f.read())
    text = text[text.index("cascade_kernel(const __grid_constant__"):]
    return text[:text.index("cascade_merge_kernel(")]
