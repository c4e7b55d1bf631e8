"""pa_varlen_cascade whose copies never come: every wait runs out, the status says so, the next call is right."""
import time

import pytest
import torch

import paged_kv_cache_75_gb300 as pk
from cascade_ref import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups", [[(160, [(9, 2), (3, 1)])], [(320, [(5, 1)] * 40)], [(64, [(200, 150)] * 30)]])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_cascade(dtype, groups):
    """Stacked, with the decode kernel beside, straight to out."""
    b = Batch(groups, 32, 8, dtype, 16, 31).device()
    m, st, out = b.bounds(), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros_like(b.qd)
    t0 = time.monotonic()
    pk.pa_varlen_cascade_test_wait_timeout(out, b.qd, b.cache, b.tab, b.cu_q, b.cu_k, m["max_q"], m["max_k"], b.scale, b.cu_g,
                                           b.sh, m["max_group"], m["max_shared"], b.workspace(), st)
    torch.cuda.synchronize()
    assert 1.0 < time.monotonic() - t0 < 60.0
    assert int(st) == 5  # PA_ERR_TIMEOUT
    b.check(b.run())
