"""attend_cache's bounded waits give up together.

The test hook (spec_test_inject_cache_copy_timeout) makes every tile wait for
16 bytes that never come: the copies themselves land, the tile's barrier phase
stays open, and the roles that wait for it, or for one another, end after the
poll limit (about 65 ms, then a bounded wait for the tiles issued) with an
error bit, never a hang or a fault."""

import numpy as np
import pytest
import torch

from . import test_gpu_cache as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,Hq,D,prefix,tree", [
    (1, 2, 64, (40,), False),                # one tile per head
    (6, 8, 128, (700, 3, 1500), False),      # two CTAs per SM, blocks that CTAs share
    (12, 8, 128, (3001, 500), True),
    (64, 8, 128, (300, 64), True),           # several blocks
    (3, 8, 256, (500, 129), False),
])
def test_attend_waits_give_up_with_internal_error(cuda_device, n, Hq, D, prefix, tree):
    import draft_verification_gb300 as dv
    from draft_verification_gb300 import _lib
    lib = _lib.lib()
    w = T.make_attend(np.random.default_rng(n), len(prefix), n, Hq, 2, D, 64, prefix, tree)
    plan = dv.AttendCachePlan(T.dev(w["q"]).bfloat16(), T.on_gpu(w["c"]), T.dev(w["table"]), T.dev(w["prefix"]),
                              parent=T.dev(w["parent"]))
    torch.cuda.synchronize()
    assert lib.spec_test_inject_cache_copy_timeout(1) == _lib.SPEC_OK
    try:
        out = plan.run()
    finally:
        assert lib.spec_test_inject_cache_copy_timeout(0) == _lib.SPEC_OK
    torch.cuda.synchronize()
    assert int(out["error_word"]) == dv.ERR_INTERNAL
    # the GPU is as it was: the same plan, the hook off, is right
    plan.clear_errors()
    out = plan.run()
    torch.cuda.synchronize()
    assert int(out["error_word"]) == 0
    T.check_attend(w, out)
