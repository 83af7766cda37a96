"""int4_product's bounded waits give up together.

The test hook (spec_test_inject_product_copy_timeout) makes every stage of
weights wait for 16 bytes that never come: the copies themselves land, the
stage's barrier phase stays open, and the roles that wait for it, or for one
another, end after the poll limit (about 65 ms, then a bounded wait for the
stages issued) with an error bit, never a hang or a fault."""

import pytest
import torch

from . import test_gpu_logits as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,V,d,group,zeros", [
    (1, 100, 256, 128, False),     # one CTA, one unit
    (5, 1000, 8192, 128, True),    # every tile is shared
    (20, 3001, 1056, 32, True),
    (33, 2500, 2048, 64, True),
    (128, 20000, 1024, 128, False),
    (300, 260, 192, 64, True),
])
def test_product_waits_give_up_with_internal_error(cuda_device, R, V, d, group, zeros):
    import draft_verification_gb300 as dv
    from draft_verification_gb300 import _lib
    lib = _lib.lib()
    x, codes, scales, z = T.make_product(R, V, d, group, zeros, 61 + R, cuda_device)
    plan = dv.Int4ProductPlan(x, codes, scales, z, group=group, out_dtype=torch.float32)
    plan.out["logits"].fill_(7.0)
    torch.cuda.synchronize()
    assert lib.spec_test_inject_product_copy_timeout(1) == _lib.SPEC_OK
    try:
        out = plan.run()
    finally:
        assert lib.spec_test_inject_product_copy_timeout(0) == _lib.SPEC_OK
    torch.cuda.synchronize()
    assert int(out["error_word"]) == dv.ERR_INTERNAL
    assert bool((out["logits"] == 7.0).all())
    # the GPU is as it was: the same plan, the hook off, is right
    plan.reset()
    out = plan.run()
    torch.cuda.synchronize()
    assert int(out["error_word"]) == 0
    T.check_product(out["logits"], x, codes, scales, z, group)
