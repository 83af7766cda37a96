"""The plans of the logit-side operators on the CPU: what they allocate and
clear, and what they refuse to launch."""

import pytest
import torch

from . import test_logits_abi as A

lib = A.lib  # the built library


def product_tensors(R=128, V=300, d=256, group=64, device="cpu"):
    return (torch.zeros(R, d, dtype=torch.bfloat16, device=device),
            torch.zeros(V, d // 2, dtype=torch.uint8, device=device),
            torch.zeros(d // group, V, dtype=torch.bfloat16, device=device))


def test_product_plan_clears_its_counters_alone(lib, monkeypatch):
    """20 MB of partial sums need no clearing: what of a workspace full of ones is zero afterwards."""
    from draft_verification_gb300 import Int4ProductPlan
    tensors, cleared = product_tensors(), []
    zeros, empty = torch.zeros, torch.empty
    monkeypatch.setattr(torch, "zeros", lambda *s, **k: (cleared.append(zeros(*s, **k)), cleared[-1])[1])
    monkeypatch.setattr(torch, "empty", lambda *s, **k: empty(*s, **k).fill_(1))
    plan = Int4ProductPlan(*tensors, group=64)
    assert sum(t.numel() * t.element_size() for t in cleared) <= 1024
    assert plan.workspace.numel() > 1 << 20
    assert not plan.workspace[:1024].any() and bool((plan.workspace[1024:] == 1).all())


def plans():
    import draft_verification_gb300 as dv
    return [lambda **k: dv.ProcessLogitsPlan(torch.zeros(2, 3, 50), **k),
            lambda **k: dv.Int4ProductPlan(*product_tensors(), group=64, **k),
            lambda **k: dv.QuantizeInt4Plan(torch.zeros(50, 128), **k)]


def test_plans_of_host_tensors_launch_nothing(lib):
    for make in plans():
        with pytest.raises(ValueError, match="CUDA tensors"):
            make().run()


def test_plans_check_their_workspace(lib):
    for make in plans()[:2]:
        need = make().workspace.numel()
        for elsewhere in (torch.zeros(need, dtype=torch.uint8, device="meta"),
                          torch.zeros(2 * need, dtype=torch.uint8)[::2]):
            with pytest.raises(ValueError):
                make(workspace=elsewhere)
        # counted in bytes, whatever the elements
        assert make(workspace=torch.zeros((need + 7) // 8, dtype=torch.int64)).args.workspace_bytes >= need


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [50, 56, 1001])
def test_process_plan_allocates_what_its_rows_need(lib, dtype, V):
    """One position of many, and columns of a wider matrix: the output takes rows, not the memory between them."""
    from draft_verification_gb300 import ProcessLogitsPlan
    E = 16 // dtype.itemsize
    wide = torch.zeros(4, 9, V, dtype=dtype)
    for logits in (wide[:, :1], wide[:, 8:], torch.zeros(4, 3, 5 * V + 3, dtype=dtype)[:, :, :V]):
        plan = ProcessLogitsPlan(logits)
        out = plan.out["logits"]
        assert out.shape == logits.shape and out.stride(2) == 1
        assert out.untyped_storage().nbytes() <= logits.shape[0] * logits.shape[1] * (V + E - 1) * dtype.itemsize
        assert (plan.args.out_ld - plan.args.ld) % E == 0 and plan.args.out_ld >= V  # rows start alike
    # ordinary rows keep their stride, as a verification of both sides' rows wants it
    for logits in (wide, torch.zeros(4, 3, V + 5, dtype=dtype)[:, :, :V]):
        assert ProcessLogitsPlan(logits).out["logits"].stride() == logits.stride()
