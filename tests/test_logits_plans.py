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
