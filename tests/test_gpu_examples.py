"""The examples run, and what they return is consistent."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_int4_draft_step(cuda_device):
    m = load("int4_draft_step")
    for B, gamma, V, d in ((8, 4, 32000, 1024), (3, 2, 5003, 256)):
        r = m.step(B=B, gamma=gamma, V=V, d=d)
        torch.cuda.synchronize()
        assert int(r["errors"].abs().sum()) == 0 and int(r["seq_error"].abs().sum()) == 0
        a, t = r["accept_len"], r["out_token"]
        assert bool(((a >= 0) & (a <= gamma)).all()) and bool(((t >= 0) & (t < V)).all())
        # every drafted and every emitted token of a masked request is one the grammar allows
        allowed = ((r["mask"][0].repeat_interleave(32) >> (torch.arange(r["mask"].shape[1] * 32, device=t.device) % 32))
                   & 1).bool()
        for b in range(B):
            if bool(r["masked"][b]):
                assert bool(allowed[r["tokens"][b].long()].all()) and bool(allowed[int(t[b])])
        # the quantised head is near the one it was made from: some drafts are kept
        assert int(a.sum()) > 0
