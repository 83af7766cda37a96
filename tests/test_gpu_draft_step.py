"""The example of a draft step with a 4-bit head processes each drafted row
once, and what it gets is the chain's processing of the raw rows."""

import pytest
import torch

from .test_gpu_examples import load

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,gamma,V,d", [(8, 4, 32000, 1024), (3, 5, 5003, 256)])
def test_each_drafted_row_is_processed_once(cuda_device, monkeypatch, B, gamma, V, d):
    m = load("int4_draft_step")
    process, seen = m.dv.process_logits, []

    def spy(logits, *args, **kw):
        seen.append((logits.clone(), kw["history"].clone(), kw["history_len"].clone(), kw))
        return process(logits, *args, **kw)

    monkeypatch.setattr(m.dv, "process_logits", spy)
    r = m.step(B=B, gamma=gamma, V=V, d=d)
    assert sum(call[0].shape[1] for call in seen) == gamma + gamma + 1
    raw = torch.cat([call[0] for call in seen[:gamma]], 1)
    _, history, history_len, kw = seen[0]
    kw = {k: v for k, v in kw.items() if k not in ("out", "mask_index", "history", "history_len")}
    index = seen[-1][3]["mask_index"][:, :gamma].contiguous()
    chain = process(raw, r["tokens"], history=history, history_len=history_len, mask_index=index, **kw)["logits"]
    assert torch.equal(chain.view(torch.int16), r["q"].contiguous().view(torch.int16))
