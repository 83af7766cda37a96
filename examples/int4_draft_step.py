"""One speculative step with a 4-bit draft head and per-request logit
processing: quantise the draft model's LM head once, draft gamma tokens from
its products, process every row with the tokens before its own position
(penalties, biases, a grammar mask), and verify the drafts against the target
rows processed in the same way.

The hidden states and weights are synthetic: what is shown is the calls.

    python examples/int4_draft_step.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import draft_verification_gb300 as dv  # noqa: E402


def draw(logits, temperature, g):
    """One token per sequence from softmax(logits / T), as the verification assumes of drafts."""
    noise = -torch.log(-torch.log(torch.rand(logits.shape, generator=g, device=logits.device)))
    return (logits.float() / temperature + noise).argmax(-1).to(torch.int32)


def step(B=8, gamma=4, V=32000, d=1024, group=128, temperature=0.8, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    f32 = lambda *s: torch.randn(*s, generator=g, device=device)
    uni = lambda *s: torch.rand(*s, generator=g, device=device)

    # once, when the draft model is loaded
    w_draft = (f32(V, d) * 0.1).bfloat16()
    head = dv.quantize_int4(w_draft, group=group)

    # per request: history (the first half is the prompt) with room for the drafted tokens, penalties, a biased token,
    # a grammar
    H = 64
    history = torch.zeros((B, H + gamma), dtype=torch.int32, device=device)
    history[:, :H] = torch.randint(0, V, (B, H), generator=g, device=device, dtype=torch.int32)
    history_len = torch.full((B,), H, dtype=torch.int32, device=device)
    request = dict(
        history=history, prompt_len=torch.full((B,), H // 2, dtype=torch.int32, device=device),
        repetition=torch.full((B,), 1.1, device=device), frequency=torch.full((B,), 0.2, device=device),
        presence=torch.full((B,), 0.1, device=device),
        bias_tokens=torch.full((B, 1), 7, dtype=torch.int32, device=device),
        bias_values=torch.full((B, 1), 2.0, device=device))
    words = (V + 31) // 32
    mask = torch.randint(-2 ** 31, 2 ** 31, (1, words), generator=g, device=device, dtype=torch.int64).to(torch.int32)
    half = torch.arange(B, device=device, dtype=torch.int32).view(B, 1) % 2 - 1  # every other request has the grammar

    # logits whose rows all start on 16 bytes, so that a position's rows can be processed where they are
    rows = lambda n: torch.empty((B, n, (V + 7) // 8 * 8), dtype=torch.bfloat16, device=device)[:, :, :V]

    # draft gamma tokens one after another: a position's row follows the history and the tokens drafted before it,
    # which are appended to the history
    hidden = f32(B, gamma, d).bfloat16()
    tokens = torch.zeros((B, gamma), dtype=torch.int32, device=device)
    draft, so_far = rows(gamma), history_len.clone()
    errors = torch.zeros_like(history_len)
    for i in range(gamma):
        dv.Int4ProductPlan(hidden[:, i], head["codes"], head["scales"], group=group, out=draft[:, i]).run()
        row = draft[:, i:i + 1]
        errors |= dv.process_logits(row, history_len=so_far, mask=mask, mask_index=half, out=row,
                                    **request)["seq_error"]
        tokens[:, i] = history[:, H + i] = draw(row[:, 0], temperature, g)
        so_far += 1

    # the target's rows at the gamma + 1 positions (here: the unquantised head), processed alike: a chain's rows
    # follow the history before the step and the drafted tokens before their own positions
    target = rows(gamma + 1)
    target[:, :gamma] = hidden @ w_draft.t()
    target[:, gamma] = f32(B, d).bfloat16() @ w_draft.t()
    p = dv.process_logits(target, tokens, history_len=history_len, mask=mask,
                          mask_index=half.expand(B, gamma + 1).contiguous(), out=target, **request)

    out = dv.verify_chain(target, draft, tokens, uni(B, gamma), uni(B), history_len, temperature=temperature)
    return dict(tokens=tokens, q=draft, p=target, mask=mask, masked=half[:, 0] >= 0, errors=errors | p["seq_error"],
                **out)


if __name__ == "__main__":
    r = step()
    for b in range(len(r["tokens"])):
        print(f"sequence {b}: drafted {r['tokens'][b].tolist()}, kept {int(r['accept_len'][b])}, "
              f"then {int(r['out_token'][b])}, rollback to {int(r['rollback_idx'][b])}")
