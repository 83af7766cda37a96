"""What the cache operators write to: outputs whose elements lie in places of their own, and error words."""

import itertools

import pytest
import torch

import draft_verification_gb300 as dv


def view(shape, strides):
    size = 1 + sum((n - 1) * s for n, s in zip(shape, strides))
    return torch.zeros(size, dtype=torch.bfloat16).as_strided(shape, strides)


def places(shape, strides):
    return [sum(i * s for i, s in zip(at, strides)) for at in itertools.product(*map(range, shape))]


@pytest.mark.parametrize("shape,strides", [
    ((2, 3, 1, 4), (9, 4, 4, 1)),      # the second sequence's first row begins in the first one's last
    ((2, 3, 2, 4), (100, 20, 21, 1)),  # heads that begin within one another
    ((2, 2, 2, 2), (10, 6, 4, 1)),     # 6 + 4 leads where 10 does
    ((3, 2, 2, 2), (0, 8, 4, 1)),
    ((2, 3, 4, 8), (96, 32, 8, 1)), ((2, 3, 4, 8), (8, 64, 16, 1)), ((2, 3, 4, 8), (1000, 8, 24, 1)),
    ((2, 2, 2, 2), (102, 100, 4, 1)),  # rows between one another's heads, none in the same place
    ((2, 3, 1, 2), (6, 4, 1, 1)), ((1, 3, 1, 4), (0, 4, 0, 1)),
])
def test_rotated_heads_lie_apart(shape, strides):
    at = places(shape, strides)
    x, out, table = torch.zeros(shape, dtype=torch.bfloat16), view(shape, strides), torch.zeros(5, 2)
    if len(set(at)) == len(at):
        dv.RotateHeadsPlan(x, table, out=out)
    else:
        with pytest.raises(ValueError, match="elements overlap"):
            dv.RotateHeadsPlan(x, table, out=out)


def test_attended_heads_lie_apart():
    cache = dv.PagedCache.empty(4, 1, 16, 16, device="cpu")
    q, pages = torch.zeros((2, 3, 1, 16), dtype=torch.bfloat16), torch.zeros((2, 4), dtype=torch.int32)
    dv.AttendCachePlan(q, cache, pages, out=view((2, 3, 1, 16), (48, 16, 16, 1)))
    with pytest.raises(ValueError, match="elements overlap"):
        dv.AttendCachePlan(q, cache, pages, out=view((2, 3, 1, 16), (33, 16, 16, 1)))


def test_error_words_of_plans_on_host_tensors():
    """(Such plans refuse to run.)"""
    cache = dv.PagedCache.empty(4, 1, 16, 16, device="cpu")
    x, pages = torch.zeros((2, 3, 1, 16), dtype=torch.bfloat16), torch.zeros((2, 4), dtype=torch.int32)
    for plan in (dv.RotateHeadsPlan(x, torch.zeros(5, 16)), dv.AppendCachePlan(x, x, cache, pages),
                 dv.AttendCachePlan(x, cache, pages)):
        assert plan.out["seq_error"].tolist() == [0, 0] and plan.out["error_word"].tolist() == [0]
        plan.out["seq_error"][1], plan.out["error_word"][0] = 2, 3
        assert plan.out["seq_error"].tolist() == [0, 2] and plan.out["error_word"].tolist() == [3]
        plan.clear_errors()
        assert not plan.out["seq_error"].any() and not plan.out["error_word"].any()
