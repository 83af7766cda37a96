"""Plans of the cache operators that are made, cleared and run on different streams, and in graphs."""

import pytest
import torch

import draft_verification_gb300 as dv

pytestmark = pytest.mark.gpu

B, N, H, D, PAGE = 3, 4, 2, 64, 16


def inputs(device):
    x = torch.ones((B, N, H, D), dtype=torch.bfloat16, device=device)
    at = torch.zeros((B, N), dtype=torch.int32, device=device)
    at[1, 2] = 99  # not in the table
    pages = torch.arange(B, dtype=torch.int32, device=device).view(B, 1)
    pages[1] = 7  # not in the cache
    return x, at, pages, dv.rotation_table(10, D, device=device), dv.PagedCache.empty(B, H, PAGE, D, device=device)


MAKE = {
    "rotate": lambda x, at, pages, table, cache: dv.RotateHeadsPlan(x, table, positions=at),
    "append": lambda x, at, pages, table, cache: dv.AppendCachePlan(x, x, cache, pages, table=table),
    "attend": lambda x, at, pages, table, cache: dv.AttendCachePlan(x, cache, pages),
}
BIT = {"rotate": dv.ERR_POSITION, "append": dv.ERR_CACHE, "attend": dv.ERR_CACHE}


def delay():
    torch.cuda._sleep(100_000_000)  # about 50 ms on the current stream


def check(plan, kind):
    torch.cuda.synchronize()
    assert plan.out["seq_error"].tolist() == [0, BIT[kind], 0] and plan.out["error_word"].tolist() == [BIT[kind]]


@pytest.mark.parametrize("kind", MAKE)
def test_runs_come_behind_making_and_clearing(cuda_device, kind):
    """A stream that does not wait for the one that zeroes the error words would have its bits wiped."""
    given = inputs(cuda_device)
    MAKE[kind](*given).run()  # (modules and memory are there from here on)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    delay()
    plan = MAKE[kind](*given)
    plan.run(side)
    check(plan, kind)
    delay()
    plan.clear_errors()
    plan.run(side)
    check(plan, kind)
    with torch.cuda.stream(other):
        delay()
    plan.clear_errors(other)
    plan.run()
    check(plan, kind)
    with torch.cuda.stream(other):
        delay()
        plan.clear_errors()
    with torch.cuda.stream(side):
        plan.run()
    check(plan, kind)


@pytest.mark.parametrize("kind", MAKE)
def test_captured_runs_of_plans_made_elsewhere(cuda_device, kind):
    given = inputs(cuda_device)
    plan = MAKE[kind](*given)
    plan.run()
    delay()
    plan.clear_errors()
    graph, fork = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        plan.run()
        fork.wait_stream(torch.cuda.current_stream())
        plan.run(fork)
        torch.cuda.current_stream().wait_stream(fork)
    torch.cuda.synchronize()
    assert not plan.out["error_word"].any()
    graph.replay()
    check(plan, kind)
    # a clearing in a graph is part of its replays, and the plan goes on as it was
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        plan.clear_errors()
    check(plan, kind)
    delay()
    plan.clear_errors()
    plan.run(fork)
    check(plan, kind)


@pytest.mark.parametrize("kind", MAKE)
def test_a_plan_made_in_a_capture(cuda_device, kind):
    given = inputs(cuda_device)
    MAKE[kind](*given).run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = MAKE[kind](*given)
        plan.run()
    for _ in range(2):
        graph.replay()
        check(plan, kind)
