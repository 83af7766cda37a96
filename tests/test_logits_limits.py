"""The logit-side operators' limits on the CPU: sizes beyond what the kernels'
arithmetic holds are refused before anything is launched, in the queries and in
the plans alike."""

import ctypes as C

import pytest

from . import test_logits_abi as A

lib = A.lib  # the built library


LIST = 1 << 28


@pytest.mark.parametrize("name", ["history_ld", "bias_ld"])
def test_process_lists_end_where_counts_and_positions_fit(lib, name):
    # 2^28 entries: an occurrence count has 29 bits, and a position is stepped past the end of its list
    for n in (LIST + 1, 1 << 29, (1 << 31) - 1):
        assert lib.spec_process_logits(C.byref(A._process(**{name: n})), None) == -1
    size = lib.spec_process_workspace_size
    sizes = lambda n: (1, 4, 100, n, 0) if name == "history_ld" else (1, 4, 100, 0, n)
    assert size(*sizes(LIST)) > 0
    assert size(*sizes(LIST + 1)) == 0 and size(*sizes((1 << 31) - 1)) == 0
    # one step further: the list is accepted, and the next refusal (a workspace that is too small) is reached
    assert lib.spec_process_logits(C.byref(A._process(**{name: LIST, "workspace_bytes": 1})), None) == -4
