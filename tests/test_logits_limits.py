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


def test_product_sizes_end_where_its_units_can_be_counted(lib):
    # 2^30 units of 128 rows x 128 entries x 256 columns: refused, which the query says as well
    size = lib.spec_int4_product_workspace_size
    most = dict(V=2097152, d=65536, group=128, codes_ld=32768, x_ld=65536, scales_ld=2097152, zeros_ld=2097152,
                out_ld=2097152)
    assert size(255 * 128, 2097152, 65536, 128) > 0
    for R in (255 * 128 + 1, 256 * 128, 65535):
        assert size(R, 2097152, 65536, 128) == 0
        assert lib.spec_int4_product(C.byref(A._product(R=R, **most)), None) == -1
    assert size(65535, 1048576, 65536, 128) == 0 and size(65535, 1048448, 65536, 128) > 0
