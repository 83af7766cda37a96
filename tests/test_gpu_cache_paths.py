"""Lengths of kept paths at the ends of the integers."""

import numpy as np
import pytest

import draft_verification_gb300 as dv
from oracle import cache as O

from . import test_gpu_cache as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("depth", [0, 3])
def test_append_path_lengths_out_of_range(cuda_device, depth):
    rng = np.random.default_rng(40 + depth)
    length = np.array([2 ** 31 - 1, -1, -2 ** 31, depth + 1, depth, 2 ** 31 - 2, 0], np.int32)
    B, n, H, D, page = len(length), 6, 2, 32, 16
    k, v = (T.rounded(rng.normal(0, 1, (B, n, H, D)), "bf16") for _ in range(2))
    path = np.tile(np.arange(depth + 1, dtype=np.int32), (B, 1))
    prefix = np.full(B, 14, np.int32)
    table = rng.permutation(2 * B).reshape(B, 2).astype(np.int32)
    c = T.make_cache(rng, 2 * B, H, page, D)
    want, err = O.append_cache(k, v, c, table, prefix, path_nodes=path, path_len=length)
    assert list(err) == [dv.ERR_CACHE] * 4 + [0, dv.ERR_CACHE, 0]
    got = T.on_gpu(c)
    out = dv.append_cache(T.dev(k).bfloat16(), T.dev(v).bfloat16(), got, T.dev(table), T.dev(prefix),
                          path_nodes=T.dev(path), path_len=T.dev(length))
    T.check_cache(got, want)
    assert np.array_equal(out["seq_error"].cpu().numpy(), err)
