"""The oracle of the cache operators, pinned by other means: the e4m3 type of
torch, complex multiplication, dense softmax attention, worked numbers."""

import numpy as np
import pytest
import torch

from oracle import cache as O


def test_e4m3_is_torchs():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    theirs = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.VALUES, theirs, equal_nan=True)
    assert O.VALUES[0x7E] == 448 and O.VALUES[0x38] == 1 and O.VALUES[1] == 2.0 ** -9
    x = np.concatenate([np.random.default_rng(0).normal(0, 60, 20000), 2.0 ** np.linspace(-14, 8.8, 5000),
                        (O.VALUES[:126] + O.VALUES[1:127]) / 2, [0.0, -0.0, 448.0, -448.0]])
    theirs = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    keep = np.abs(x) <= 448
    assert np.array_equal(O.VALUES[O.to_e4m3(x)][keep], theirs[keep])
    assert np.isnan(O.VALUES[O.to_e4m3([449.0, np.inf, np.nan])]).all()


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_is_a_complex_product(pairs):
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1, (2, 3, 4, 16)).astype(np.float32)
    freq = 10.0 ** -np.arange(6)
    table = O.rotation_table(50, freq, magnitude=1.5)
    at = np.array([[0, 49, 7], [3, 3, 20]])
    y, err = O.rotate_heads(x, table, at, pairs=pairs)
    turn = 1.5 * np.exp(1j * at[..., None] * freq)[:, :, None]
    a, b = (x[..., 0:12:2], x[..., 1:12:2]) if pairs else (x[..., :6], x[..., 6:12])
    z = (a + 1j * b) * turn
    got = (y[..., 0:12:2], y[..., 1:12:2]) if pairs else (y[..., :6], y[..., 6:12])
    # table entries, two products and a sum: at most four half steps of the magnitudes
    assert np.abs(got[0] + 1j * got[1] - z).max() <= 8 * 2.0 ** -24 * 1.5 * np.abs(x).max() * 2
    assert np.array_equal(y[..., 12:], x[..., 12:]) and not err.any()
    back, _ = O.rotate_heads(y / np.float32(1.5 ** 2), table, at, pairs=pairs, transpose=True)
    assert np.allclose(back[..., :12], x[..., :12], atol=1e-5)
    _, err = O.rotate_heads(x, table, np.where(at == 49, 50, at), pairs=pairs)
    assert list(err) == [O.ERR_POSITION, 0]


def test_exponents():
    assert O.exponent_of([128.0, -3.0]) == 0 and O.exponent_of([128.5]) == 1 and O.exponent_of([64.0]) == -1
    assert O.exponent_of([0.0]) == O.LOW and O.exponent_of([np.nan, np.inf, 2.0]) == -6
    assert O.exponent_of([1e38]) == O.HIGH


def test_append_worked_numbers():
    cache = dict(k_codes=np.zeros((3, 1, 16, 16), np.uint8), v_codes=np.zeros((3, 1, 16, 16), np.uint8),
                 k_exps=np.zeros((3, 1), np.int8), v_exps=np.zeros((3, 1), np.int8))
    cache["v_codes"][2, 0, 0, 0] = 0x38  # a token already there: 1.0
    k = np.ones((1, 2, 1, 16))
    v = np.full((1, 2, 1, 16), 200.0)
    out, err = O.append_cache(k, v, cache, np.array([[2, 0]]), prefix_len=[1])
    assert not err.any()
    # keys: the page's exponent 0 stays (it holds a token), 1 is 0x38; values: 200 needs exponent 1
    assert out["k_exps"][2, 0] == 0 and (out["k_codes"][2, 0, 1:3] == 0x38).all()
    assert out["v_exps"][2, 0] == 1 and O.VALUES[out["v_codes"][2, 0, 0, 0]] == 0.5
    # 100 is half way between 96 = 12 * 8 and 104 = 13 * 8: the even one
    assert (O.VALUES[out["v_codes"][2, 0, 1:3]] * 2 == 192).all()
    assert (out["k_codes"][2, 0, 3:] == 0).all() and (out["k_codes"][:2] == 0).all()


def test_attention_is_a_masked_softmax():
    rng = np.random.default_rng(2)
    B, n, Hq, H, D, page = 2, 5, 4, 2, 16, 16
    cache = {f"{m}_codes": rng.integers(0, 120, (9, H, page, D)).astype(np.uint8) for m in "kv"}
    cache.update({f"{m}_exps": rng.integers(-8, -3, (9, H)).astype(np.int8) for m in "kv"})
    table = rng.permutation(9)[:8].reshape(2, 4)
    q = rng.normal(0, 0.1, (B, n, Hq, D))
    past = np.array([0, 37])
    parent = np.array([[-1, 0, 0, 1, 3], [-1, 0, 1, 1, 0]])
    for tree in (None, parent):
        out, bound, err = O.attend_cache(q, cache, table, past, parent=tree)
        assert not err.any()
        for b in range(B):
            k = torch.from_numpy(O.cache_values(cache["k_codes"], cache["k_exps"])[table[b]]).transpose(0, 1)
            v = torch.from_numpy(O.cache_values(cache["v_codes"], cache["v_exps"])[table[b]]).transpose(0, 1)
            k, v = (x.reshape(H, -1, D)[:, :past[b] + n].repeat_interleave(2, 0) for x in (k, v))
            mask = torch.ones(n, past[b] + n, dtype=torch.bool)
            own = torch.eye(n, dtype=torch.bool) if tree is not None else torch.ones(n, n).tril().bool()
            if tree is not None:
                for i in range(1, n):
                    own[i] |= own[tree[b, i]]
            mask[:, past[b]:] = own
            want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[b]).transpose(0, 1), k, v, mask)
            assert np.allclose(out[b], want.transpose(0, 1).numpy(), atol=1e-12)
        assert (bound["mass"] >= np.abs(out) - 1e-12).all()
    _, _, err = O.attend_cache(q, cache, table, [60, -1], count=[5, 5])
    assert list(err) == [O.ERR_CACHE, O.ERR_CACHE]
