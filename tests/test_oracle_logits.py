"""Pins of oracle/logits.py: hand-worked examples, closed forms, and planted
mistakes that the examples catch."""

import numpy as np

from oracle import logits as O


def test_chain_example():
    # one sequence, three rows, five tokens.  history: prompt [0], generated [1, 1]; drafted [2, 1]
    x = np.array([[[2.0, 2.0, -1.0, 3.0, 0.5]] * 3])
    y, touched, _, err = O.process_logits(
        x, np.array([[2, 1]]), history=np.array([[0, 1, 1]]), prompt_len=np.array([1]),
        repetition=np.array([2.0]), frequency=np.array([0.25]), presence=np.array([1.0]),
        bias_tokens=np.array([[3, 3]]), bias_values=np.array([[0.5, -2.0]]))
    # token 0: prompt only -> repetition alone; token 1: 2 then 2, 2, 3 occurrences; token 2 from row 1 on
    want = [[1.0, 1.0 - 1.5, -1.0, 1.5, 0.5],
            [1.0, 1.0 - 1.5, -2.0 - 1.25, 1.5, 0.5],
            [1.0, 1.0 - 1.75, -2.0 - 1.25, 1.5, 0.5]]
    assert np.array_equal(y[0], want) and err[0] == 0
    assert touched[0].tolist() == [[True, True, False, True, False]] + [[True, True, True, True, False]] * 2


def test_tree_example_and_mask():
    # node 0 root; 1 and 2 its children; 3 a child of 1
    x = np.zeros((1, 4, 6))
    parent = np.array([[-1, 0, 0, 1]])
    tokens = np.array([[5, 1, 2, 1]])  # the root's entry is not read
    mask = np.array([[0b110111], [0]], np.int32)
    y, _, _, err = O.process_logits(x, tokens, parent, presence=np.array([1.0]), frequency=np.array([1.0]),
                                    mask=mask, mask_index=np.array([[-1, 0, -1, 1]]))
    inf = -np.inf
    assert err[0] == 0
    assert np.array_equal(y[0, 0], [0, 0, 0, 0, 0, 0])
    assert np.array_equal(y[0, 1], [0, -2, 0, inf, 0, 0])
    assert np.array_equal(y[0, 2], [0, 0, -2, 0, 0, 0])
    assert np.array_equal(y[0, 3], [inf] * 6)
    y, _, _, _ = O.process_logits(x, tokens, parent, presence=np.array([1.0]), frequency=np.array([1.0]))
    assert np.array_equal(y[0, 3], [0, -3, 0, 0, 0, 0])


def test_a_chain_shaped_tree_is_the_chain():
    rng = np.random.default_rng(0)
    n, V = 9, 12
    x = rng.normal(size=(2, n, V))
    tok = rng.integers(0, V, (2, n))
    kw = dict(repetition=np.array([1.5, 0.5]), frequency=np.array([0.3, -0.1]), presence=np.array([0.0, 1.0]))
    parent = np.tile(np.arange(-1, n - 1), (2, 1))
    chain = O.process_logits(x, tok[:, 1:], **kw)[0]
    assert np.array_equal(chain, O.process_logits(x, tok, parent, **kw)[0])


def test_process_errors():
    x = np.zeros((1, 3, 4))
    run = lambda **kw: int(O.process_logits(x, **kw)[3][0])
    assert run(tokens=np.array([[0, 4]])) == O.ERR_TOKEN
    assert run(tokens=np.array([[0, 1, 9]])) == 0  # a chain of 3 rows reads two drafted tokens
    assert run(history=np.array([[-1, 2]])) == O.ERR_TOKEN
    assert run(history=np.array([[-1, 2]]), history_len=np.array([0])) == 0
    assert run(history=np.array([[1]]), history_len=np.array([2])) == O.ERR_TOKEN
    assert run(bias_tokens=np.array([[4]]), bias_values=np.array([[1.0]])) == O.ERR_TOKEN
    assert run(tokens=np.array([[0, 1, 1]]), parent=np.array([[-1, 0, 2]])) == O.ERR_PARENT
    assert run(mask=np.array([[1]], np.int32), mask_index=np.array([[0, 1, -1]])) == O.ERR_MASK


def test_quantize_example():
    w = np.zeros((1, 32), np.float32)
    w[0, :5] = [7.0, -7.0, 0.5, 1.5, -2.5]  # scale 1: ties go to even
    codes, scales, _ = O.quantize_int4(w, 32, False)
    assert O.bf16_values(scales)[0, 0] == 1.0
    q = np.stack([codes & 15, codes >> 4], 2).reshape(-1).astype(int) - 8
    assert q[:6].tolist() == [7, -7, 0, 2, -2, 0]
    w[0, :4] = [10.0, -5.0, 0.5, 0.0]
    w[0, 4] = 0
    codes, scales, zeros = O.quantize_int4(w, 32, True)
    q = np.stack([codes & 15, codes >> 4], 2).reshape(-1)
    assert O.bf16_values(scales)[0, 0] == 1.0 and zeros[0, 0] == 5
    assert q[:4].tolist() == [15, 0, 5, 5]


def test_quantize_is_within_half_a_step():
    rng = np.random.default_rng(1)
    w = rng.normal(size=(20, 256)).astype(np.float32)
    for group in (32, 64, 128):
        for with_zeros in (False, True):
            codes, scales, zeros = O.quantize_int4(w, group, with_zeros)
            s = np.repeat(O.bf16_values(scales).T, group, axis=1)
            back = O.int4_weights(codes, scales, zeros, group)
            # half a step, and what the rounding of s (2^-8) and of z (half a step) moves the ends by
            assert (np.abs(back - w) <= s * (0.5 + 15 * 2.0 ** -8 + (0.5 if with_zeros else 0.0))).all()


def test_quantize_zero_and_non_finite_groups():
    w = np.zeros((3, 64), np.float32)
    w[1, 3] = np.inf
    w[2, 40] = np.nan
    for with_zeros in (False, True):
        codes, scales, zeros = O.quantize_int4(w, 32, with_zeros)
        v = O.bf16_values(scales)
        assert v[0, 0] == 0 and np.isnan(v[0, 1]) and np.isnan(v[1, 2]) and v[0, 2] == 0
        assert (codes == (0x00 if with_zeros else 0x88)).all()


def test_product_example_and_bound():
    codes = np.array([[0x9A] * 16, [0x08] * 16], np.uint8)  # low nibbles first: 2, 1, 2, 1 ... and 0, -8 ...
    scales = O.to_bf16(np.array([[0.5, 2.0]], np.float32))
    x = np.arange(32, dtype=np.float64)[None]
    y, mag = O.int4_product(x, codes, scales, None, 32)
    even, odd = x[0, 0::2].sum(), x[0, 1::2].sum()
    assert y[0, 0] == 0.5 * (2 * even + odd) and y[0, 1] == 2.0 * (-8 * odd)
    assert np.array_equal(mag, np.abs(y))


def test_planted_mistakes_are_caught():
    x = np.array([[[2.0, -2.0]]])
    kw = dict(history=np.array([[0, 1]]), repetition=np.array([2.0]))
    y = O.process_logits(x, **kw)[0][0, 0]
    assert not np.array_equal(y, x[0, 0] / 2.0)      # dividing whatever the sign
    assert not np.array_equal(y, x[0, 0] * [0.5, 1])  # negative logits left alone
    codes, scales, _ = O.quantize_int4(np.array([[0.5] + [7.0] + [0.0] * 30], np.float32), 32, False)
    assert (codes[0, 0] & 15) - 8 != 1               # ties away from zero
