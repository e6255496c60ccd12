"""Pins of oracle/awq_attn.py: values worked out by hand, and properties that its definitions imply."""
import numpy as np
import pytest

from oracle import awq_attn as A


def test_rope_by_hand():
    x = np.array([[[1.0, 0.0, 0.0, 2.0, 9.0]]])
    got = A.rope(x, [[1]], [np.pi / 2, np.pi], None, False, 1.0)  # pairs (0, 2) a quarter turn, (1, 3) half a turn
    assert np.allclose(got, [[[0.0, 0.0, 1.0, -2.0, 9.0]]], atol=1e-7)
    got = A.rope(x, [[1]], [np.pi / 2, np.pi], None, True, 2.0)  # pairs (0, 1), (2, 3)
    assert np.allclose(got, [[[0.0, 2.0, 0.0, -4.0, 9.0]]], atol=1e-6)
    got = A.rope(x, [[7], [1]], [1.0, np.pi], [5, 1], False, 1.0)  # an axis that is not there turns by nothing
    assert np.allclose(got, [[[1.0, 0.0, 0.0, -2.0, 9.0]]], atol=1e-6)


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_turns_back(pairs):
    rng = np.random.default_rng(0)
    x, d = rng.standard_normal((2, 5, 3, 10))
    pos, f, axis = rng.integers(0, 99, (2, 5)), rng.random(4), [0, 1, 1, 0]
    y = A.rope(x, pos, f, axis, pairs, 1.5)
    assert np.allclose(A.rope(y, pos, f, axis, pairs, 1 / 1.5, backward=True), x)
    assert np.isclose(np.sum(y[..., :8] * d[..., :8]), np.sum(x * A.rope(d, pos, f, axis, pairs, 1.5, backward=True)[..., :], where=np.arange(10) < 8))


def test_quantizer_by_hand():
    x = np.zeros(32)
    x[:4] = -2.0, 5.5, 0.25, 0.26  # step 0.5: 0.25 lies on the border of codes 4 and 5 (4.5 -> 4), 0.26 past it
    codes, step, offset = A.quantize(x[None])
    assert step.tolist() == [[0.5]] and offset.tolist() == [[-2.0]]
    assert codes[0, :5].tolist() == [0, 15, 4, 5, 4]
    assert A.dequantize(codes, step, offset)[0, :4].tolist() == [-2.0, 5.5, 0.0, 0.5]
    assert A.unpack(A.pack(codes)).tolist() == codes.tolist() and A.pack(codes)[0, 1] == 4 | 5 << 4


def test_quantizer_of_extremes():
    x = np.zeros((5, 32))
    x[1], x[2], x[3, 3], x[4, 0] = 1.25, 1e9, np.nan, -1e9
    codes, step, offset = A.quantize(x)
    assert step[:3].tolist() == [[0.0]] * 3 and offset[:3].tolist() == [[0.0], [1.25], [65024.0]] and not codes[:4].any()
    assert np.isnan(step[3]) and np.isnan(offset[3]) and np.isnan(A.dequantize(codes, step, offset)[3]).all()
    assert codes[4, 0] == 0 and codes[4, 1] == 15 and offset[4] == -65024.0


def test_quantizer_is_within_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 160)) * 3
    codes, step, offset = A.quantize(x)
    y = A.dequantize(codes, step, offset)
    s = np.repeat(step.astype(float), 128, -1)[:, :160]
    # half a step, and at the ends what the step's and the offset's own roundings leave out
    assert (np.abs(y - x) <= s * (0.5 + 15 * 2.0 ** -10) + 20 * 2.0 ** -11).all()
    assert step.shape == (50, 2)


def _cache(keys, values):
    """A one-page, one-head cache of 16 tokens whose numbers are the codes' (step 1, offset 0)."""
    codes = np.zeros((1, 2, 1, 16, 32), np.uint8)
    codes[0, 0, 0, :len(keys)], codes[0, 1, 0, :len(values)] = keys, values
    params = np.zeros((1, 2, 1, 1, 16, 2), np.float16)
    params[..., 0] = 1
    return A.pack(codes), params


def test_attention_by_hand():
    keys, values = np.zeros((3, 32), int), np.zeros((3, 32), int)
    keys[1, 0], keys[2, 0] = 1, 2
    values[:, 0] = 3, 6, 12
    codes, params = _cache(keys, values)
    q = np.zeros((3, 1, 32))
    q[:, 0, 0] = np.log(2.0)  # scores 0, log 2, 2 log 2: weights 1, 2, 4
    out, lse = A.attention(q, codes, params, np.array([[0]]), [3], [0, 3], 1.0, True, 0)
    assert np.allclose(out[:, 0, 0], [3.0, (3 + 12) / 3, (3 + 12 + 48) / 7]) and np.allclose(lse[:, 0], np.log([1, 3, 7]))
    out, _ = A.attention(q, codes, params, np.array([[0]]), [3], [0, 3], 1.0, True, 2)
    assert np.allclose(out[:, 0, 0], [3.0, 5.0, (12 + 48) / 6])
    out, _ = A.attention(q, codes, params, np.array([[0]]), [3], [0, 3], 1.0, False, 0)
    assert np.allclose(out[:, 0, 0], 9.0)
    out, _ = A.attention(q, codes, params, np.array([[0]]), [3], [0, 3], 1.0, False, 2)
    assert np.allclose(out[:, 0, 0], [9.0, 9.0, 10.0])


def test_attention_of_rows_that_see_nothing_and_of_missing_pages():
    codes, params = _cache(np.ones((2, 32), int), np.full((2, 32), 5))
    q = np.ones((4, 2, 32))
    out, lse = A.attention(q, codes, params, np.array([[0]]), [2], [0, 4], 1.0, True, 0)
    assert not out[:2].any() and np.isneginf(lse[:2]).all() and np.allclose(out[2:], 5.0)
    for page in (-1, 1):
        out, lse = A.attention(q, codes, params, np.array([[page]]), [2], [0, 4], 1.0, True, 0)
        assert not out.any() and np.isneginf(lse).all()
    kept = np.full((4, 2, 32), 9.0)
    out, _ = A.attention(q, codes, params, np.array([[0]]), [2], [1, 3], 1.0, True, 0, out=kept)
    assert (out[[0, 3]] == 9).all() and np.allclose(out[1:3], 5.0)


def test_an_unseen_nan_leaves_a_row_alone():
    codes, params = _cache(np.ones((3, 32), int), np.full((3, 32), 5))
    params[0, 1, 0, 0, 2] = np.nan
    q = np.ones((2, 1, 32))
    out, _ = A.attention(q, codes, params, np.array([[0]]), [3], [0, 2], 1.0, True, 0)
    assert np.allclose(out[0], 5.0) and np.isnan(out[1]).all()
