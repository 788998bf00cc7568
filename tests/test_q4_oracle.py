"""The oracle of the 4-bit cache and of token scoring, by hand-worked and closed-form facts."""
import math

import numpy as np
import pytest

import oracle.q4_oracle as Q


def test_a_group_by_hand():
    """0 .. 15 and back in steps of 1: s = 1, b = -16, codes the numbers themselves."""
    x = np.array([list(range(16)) + list(range(15, -1, -1))], np.float32)
    codes, scales = Q.quantize(x, 32)
    assert scales[0, 0].tolist() == [1.0, -16.0]
    assert codes[0].tolist() == [2 * j | (2 * j + 1) << 4 for j in range(8)] + [15 - 2 * j | (14 - 2 * j) << 4
                                                                               for j in range(8)]
    assert np.array_equal(Q.values(codes, scales)[0], x[0])


def test_ties_go_to_the_even_code_and_groups_are_apart():
    # least 0, largest 15: s = 1; 0.5, 1.5, 2.5 lie between two codes; the second group is constant
    x = np.zeros(64, np.float32)
    x[:5] = [15, 0.5, 1.5, 2.5, 2.5000002]
    x[32:] = 3.25
    codes, scales = Q.quantize(x, 32)
    c = [(codes[j // 2] >> 4 * (j % 2)) & 15 for j in range(64)]
    assert c[:5] == [15, 0, 2, 2, 2] and not any(c[32:])      # 2.5000002 + 16 rounds to 18.5 in fp32
    assert scales.tolist() == [[1.0, -16.0], [0.0, 3.25]]
    assert (Q.values(codes, scales)[32:] == np.float16(3.25)).all()


@pytest.mark.parametrize("size", [1e-3, 1.0, 300.0, 1e5])
@pytest.mark.parametrize("offset", [0.0, 5.0])
def test_values_are_within_half_a_step(size, offset):
    """|x - value| <= s / 2 plus the roundings of s (a code can be 15 half-ulps short), of b and of the value itself."""
    rng = np.random.default_rng(3)
    x = ((rng.standard_normal((50, 128)) + offset) * size).astype(np.float32)
    codes, scales = Q.quantize(x, 64)
    s = np.repeat(scales[..., 0].astype(np.float64), 64, -1)
    b = np.repeat(np.abs(scales[..., 1].astype(np.float64)), 64, -1)
    v = Q.values(codes, scales).astype(np.float64)
    y = np.clip(x.astype(np.float64), -16384, 16384)
    bound = s / 2 + 2.0 ** -11 * (15 * s + b + np.abs(y)) + 15 * 2.0 ** -24
    assert (np.abs(v - y) <= bound).all()


def test_not_finite_and_out_of_range():
    x = np.zeros((1, 64), np.float32)
    x[0, :4] = [np.nan, np.inf, -np.inf, 1e9]
    codes, scales = Q.quantize(x, 64)
    v = Q.values(codes, scales)[0]
    assert np.isfinite(v).all() and abs(v[3] - 16384) <= 16 and not v[:3].any()


def test_append_writes_only_its_slots():
    rng = np.random.default_rng(4)
    codes = rng.integers(0, 256, (3, 2, 16, 32), dtype=np.uint8)
    scales = rng.standard_normal((3, 2, 16, 2, 2)).astype(np.float16)
    x = rng.standard_normal((4, 2, 64)).astype(np.float32)
    c, s = Q.append(x, [5, -1, 47, 99], codes, scales)
    touched = np.zeros((3, 16), bool)
    touched[0, 5] = touched[2, 15] = True
    assert np.array_equal(c.transpose(0, 2, 1, 3)[~touched], codes.transpose(0, 2, 1, 3)[~touched])
    assert np.array_equal(s[2, :, 15], Q.quantize(x[2], 32)[1])


def test_attention_of_one_token_and_of_equal_scores():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((2, 20, 1, 64)).astype(np.float32)
    cache = []
    for n in range(2):
        c = np.zeros((2, 1, 16, 32), np.uint8)
        s = np.zeros((2, 1, 16, 2, 2), np.float16)
        cache += Q.append(x[n], range(20), c, s)
    table = np.array([[0, 1]])
    v = Q.values(cache[2], cache[3])[:, 0].reshape(32, 64).astype(np.float64)
    q = rng.standard_normal((1, 3, 64))
    one = Q.attention(q, [0, 1], [1], table, *cache, 0.1)
    assert np.allclose(one[0], v[0])
    equal = Q.attention(np.zeros((1, 3, 64)), [0, 1], [20], table, *cache, 0.1)
    assert np.allclose(equal[0], v[:20].mean(0))
    assert not Q.attention(q, [0, 1], [0], table, *cache, 0.1).any()


def test_scores_by_hand():
    x = np.array([[0.0, math.log(2), -math.inf, 0.0], [1.0, 1.0, 1.0, 1.0]])
    lp, h, rank, top, tlp = Q.token_logprobs(x, [3, -1], 3)
    assert np.allclose(lp, [math.log(0.25), 0]) and rank.tolist() == [2, -1]
    assert np.allclose(h, [1.5 * math.log(2), math.log(4)])
    assert top.tolist() == [[1, 0, 3], [0, 1, 2]]
    assert np.allclose(tlp[0], np.log([0.5, 0.25, 0.25]))
