"""How far a value of the 4-bit cache is from what was written, as include/lq.h says it, by the oracle."""
import numpy as np
import pytest

import oracle.q4_oracle as Q


def errors(x, group):
    """|value - x|, the group's scale and its least element, in float64, by element."""
    codes, scales = Q.quantize(x, group)
    spread = lambda a: np.repeat(a.astype(np.float64), group, -1)
    least = x.reshape(*x.shape[:-1], -1, group).min(-1)
    v = Q.values(codes, scales).astype(np.float64)
    return np.abs(v - x.astype(np.float64)), spread(scales[..., 0]), np.abs(spread(least)), np.abs(v)


def bound(s, least, v):
    """Half a step, or where that is more the rounding of the base to fp16 (half a unit, 2^-11 of |least - 16 s|) and of
    fifteen scales; the value's own rounding; fp16's least numbers (half of 2^-24 for each of these seventeen).  The code
    is chosen in fp32: three roundings of at most 31 steps, 2^-17 of one."""
    return np.maximum(s / 2, 2.0 ** -11 * (least + 31 * s)) + 2.0 ** -17 * s + 2.0 ** -11 * v + 17 * 2.0 ** -25


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("mean,size", [(0, 1), (20, 1), (100, 1), (100, 0.1), (100, 0.01), (-3000, 1), (16000, 3), (5, 1e-4),
                                       (-0.5, 1e-3), (0, 1e-6)])
def test_groups_near_zero_and_far_from_it(group, mean, size):
    rng = np.random.default_rng(group)
    x = (mean + size * rng.standard_normal((300, 128))).astype(np.float32)
    e, s, least, v = errors(x, group)
    assert (e <= bound(s, least, v)).all()


def test_half_a_step_is_not_the_bound_far_from_zero():
    """Least values of a thousand scales and more: the base's rounding is more than half a step, and codes are cut."""
    x = (100 + 0.1 * np.random.default_rng(0).standard_normal((300, 128))).astype(np.float32)
    e, s, least, _ = errors(x, 64)
    assert (least > 1024 * s).all() and (e > s / 2 + 2.0 ** -5).any()      # (the value's own rounding near 100)
    near = np.random.default_rng(1).standard_normal((300, 128)).astype(np.float32)
    e, s, least, v = errors(near, 64)
    assert (e <= s / 2 * (1 + 2.0 ** -16) + 2.0 ** -11 * v).all()


def test_groups_that_become_one_value():
    """The scale is 0 up to a range of 15 2^-25 (half of fp16's least number, to the even one), and no further."""
    for least in (0.0, -2.0 ** -20):       # (bases that fp16 has)
        for width, one in ((2.0 ** -24, True), (15 * 2.0 ** -25, True), (16 * 2.0 ** -25, False)):
            x = np.full((1, 64), least, np.float32)
            x[0, 7] = least + width
            codes, scales = Q.quantize(x, 64)
            assert (scales[0, 0, 0] == 0) == one and codes.any() != one
