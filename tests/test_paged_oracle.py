"""Hand-worked and closed-form facts that pin the oracle of the paged cache's operators."""
import numpy as np
import pytest

import oracle.paged_oracle as P


def test_plan_by_hand():
    # blocks of 16: 20 cached tokens in blocks 7, 3; 13 new ones fill positions 20..32 and need one more block
    table = [[7, 3, -1, -1], [-1, -1, -1, -1]]
    t, cu, lens, slots, pos, used, ok = P.plan([20, 0], [13, 17], 16, [9, 4, 5, 1], table, 32)
    assert ok and used == 3 and cu.tolist() == [0, 13, 30] and lens.tolist() == [33, 17]
    assert t.tolist() == [[7, 3, 9, -1], [4, 5, -1, -1]]
    assert pos[:13].tolist() == list(range(20, 33)) and pos[13:].tolist() == list(range(17)) + [0, 0]
    assert slots[0] == 3 * 16 + 4 and slots[12] == 9 * 16 and slots[13] == 64 and slots[29] == 5 * 16
    assert slots[30:].tolist() == [-1, -1]


def test_plan_says_when_something_is_short():
    blank = [[-1, -1]]
    assert P.plan([0], [32], 16, [1, 2], blank, 32)[-1]
    assert not P.plan([0], [33], 16, [1, 2, 3], blank, 64)[-1]       # table
    assert not P.plan([0], [32], 16, [1], blank, 32)[-1]             # pool
    assert not P.plan([0], [32], 16, [1, 2], blank, 31)[-1]          # token maps
    assert not P.plan([-1], [3], 16, [1, 2], blank, 31)[-1]


def test_norm_rope_closed_forms():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 32))
    ang = rng.uniform(0, 6, (5, 8))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for inter in (False, True):
        y = P.norm_rope(x, None, 0.0, [4, 0, 2], table, 16, inter)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))   # a rotation
        assert np.array_equal(y[..., 16:], x[..., 16:])
        back = P.norm_rope(y, None, 0.0, [4, 0, 2], np.concatenate([np.cos(ang), -np.sin(ang)], 1), 16, inter)
        assert np.allclose(back, x)
        n = P.norm_rope(x, np.ones(32), 0.0, [4, 0, 2], table, 16, inter)
        assert np.allclose(np.mean(n * n, -1), 1)


def test_append_keeps_the_larger_scale_and_forgets_a_restarted_block():
    codes, scales = np.full((2, 1, 16, 4), 100.0), np.array([[0.5], [0.25]])
    x = np.zeros((3, 1, 4))
    x[0, 0] = [127, -63.5, 0, 1]
    x[1, 0] = [12.7, 0, 0, 0]
    x[2, 0] = [1.27, 0, 0, 0]
    c, s = P.append(x, [5, 16, -1], codes, scales)
    assert s[0, 0] == 1.0 and np.allclose(c[0, 0, :5], 50) and np.allclose(c[0, 0, 5], [127, -63.5, 0, 1])
    assert np.allclose(c[0, 0, 6:], 100)
    assert np.isclose(s[1, 0], 0.1) and np.allclose(c[1, 0, 0], [127, 0, 0, 0])


def test_attention_against_dense_softmax():
    rng = np.random.default_rng(1)
    nb, hk, bs, d, hq = 4, 2, 16, 8, 4
    kc, vc = (rng.integers(-127, 128, (nb, hk, bs, d)) for _ in range(2))
    ks, vs = (rng.uniform(0.01, 0.02, (nb, hk)) for _ in range(2))
    q = rng.standard_normal((3, hq, d))
    out = P.attention(q, [0, 3], [20], np.array([[2, 0, -1]]), kc, ks, vc, vs, 0.3)
    for h in range(hq):
        k = np.concatenate([kc[2, h // 2] * ks[2, h // 2], kc[0, h // 2] * ks[0, h // 2]])[:20]
        v = np.concatenate([vc[2, h // 2] * vs[2, h // 2], vc[0, h // 2] * vs[0, h // 2]])[:20]
        s = 0.3 * q[:, h] @ k.T
        s[np.triu(np.ones((3, 20), bool), 18)] = -np.inf
        w = np.exp(s - s.max(1, keepdims=True))
        assert np.allclose(out[:, h], (w / w.sum(1, keepdims=True)) @ v)
    assert not P.attention(q, [0, 3], [0], np.array([[2]]), kc, ks, vc, vs, 0.3).any()


@pytest.mark.parametrize("onehot", [False, True])
def test_verify_draws_the_target_distribution(onehot):
    """Accepting x with min(1, p/q) and drawing the rest from max(p - q, 0) leaves the first token distributed as p."""
    rng = np.random.default_rng(2)
    n, v = 20000, 5
    p = np.array([0.1, 0.4, 0.05, 0.25, 0.2], np.float32)
    q = np.array([0.3, 0.1, 0.3, 0.2, 0.1], np.float32)
    x = np.full((n, 1), 3) if onehot else rng.choice(v, (n, 1), p=q / q.sum(dtype=np.float64))
    target = np.broadcast_to(p, (n, 2, v))
    draft = None if onehot else np.broadcast_to(q, (n, 1, v))
    out, acc = P.verify(x, None, target, draft, rng.random((n, 1), np.float32), rng.random(n, np.float32))
    freq = np.bincount(out[:, 0], minlength=v) / n
    assert np.abs(freq - p).max() < 5 * np.sqrt(0.25 / n)            # five standard deviations
    want = 0.25 if onehot else np.minimum(p, q).sum()
    assert abs(acc.mean() - want) < 5 * np.sqrt(0.25 / n)
    assert ((out[:, 1] >= 0) == (acc == 1)).all()
