"""What pins the oracles of linear attention and of the norm and rotation of queries and keys: hand-worked values, the sum over
pairs of tokens, single tokens in a row, and gradients against differences."""
import numpy as np
import pytest

import oracle as O


def _inputs(seed=3, T=7, H=4, Hq=2, Hk=4, Hv=1, d=3):
    r = np.random.default_rng(seed)
    return (r.normal(size=(T, Hq, d)), r.normal(size=(T, Hk, d)), r.normal(size=(T, Hv, d)), -r.uniform(0.05, 1.0, size=H),
            r.normal(size=(5, H, d, d)), r)


def test_hand_worked_tokens():
    """One head of size 1, decay 1/2: states 2 3 = 6, then 3 + 1 5 = 8, then 4 + 4 (-1) = 0; scale 1."""
    q, k, v = (np.array(x, float).reshape(3, 1, 1) for x in ([1, 10, 7], [2, 1, 4], [3, 5, -1]))
    o, end = O.linear_scan(q, k, v, np.log([0.5]), [0, 3])
    np.testing.assert_allclose(o[:, 0, 0], [6, 80, 0], atol=1e-14)
    o, end = O.linear_scan(q, k, v, np.log([0.5]), [0, 1, 3], np.full((2, 1, 1, 1), 4.0), [1, 0])
    np.testing.assert_allclose(o[:, 0, 0], [8, 70, 7 * (3.5 - 4)], atol=1e-14)
    np.testing.assert_allclose(end[:, 0, 0, 0], [8, -0.5], atol=1e-14)


def test_scan_is_the_sum_over_pairs():
    q, k, v, g, init, _ = _inputs()
    o, _ = O.linear_scan(q, k, v, g, [0, 7], init, [2], scale=0.7)
    for h in range(4):
        for t in range(7):
            want = np.exp(g[h] * (t + 1)) * q[t, h // 2] @ init[2, h]
            want = want + sum(np.exp(g[h] * (t - j)) * (q[t, h // 2] @ k[j, h]) * v[j, 0] for j in range(t + 1))
            np.testing.assert_allclose(o[t, h], 0.7 * want, rtol=1e-12, atol=1e-12)


def test_steps_are_the_scan_and_padding_is_left_out():
    q, k, v, g, init, _ = _inputs()
    o, ends = O.linear_scan(q, k, v, g, [0, 3, 3, 7], init, [1, 5, -1])
    assert not o[3:].any() and not ends[1:].any()
    S = init[1][None]
    for t in range(3):
        y, S = O.linear_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], g, S)
        np.testing.assert_allclose(y[0], o[t], rtol=1e-13, atol=1e-13)
    np.testing.assert_allclose(S[0], ends[0], rtol=1e-13, atol=1e-13)


def _differences(f, args, grads, step=1e-5):
    """Central differences: truncation about 1e-10, rounding about 1e-11 over 1e-5 steps."""
    r = np.random.default_rng(1)
    for i, (x, dx) in enumerate(zip(args, grads)):
        for _ in range(6):
            at = tuple(r.integers(n) for n in x.shape)
            up, down = ([a.copy() for a in args] for _ in range(2))
            up[i][at] += step
            down[i][at] -= step
            assert abs((f(*up) - f(*down)) / (2 * step) - dx[at]) < 1e-6 * (1 + abs(dx[at])), (i, at)


def test_scan_gradients_against_differences():
    q, k, v, g, init, r = _inputs()
    cu, slots = [0, 3, 3, 7], [4, 1, 0]
    do, df = r.normal(size=(7, 4, 3)), r.normal(size=(3, 4, 3, 3))

    def f(q, k, v, init):
        o, ends = O.linear_scan(q, k, v, g, cu, init, slots)
        ends[1] = init[slots[1]]
        return (o * do).sum() + (ends * df).sum()

    dq, dk, dv, dinit = O.linear_scan_backward(do, q, k, v, g, cu, init, slots, df)
    by_slot = np.zeros_like(init)
    by_slot[slots] = dinit
    _differences(f, (q, k, v, init), (dq, dk, dv, by_slot))


def test_rotation_by_hand():
    """(3, 4, 0, 0) has mean square 25/4; with eps 75/4 the norm is (3, 4, 0, 0) / 5.  A quarter turn of the pairs."""
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    f = np.array([np.pi / 2, 0.0])
    y = O.qk_norm_rope(x, np.full(4, 5.0), [1], f, eps=75 / 4)
    np.testing.assert_allclose(y[0, 0], [0, 4, 3, 0], atol=1e-14)
    y = O.qk_norm_rope(x, np.full(4, 5.0), [1], f, eps=75 / 4, neighbours=True)
    np.testing.assert_allclose(y[0, 0], [-4, 3, 0, 0], atol=1e-14)
    y = O.qk_norm_rope(x, np.full(4, 5.0), [[5], [1]], np.array([0.0, np.pi]), eps=75 / 4, axes=[0, 1])
    np.testing.assert_allclose(y[0, 0], [3, -4, 0, 0], atol=1e-14)
    y = O.qk_norm_rope(x, np.full(4, 5.0), [2], np.array([np.pi / 2]), eps=75 / 4)  # the first two values only
    np.testing.assert_allclose(y[0, 0], [-3, -4, 0, 0], atol=1e-14)


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("axes", [None, [0, 2, 1]])
def test_rotation_gradients_against_differences(neighbours, axes):
    r = np.random.default_rng(5)
    T, heads, d = 3, 2, 8
    x, w, dy, f = r.normal(size=(T, heads, d)), r.normal(size=d), r.normal(size=(T, heads, d)), r.uniform(0.1, 2, size=3)
    pos = r.integers(-5, 50, size=(3, T)) if axes else r.integers(-5, 50, size=T)
    form = dict(eps=0.01, neighbours=neighbours, axes=axes)
    dx, dw = O.qk_norm_rope_backward(dy, x, w, pos, f, **form)
    _differences(lambda x, w: (O.qk_norm_rope(x, w, pos, f, **form) * dy).sum(), (x, w), (dx, dw))
