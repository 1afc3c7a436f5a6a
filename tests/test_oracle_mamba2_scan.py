"""What pins the sequence scan's oracle: the decode oracle token by token, the unrolled sum, and differences for its gradients."""
import numpy as np
import pytest

import oracle as O


def _case(lens, H, G, d, n, seed=3):
    r = np.random.default_rng(seed)
    T = sum(lens)
    c = dict(x=r.normal(size=(T, H, d)), Bm=r.normal(size=(T, G, n)), Cm=r.normal(size=(T, G, n)), dt=r.normal(size=(T, H)),
             A_log=r.normal(size=H) * 0.5, dt_bias=r.normal(size=H), Dskip=r.normal(size=H))
    return c, np.concatenate([[0], np.cumsum(lens)]).astype(int), r


def test_scan_equals_decode_steps():
    lens = [3, 0, 5]
    c, cu, r = _case(lens, 4, 2, 16, 16)
    f32 = {k: v.astype(np.float32) for k, v in c.items()}
    c = {k: v.astype(np.float64) for k, v in f32.items()}
    pool = r.normal(size=(4, 4, 16, 16)).astype(np.float32)
    slots = np.array([2, 0, 3], np.int32)
    y, final = O.mamba2_scan(**c, cu=cu, init=pool.astype(np.float64), slot_map=slots)
    for s, n in enumerate(lens):
        p = pool.copy()
        for t in range(cu[s], cu[s + 1]):
            p, yt = O.mamba2_decode_step(p, slots[s:s + 1], f32["x"][t:t + 1], f32["Bm"][t:t + 1], f32["Cm"][t:t + 1], f32["dt"][t:t + 1],
                                         f32["A_log"], f32["dt_bias"], f32["Dskip"])
            np.testing.assert_allclose(y[t], yt[0], atol=1e-5)  # the decode's states are rounded to float32 at every step
        np.testing.assert_allclose(final[s], p[slots[s]], atol=1e-5)


def test_unrolled_sum_and_padded_sequence():
    c, cu, r = _case([6, 4], 2, 1, 3, 5)
    init = r.normal(size=(1, 2, 3, 5))
    y, final = O.mamba2_scan(**c, cu=cu, init=init, slot_map=[0, 7])
    assert not y[6:].any() and not final[1].any()
    g, dtp = O.m2_gates(c["dt"], c["A_log"], c["dt_bias"])
    for h in range(2):
        want = np.exp(g[:6, h].sum()) * init[0, h]
        for j in range(6):
            want = want + np.exp(g[j + 1:6, h].sum()) * dtp[j, h] * np.outer(c["x"][j, h], c["Bm"][j, 0])
        np.testing.assert_allclose(final[0, h], want, rtol=1e-12)


@pytest.mark.parametrize("state", [False, True])
def test_gradients_against_differences(state):
    """Central differences with step 1e-5: truncation about 1e-9, rounding about 1e-10."""
    c, cu, r = _case([4, 0, 3], 4, 2, 2, 3)
    init = r.normal(size=(3, 4, 2, 3)) if state else None
    slots = [1, 2, 0] if state else None
    dy, dfinal = r.normal(size=c["x"].shape), r.normal(size=(3, 4, 2, 3)) if state else None
    got = O.mamba2_scan_backward(dy, **c, cu=cu, init=init, slot_map=slots, dfinal=dfinal)

    def loss(a, i):
        y, final = O.mamba2_scan(**a, cu=cu, init=i, slot_map=slots)
        return float((y * dy).sum() + (0.0 if dfinal is None else (final * dfinal).sum()))
    for name, grad in zip(("x", "Bm", "Cm", "dt", "A_log", "dt_bias", "Dskip", "init"), got):
        if name == "init" and not state:
            continue
        base = init if name == "init" else c[name]
        num = np.zeros_like(base)
        for i in np.ndindex(num.shape):
            ends = []
            for step in (1e-5, -1e-5):
                v = base.copy()
                v[i] += step
                ends.append(loss(c, v) if name == "init" else loss(dict(c, **{name: v}), init))
            num[i] = (ends[0] - ends[1]) / 2e-5
        if name == "init":
            num = num[slots]
        np.testing.assert_allclose(grad, num, atol=1e-6, err_msg=name)


def test_sizes_bound_the_sums():
    c, cu, r = _case([9], 4, 2, 4, 4)
    dy = r.normal(size=c["x"].shape)
    for p, q in zip(O.mamba2_scan(**c, cu=cu), O.mamba2_scan(**c, cu=cu, sizes=True)):
        assert (np.abs(p) <= q * (1 + 1e-12)).all()
    for p, q in zip(O.mamba2_scan_backward(dy, **c, cu=cu), O.mamba2_scan_backward(dy, **c, cu=cu, sizes=True)):
        assert (np.abs(p) <= q * (1 + 1e-12)).all()
