"""What pins the norm's oracle: a hand-worked row, and its gradients against differences."""
import numpy as np
import pytest

import oracle as O


def test_hand_worked_row():
    """(1, 3, 5, 7): mean 4, variance 5; with eps 4, rstd 1/3.  RMS form: mean square 21, with eps 4 rstd 1/5."""
    x = np.array([[1.0, 3.0, 5.0, 7.0]])
    w, b = np.array([3.0, 3.0, 6.0, 6.0]), np.array([0.0, 1.0, 0.0, 1.0])
    y, mean, rstd = O.layer_norm(x, w, b, eps=4.0)
    np.testing.assert_allclose(y, [[-3.0, 0.0, 2.0, 7.0]], rtol=1e-14)
    np.testing.assert_allclose([mean[0, 0], rstd[0, 0]], [4.0, 1 / 3], rtol=1e-14)
    y, mean, rstd = O.layer_norm(x, np.full(4, 5.0), rms=True, eps=4.0)
    np.testing.assert_allclose(y, x, rtol=1e-14)
    assert mean[0, 0] == 0.0 and abs(rstd[0, 0] - 0.2) < 1e-15
    y, mean, _ = O.layer_norm(x, np.ones(4), groups=2, eps=0.0)
    np.testing.assert_allclose(y, [[-1.0, 1.0, -1.0, 1.0]], rtol=1e-14)
    np.testing.assert_allclose(mean, [[2.0, 6.0]], rtol=1e-14)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("gate", ["none", "before", "after"])
def test_gradients_against_differences(rms, bias, gate):
    """Central differences with step 1e-5: truncation about 1e-10, rounding about 1e-11 over 1e-5 steps."""
    r = np.random.default_rng(7)
    rows, width, groups = 3, 12, 2
    args = dict(x=r.normal(size=(rows, width)), w=r.normal(size=width), b=r.normal(size=width) if bias else None,
                z=r.normal(size=(rows, width)) if gate != "none" else None)
    form = dict(groups=groups, rms=rms, gate_after=gate == "after", eps=1e-3)
    dy = r.normal(size=(rows, width))
    dx, dw, db, dz = O.layer_norm_backward(dy, **args, **form)
    loss = lambda a: float((O.layer_norm(**a, **form)[0] * dy).sum())  # noqa: E731
    for name, grad in (("x", dx), ("w", dw), ("b", db), ("z", dz)):
        if args[name] is None:
            continue
        num = np.zeros_like(args[name])
        for i in np.ndindex(num.shape):
            ends = []
            for step in (1e-5, -1e-5):
                a = dict(args)
                a[name] = args[name].copy()
                a[name][i] += step
                ends.append(loss(a))
            num[i] = (ends[0] - ends[1]) / 2e-5
        np.testing.assert_allclose(grad, num, atol=1e-7, err_msg=name)
