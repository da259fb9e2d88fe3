"""Pins of oracle/block_oracle.py: closed forms, torch's float64 functions, central differences
and float64 autograd of formulas written apart from it.  No GPU needed."""
import numpy as np
import pytest
import torch

import oracle.block_oracle as O

EPS = 1e-5


def _rng(seed):
    return np.random.default_rng(seed)


def _slope(f, x, i, h=1e-5):
    """The central difference of f at element i of x (f reads x in place)."""
    flat = x.reshape(-1)
    keep = flat[i]
    flat[i] = keep + h
    up = f()
    flat[i] = keep - h
    down = f()
    flat[i] = keep
    return (up - down) / (2 * h)


def test_norm_closed_forms():
    w = np.array([1.0, 2.0, -0.5, 3.0])
    np.testing.assert_allclose(O.norm(np.full((1, 4), 7.0), w, 1e-300), [w], rtol=1e-15)   # a constant row: w
    np.testing.assert_array_equal(O.norm(np.zeros((2, 4)), w, EPS), 0.0)
    x = _rng(0).normal(size=(3, 4))
    got = O.norm(x, np.ones(4), 1e-300)
    np.testing.assert_allclose((got ** 2).mean(1), 1.0, rtol=1e-14)
    np.testing.assert_allclose(O.norm(8 * x, w, 64 * EPS), O.norm(x, w, EPS), rtol=1e-14)   # scale invariance
    np.testing.assert_allclose(O.norm(x, w, EPS), torch.nn.functional.rms_norm(
        torch.from_numpy(x), (4,), torch.from_numpy(w), EPS).numpy(), rtol=1e-13)


def test_norm_backward_against_differences():
    r = _rng(1)
    x, w, d = r.normal(size=(3, 7)), r.normal(size=7), r.normal(size=(3, 7))
    f = lambda: float((O.norm(x, w, EPS) * d).sum())
    dx, dw, _, _ = O.norm_backward(d, x, w, EPS)
    np.testing.assert_allclose(dx.reshape(-1), [_slope(f, x, i) for i in range(21)], rtol=1e-7, atol=1e-8)
    np.testing.assert_allclose(dw, [_slope(f, w, i) for i in range(7)], rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("post,nxt", [(True, True), (True, False), (False, True), (False, False)])
def test_combine_norm_backward_against_differences(post, nxt):
    """The whole chain -- combine, output norm, scaled residual, next norm -- as one function of
    every input, by central differences."""
    r = _rng(2)
    T, k, N, scale = 2, 3, 5, 0.7
    proj, gates, x = r.normal(size=(T, k, N)), r.uniform(0.1, 1, size=(T, k)), r.normal(size=(T, N))
    w_post = r.normal(size=N) if post else None
    w_next = r.normal(size=N) if nxt else None
    dx_out, dxn = r.normal(size=(T, N)), r.normal(size=(T, N)) if nxt else None

    def f():
        out = O.combine_norm(proj, gates, w_post, x, scale, EPS)
        total = float((out * dx_out).sum())
        return total + (float((O.norm(out, w_next, EPS) * dxn).sum()) if nxt else 0.0)

    x_out = O.combine_norm(proj, gates, w_post, x, scale, EPS)
    g = O.combine_norm_backward(dx_out, dxn, x_out, w_next, proj, gates, w_post, scale, EPS)
    for name, arr in (("dproj", proj), ("dgates", gates), ("dx", x), ("dw_post", w_post), ("dw_next", w_next)):
        if arr is not None:
            want = [_slope(f, arr, i) for i in range(arr.size)]
            np.testing.assert_allclose(g[name].reshape(-1), want, rtol=1e-6, atol=1e-8, err_msg=name)
        else:
            assert g[name] is None


def test_combine_skips_unrouted_slots():
    proj = np.ones((1, 2, 3))
    proj[0, 1] = np.nan
    h, _ = O.combine(proj, np.array([[0.5, 0.0]]))
    np.testing.assert_array_equal(h, 0.5)
    g = O.combine_norm_backward(np.ones((1, 3)), None, None, None, proj, np.array([[0.5, 0.0]]), None, 1.0, EPS)
    np.testing.assert_array_equal(g["dproj"], [[[0.5] * 3, [0.0] * 3]])
    np.testing.assert_array_equal(g["dgates"], [[3.0, 0.0]])


def test_balance_closed_forms():
    # even logits: every p is 1 / E, so the balance loss is 1 whatever the counts; z = log E
    T, E, k = 6, 4, 2
    ids = np.array([[0, 1]] * T)
    counts, tokens, losses = O.balance(np.zeros((T, E)), ids, [0, T])
    np.testing.assert_array_equal(counts, [[6, 6, 0, 0]])
    np.testing.assert_array_equal(tokens, [6, 6, 1])
    np.testing.assert_allclose(losses, [1.0, np.log(4) ** 2], rtol=1e-14)
    # all mass and all slots on one expert: the loss is E
    l = np.full((T, E), -np.inf)
    l[:, 2] = 3.0
    _, _, losses = O.balance(l, np.full((T, 1), 2), [0, T])
    np.testing.assert_allclose(losses, [E, 9.0], rtol=1e-14)


def test_balance_leaves_out():
    l = np.zeros((8, 3))
    l[1] = np.nan            # unrouted
    l[3] = -np.inf           # no logit
    ids = np.array([[0], [-1], [2], [0], [7], [1], [1], [1]])
    counts, tokens, _ = O.balance(l, ids, [1, 3, 3, 6])    # token 0 before, 6 and 7 behind
    np.testing.assert_array_equal(counts, [[0, 0, 1], [0, 0, 0], [0, 1, 0]])
    np.testing.assert_array_equal(tokens, [1, 0, 1, 2, 2])
    d, _ = O.route_backward(l, ids, np.ones((8, 1)), None, [1, 3, 3, 6], [1.0, 1.0])
    assert not d[[0, 1, 3, 4, 6, 7]].any() and d[2].any() and d[5].any()


def test_route_backward_against_differences():
    r = _rng(3)
    T, E, k, seq, dl = 7, 5, 2, [0, 3, 7], [0.8, 0.3]
    l = r.normal(size=(T, E))
    ids = np.argsort(-l, axis=1)[:, :k]
    ids[4, 1] = -1
    dg = r.normal(size=(T, k))

    def gates():
        g = np.zeros((T, k))
        for t in range(T):
            ok = ids[t] >= 0
            g[t, ok] = O.softmax(l[t, ids[t, ok]])[0]
        return g

    def f():
        losses = O.balance(l, ids, seq)[2]
        return float((gates() * dg).sum()) + dl[0] * losses[0] + dl[1] * losses[1]

    got, _ = O.route_backward(l, ids, gates(), dg, seq, dl)
    np.testing.assert_allclose(got.reshape(-1), [_slope(f, l, i) for i in range(T * E)], rtol=1e-6, atol=1e-8)


def test_route_backward_repeated_expert():
    """An expert given twice: both slots' shares meet in its logit."""
    l = np.array([[0.3, -0.2, 1.0]])
    ids = np.array([[1, 1, 2]])
    dg = np.array([[1.0, -2.0, 0.5]])
    q = lambda: O.softmax(l[0, ids[0]])[0]
    f = lambda: float(q() @ dg[0])
    got, _ = O.route_backward(l, ids, q()[None], dg, None, None)
    np.testing.assert_allclose(got[0], [_slope(f, l, i) for i in range(3)], rtol=1e-6, atol=1e-9)


def test_planted_mistakes_are_seen():
    """The differences reject a wrong sign, a dropped mean and a dropped factor."""
    r = _rng(4)
    x, w, d = r.normal(size=(2, 6)), r.normal(size=6), r.normal(size=(2, 6))
    f = lambda: float((O.norm(x, w, EPS) * d).sum())
    want = np.array([_slope(f, x, i) for i in range(12)]).reshape(2, 6)
    rr = 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + EPS)
    unit = x * rr
    for wrong in (rr * d * w, rr * (d * w + unit * (d * w * unit).mean(1, keepdims=True)),
                  rr * (d * w - unit * (d * w * unit).sum(1, keepdims=True)),
                  rr * (d - unit * (d * unit).mean(1, keepdims=True))):
        assert np.abs(wrong - want).max() > 1e-3
