"""The routed-expert layer's oracle against hand-worked cases, invariants and
central differences (CPU only)."""

import numpy as np
import pytest

from oracle import moe


def rng(seed=0):
    return np.random.default_rng(seed)


def test_route_hand_worked():
    x = np.array([[0.0, 2.0, 2.0, -1.0, 3.0, -np.inf]])
    w, e = moe.route(x, 3, "softmax", renormalize=True)
    assert e.tolist() == [[4, 1, 2]]                      # the tie goes to the lower expert
    want = np.exp([3.0, 2.0, 2.0])
    np.testing.assert_allclose(w[0], want / want.sum(), rtol=1e-15)
    w, e = moe.route(x, 6, "sigmoid", renormalize=False, scale=2.0)
    assert e.tolist() == [[4, 1, 2, 0, 3, -1]] and w[0, 5] == 0
    np.testing.assert_allclose(w[0, 3], 1.0, rtol=1e-15)  # 2 sigmoid(0)


def test_route_bias_moves_the_choice_only():
    x = np.array([[1.0, 0.0, -1.0, -2.0]])
    w, e = moe.route(x, 1, "sigmoid", bias=[0, 0, 0, 5.0], renormalize=False)
    assert e.tolist() == [[3]]
    np.testing.assert_allclose(w, moe.sigmoid([[-2.0]]), rtol=1e-15)


def test_route_groups():
    # groups of three: values 0.9 + 0.1, 0.6 + 0.5, 0.95 (its others are out)
    s = np.array([[0.9, 0.1, 0.05, 0.6, 0.5, 0.2, 0.95, 0.0, 0.0]])
    x = np.log(np.where(s > 0, s, 0.5) / (1 - np.where(s > 0, s, 0.5)))
    x[0, 7:] = -np.inf
    assert moe.route(x, 2, "sigmoid", groups=3, top_groups=1)[1].tolist() == [[3, 4]]
    assert moe.route(x, 2, "sigmoid", groups=3, top_groups=1, group_best=1)[1].tolist() == [[6, -1]]
    assert moe.route(x, 3, "sigmoid", groups=3, top_groups=2)[1].tolist() == [[0, 3, 4]]


def test_route_masks():
    x = np.array([[np.nan, np.nan], [-np.inf, -np.inf], [np.nan, 0.0]])
    w, e = moe.route(x, 2, "softmax", token_mask=[False, True, True])
    assert e.tolist() == [[-1, -1], [-1, -1], [1, -1]] and w.tolist() == [[0, 0], [0, 0], [1, 0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_grad_against_differences(score, renormalize):
    g = rng(3)
    x = g.standard_normal((4, 9))
    x[1, 2] = -np.inf
    gw = g.standard_normal((4, 3))
    kw = dict(score=score, renormalize=renormalize, scale=1.7)
    w, e = moe.route(x, 3, **kw)
    grad = moe.route_grad(x, e, gw, **kw)
    h = 1e-6
    for t, i in np.ndindex(x.shape):
        if x[t, i] == -np.inf:
            assert grad[t, i] == 0
            continue
        hi, lo = x.copy(), x.copy()
        hi[t, i] += h
        lo[t, i] -= h
        wh, eh = moe.route(hi, 3, **kw)
        wl, el = moe.route(lo, 3, **kw)
        assert np.array_equal(eh, e) and np.array_equal(el, e)
        diff = ((wh - wl) * gw).sum() / (2 * h)
        assert abs(diff - grad[t, i]) < 1e-8             # h^2 / 6 of the third derivative, and 1e-16 / h


def test_plan_orders_slots_stably():
    e = np.array([[2, 0], [-1, 2], [0, 1], [5, 2]], np.int32)
    offs, rows, slots = moe.plan(e, 0, 3)
    assert offs.tolist() == [2, 3, 6]
    assert slots.tolist() == [1, 4, 5, 0, 3, 7, 2, 6]
    assert rows.tolist() == [[3, 0], [~6, 4], [1, 2], [~7, 5]]
    offs, rows, slots = moe.plan(e, 2, 2)                 # experts 2 and 3 only
    assert offs.tolist() == [3, 3] and slots.tolist() == [0, 3, 7, 1, 2, 4, 5, 6]
    assert (rows.reshape(-1)[slots] == [0, 1, 2, ~3, ~4, ~5, ~6, ~7]).all()


def test_dispatch_and_combine_are_adjoint():
    g = rng(5)
    e = g.integers(-1, 6, (7, 3)).astype(np.int32)
    _, rows, _ = moe.plan(e, 1, 4)
    x, y = g.standard_normal((7, 5)), g.standard_normal((21, 5))
    w, go = g.standard_normal((7, 3)), g.standard_normal((7, 5))
    assert np.isclose((moe.dispatch(x, rows) * y).sum(), (x * moe.dispatch_grad(y, rows)).sum(), rtol=1e-12)
    gy, gw = moe.combine_grad(go, y, w, rows)
    total = (moe.combine(y, w, rows) * go).sum()          # linear in y and in w
    assert np.isclose(total, (gy * y).sum(), rtol=1e-12) and np.isclose(total, (gw * w).sum(), rtol=1e-12)


def test_swiglu_grad_against_differences():
    g = rng(6)
    x, gh = g.standard_normal((3, 8)) * 2, g.standard_normal((3, 4))
    grad = moe.swiglu_grad(x, gh)
    h = 1e-6
    for i in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += h
        lo[i] -= h
        assert abs(((moe.swiglu(hi) - moe.swiglu(lo)) * gh).sum() / (2 * h) - grad[i]) < 1e-8


def test_kept_values_are_within_half_a_step():
    x = (rng(7).standard_normal((5, 128)) * 4).astype(np.float32)
    x[1] = 0
    k = moe.kept(x)
    blocks = np.abs(x.reshape(5, 4, 32)).max(-1)
    with np.errstate(divide="ignore"):
        unit = np.where(blocks > 0, np.exp2(np.ceil(np.log2(np.where(blocks > 0, blocks, 1) / 448))), 0)
    # half an E4M3 step: 2^-4 of a normal value, 2^-10 of the scale below 2^-6 of it
    bound = np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(unit, 32, -1) * 2.0 ** -10)
    assert (np.abs(k - x) <= bound).all() and (k[1] == 0).all()
