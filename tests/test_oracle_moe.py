"""Pins of the mixture-of-experts oracle (oracle/awq_moe.py): gradients against central differences, the
sort against its definition, gather and combine against dense one-hot products."""
import numpy as np
import pytest

from oracle import awq_moe as M


def _difference(f, a, delta, h=1e-5):
    """d/dt f(a + t delta) at t = 0."""
    return (f(a + h * delta) - f(a - h * delta)) / (2 * h)


@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_norm_gradients_are_the_differences(pre, post, gate):
    rng = np.random.default_rng(5)
    n, d, eps, a = 3, 7, 1e-3, 0.7
    v = {"y": rng.normal(size=(n, d)), "residual": rng.normal(size=(n, d)), "w_pre": rng.normal(size=d) if pre else None,
         "w_post": rng.normal(size=d) if post else None,
         "gate": None if gate is None else rng.normal(size=d if gate == "channel" else (n, d))}
    d_res, d_h = rng.normal(size=(n, d)), rng.normal(size=(n, d)) if pre else None

    def loss(**kw):
        r, h = M.block_norm(*[{**v, **kw}[k] for k in ("y", "residual", "w_pre", "w_post", "gate")], a, eps)
        return np.sum(r * d_res) + (np.sum(h * d_h) if pre else 0.0)

    got = M.block_norm_backward(v["y"], v["residual"], v["w_pre"], v["w_post"], v["gate"], a, eps, d_res, d_h)
    names = {"d_" + k: k for k, x in v.items() if x is not None}
    assert sorted(got) == sorted(names)
    for g, k in names.items():
        delta = rng.normal(size=v[k].shape)
        want = _difference(lambda x: loss(**{k: x}), v[k], delta)
        assert abs(np.sum(got[g] * delta) - want) < 1e-7 * (1 + abs(want)), g


def test_sort_is_the_stable_order():
    rng = np.random.default_rng(6)
    ids = rng.integers(-1, 6, (40, 3))  # -1 and 5 are out of range for 5 experts
    off, order, pos = M.sort_slots(ids, 5)
    flat = ids.reshape(-1)
    kept = np.flatnonzero((flat >= 0) & (flat < 5))
    want = kept[np.argsort(flat[kept], kind="stable")]
    assert np.array_equal(order[:kept.size], want) and np.all(order[kept.size:] == -1)
    assert np.array_equal(np.diff(off), np.bincount(flat[kept], minlength=5))
    assert np.array_equal(pos.reshape(-1)[want], np.arange(kept.size))
    assert np.all(pos.reshape(-1)[(flat < 0) | (flat >= 5)] == -1)


def test_routes_are_products_with_the_permutation():
    rng = np.random.default_rng(7)
    n, k, e, d = 9, 2, 4, 5
    ids = rng.integers(-1, e, (n, k))
    _, _, pos = M.sort_slots(ids, e)
    scales, w = rng.uniform(0.5, 2, (e, d)), rng.normal(size=(n, k))
    x, rows, g, gr = (rng.normal(size=s) for s in ((n, d), (n * k, d), (n, d), (n * k, d)))
    P = np.zeros((n, k, n * k))
    for t, j in np.argwhere(pos >= 0):
        P[t, j, pos[t, j]] = 1.0
    S = np.where((ids >= 0)[..., None], scales[np.maximum(ids, 0)], 0.0)
    named = P.sum((0, 1)) > 0
    got = M.gather(x, pos, ids, scales, np.full((n * k, d), 7.0))
    assert np.allclose(got[named], np.einsum("tjr,td,tjd->rd", P, x, S)[named]) and np.all(got[~named] == 7.0)
    assert np.allclose(M.gather_backward(gr, pos, ids, scales), np.einsum("tjr,rd,tjd->td", P, gr, S))
    assert np.allclose(M.combine(rows, pos, w), np.einsum("tjr,rd,tj->td", P, rows, w))
    d_rows, d_w = M.combine_backward(g, rows, pos, w, np.full((n * k, d), 3.0))
    assert np.allclose(d_w, np.einsum("tjr,rd,td->tj", P, rows, g))
    assert np.allclose(d_rows[named], np.einsum("tjr,tj,td->rd", P, w, g)[named]) and np.all(d_rows[~named] == 3.0)


def test_grouped_products_and_their_gradient():
    rng = np.random.default_rng(8)
    W = [rng.normal(size=(6, 4)) for _ in range(3)]
    off = np.array([0, 2, 2, 5])
    x = rng.normal(size=(7, 4))
    y = M.grouped(x, W, off, np.full((7, 6), 9.0))
    assert np.allclose(y[:2], x[:2] @ W[0].T) and np.allclose(y[2:5], x[2:5] @ W[2].T) and np.all(y[5:] == 9.0)
    h = M.grouped(x, W, off, np.zeros((7, 3)), act="silu")
    g, u = y[:5, :3], y[:5, 3:]
    assert np.allclose(h[:5], g / (1 + np.exp(-g)) * u)
    dy, delta = rng.normal(size=(7, 6)), rng.normal(size=(7, 4))
    dx = M.grouped(dy, W, off, np.zeros((7, 4)), backward=True)
    want = _difference(lambda a: np.sum(M.grouped(a, W, off, np.zeros((7, 6))) * dy), x, delta)
    assert abs(np.sum(dx[:5] * delta[:5]) - want) < 1e-8 * (1 + abs(want))
