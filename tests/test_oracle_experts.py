"""Pins of the expert operators' oracle: gradients against central differences,
and the identities that tie the operators together."""
import numpy as np

from nerf_inputs import kilonerf_weights
from oracle import experts as E
from oracle import march


def _route(rng, n, k, e):
    ids = np.stack([rng.permutation(e)[:k] for _ in range(n)])
    ids[rng.random((n, k)) < 0.2] = -1
    return ids


def test_sort_orders_by_expert_then_pair():
    rng = np.random.default_rng(0)
    for e in (3, 100):
        ids = rng.integers(-2, e + 2, size=(40, 3))
        offset, order, pos = E.sort(ids, e)
        flat = ids.ravel()
        assert offset[0] == 0 and offset[-1] == order.size == ((flat >= 0) & (flat < e)).sum()
        for c in range(e):
            seg = order[offset[c]:offset[c + 1]]
            assert (flat[seg] == c).all() and (np.diff(seg) > 0).all()
        assert (pos.ravel()[order] == np.arange(order.size)).all()


def test_row_gradients_against_differences():
    """L = <combine(rows(x, w), v), G> with both weights: every gradient by differences."""
    rng = np.random.default_rng(1)
    n, k, e, c = 5, 2, 4, 3
    _, _, pos = E.sort(_route(rng, n, k, e), e)
    x, w, v, G = rng.normal(size=(n, c)), rng.normal(size=(n, k)), rng.normal(size=(n, k)), rng.normal(size=(n, c))
    zero = np.zeros((n * k, c))

    def loss(x, w, v):
        return (E.combine(E.dispatch(x, pos, w, zero), pos, v) * G).sum()

    rows = E.dispatch(x, pos, w, zero)
    d_rows = E.dispatch(G, pos, v, zero)           # combine's backward
    grads = {"x": E.combine(d_rows, pos, w), "w": E.dots(d_rows, x, pos), "v": E.dots(rows, G, pos)}
    args = {"x": x, "w": w, "v": v}
    for name, g in grads.items():
        for at in np.ndindex(g.shape):
            hi, lo = {k2: a.copy() for k2, a in args.items()}, {k2: a.copy() for k2, a in args.items()}
            hi[name][at] += 1e-6
            lo[name][at] -= 1e-6
            assert abs((loss(**hi) - loss(**lo)) / 2e-6 - g[at]) < 1e-7


def test_distill_gradient_against_differences():
    rng = np.random.default_rng(2)
    s, t = rng.normal(size=(4, 7)), rng.normal(size=(4, 3))
    ids = np.array([[1, 4, 6], [0, -1, 2], [-1, -1, -1], [3, 3, 5]])     # short, empty and repeated rows
    scale = rng.random(4) + 0.5
    loss, grad = E.distill(s, t, ids, 1.7, scale)
    assert loss[2] == 0 and (grad[2] == 0).all() and (loss[[0, 1]] >= 0).all()
    for at in np.ndindex(s.shape):
        hi, lo = s.copy(), s.copy()
        hi[at] += 1e-6
        lo[at] -= 1e-6
        num = ((E.distill(hi, t, ids, 1.7)[0] - E.distill(lo, t, ids, 1.7)[0]) * scale).sum() / 2e-6
        assert abs(num - grad[at]) < 1e-7


def test_cells_forward_is_the_march_oracles_network():
    rng = np.random.default_rng(3)
    w = kilonerf_weights(5, n_cells=3)
    x, d = rng.uniform(-1.5, 1.5, size=(20, 3)).astype(np.float32), rng.normal(size=(20, 3)).astype(np.float32)
    cells = np.sort(rng.integers(0, 3, size=20))
    offset = np.searchsorted(cells, np.arange(4))
    raw, _ = E.cells_forward(x, d, offset, w)
    from oracle import nerf
    sigma, rgb = march.kilonerf_eval(w, cells, x, nerf.unit(d))
    assert np.abs(nerf.relu(raw[:, 3]) - sigma).max() < 1e-12
    assert np.abs(nerf.sigmoid(raw[:, :3]) - rgb).max() < 1e-12


def test_cells_gradient_against_differences():
    rng = np.random.default_rng(4)
    w = kilonerf_weights(6, n_cells=3).astype(np.float64)
    x, d = rng.uniform(-1.5, 1.5, size=(9, 3)), rng.normal(size=(9, 3))
    offset = np.array([0, 5, 5, 9])                      # the middle cell is empty
    g = rng.normal(size=(9, 4))
    _, hidden = E.cells_forward(x, d, offset, w)
    grad = E.cells_backward(x, d, offset, w, hidden, g)
    assert (grad[1] == 0).all()

    def loss(w):
        return (E.cells_forward(x, d, offset, w)[0] * g).sum()

    for q in list(rng.integers(0, E.N_CELL, size=150)) + [2016, 2048, 2048 + 32 * 32, 3104, 3136, 3137, 3314, 3316]:
        for c in (0, 2):
            hi, lo = w.copy(), w.copy()
            hi[c, q] += 1e-6
            lo[c, q] -= 1e-6
            assert abs((loss(hi) - loss(lo)) / 2e-6 - grad[c, q]) < 1e-5 * max(1.0, abs(grad[c, q]))
