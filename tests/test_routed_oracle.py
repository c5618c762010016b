"""The routed layers' oracle against things other than itself (CPU)."""
import numpy as np
import pytest

from oracle import routed


def _ids(T, k, E, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, size=(T, k))
    ids[rng.random((T, k)) < drop] = -1
    return ids


@pytest.mark.parametrize("T,k,E,drop", [(1, 1, 1, 0.0), (7, 3, 4, 0.0), (40, 2, 9, 0.3), (5, 4, 64, 1.0)])
def test_sort_is_numpys_stable_argsort(T, k, E, drop):
    ids = _ids(T, k, E, seed=T + k, drop=drop)
    offsets, rows, slots = routed.sort(ids, E)
    flat = ids.reshape(-1)
    live = np.flatnonzero(flat >= 0)
    assert np.array_equal(rows, live[np.argsort(flat[live], kind="stable")])
    assert np.array_equal(np.diff(offsets), np.bincount(flat[live], minlength=E))
    for i, s in enumerate(slots.reshape(-1)):
        assert (s == -1) if flat[i] < 0 else rows[s] == i


def test_combine_of_one_expert_per_token_is_a_scaled_copy():
    ids = _ids(6, 1, 3, seed=1)
    _, rows, slots = routed.sort(ids, 3)
    X = np.random.default_rng(2).standard_normal((6, 8))
    Y, _ = routed.combine(X[rows], slots, np.full((6, 1), 0.5))
    assert np.array_equal(Y, 0.5 * X)


def test_combine_grad_matches_differences():
    """d/dp of L = sum(dY * combine(...)), by central differences (L is linear in each argument,
    so they are exact up to rounding)."""
    rng = np.random.default_rng(3)
    T, k, E, H = 4, 3, 5, 8
    ids = _ids(T, k, E, seed=4, drop=0.25)
    _, rows, slots = routed.sort(ids, E)
    Ys, w, dY = rng.standard_normal((T * k, H)), rng.random((T, k)), rng.standard_normal((T, H))
    dYs, dw, _ = routed.combine_grad(dY, Ys, slots, w)

    def loss(Ys, w):
        return float((dY * routed.combine(Ys, slots, w)[0]).sum())

    for t in range(T):
        for j in range(k):
            a, b = w.copy(), w.copy()
            a[t, j] += 0.5
            b[t, j] -= 0.5
            assert abs(loss(Ys, a) - loss(Ys, b) - dw[t, j]) < 1e-12
    for s in range(T * k):
        for h in (0, H - 1):
            a, b = Ys.copy(), Ys.copy()
            a[s, h] += 0.5
            b[s, h] -= 0.5
            want = dYs[s][h] if s in dYs else 0.0
            assert abs(loss(a, w) - loss(b, w) - want) < 1e-12


def test_lora_is_the_merged_weight():
    """A row of adapter a sees the weight s La_a^T Lb_a^T; rows without one see none."""
    rng = np.random.default_rng(5)
    M, K, N, r, L = 6, 12, 10, 4, 3
    A, La, Lb = rng.standard_normal((M, K)), rng.standard_normal((L, r, K)), rng.standard_normal((L, N, r))
    scale, ids = rng.standard_normal(L), np.array([0, 2, -1, 1, 3, 2])
    delta, mag, mag2, _ = routed.lora(A, La, Lb, scale, ids)
    for m, a in enumerate(ids):
        want = A[m] @ (scale[a] * La[a].T @ Lb[a].T) if 0 <= a < L else np.zeros(N)
        assert np.allclose(delta[m], want, rtol=1e-12, atol=1e-12)
        assert (np.abs(delta[m]) <= mag[m] + 1e-12).all() and (mag[m] <= mag2[m] + 1e-12).all()
