"""Pins of the sequence and tree oracle: the dense recurrences, differences, a chain."""

import numpy as np
import pytest

from oracle import recurrences, sequence
from workloads import FORM_GDN, FORM_KDA, FORM_MAMBA2

FORMS = [FORM_GDN, FORM_KDA, FORM_MAMBA2]


def _inputs(form, T, H, dk, dv, rng):
    q, k = rng.normal(size=(2, T, H, dk)) / dk ** 0.5
    v = rng.normal(size=(T, H, dv))
    alpha = rng.uniform(0.5, 1.0, size=(T, H, dk) if form == FORM_KDA else (T, H))
    beta = rng.uniform(0.1, 0.9, size=(T, H))
    return q, k, v, alpha, beta


@pytest.mark.parametrize("form", FORMS)
def test_scan_is_the_dense_recurrence(form):
    rng = np.random.default_rng(form)
    q, k, v, alpha, beta = _inputs(form, 7, 3, 5, 4, rng)
    S0 = rng.normal(size=(3, 5, 4))
    o, S = sequence.scan(form, q, k, v, alpha, beta, S0)
    R = S0
    for t in range(7):
        R = recurrences.dense_step(form, R, k[t], v[t], alpha[t], beta[t])
        np.testing.assert_allclose(o[t], recurrences.readout(R, q[t]), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S, R, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("form", FORMS)
def test_gradients_match_differences(form):
    rng = np.random.default_rng(10 + form)
    q, k, v, alpha, beta = _inputs(form, 5, 2, 4, 3, rng)
    S0 = rng.normal(size=(2, 4, 3))
    do, dS = rng.normal(size=v.shape), rng.normal(size=S0.shape)
    grads = sequence.scan_backward(form, q, k, v, alpha, beta, S0, do, dS)

    def loss(q, k, v, la, beta, S0):
        o, S = sequence.scan(form, q, k, v, np.exp(la), beta, S0)
        return np.sum(o * do) + np.sum(S * dS)

    args = [q, k, v, np.log(alpha), beta, S0]
    h = 1e-5      # central differences: error h^2 of the third derivative, 1e-16 / h of rounding
    for i, g in enumerate(grads):
        num = np.zeros(g.shape)
        for at in np.ndindex(*g.shape):
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[i][at] += h
            lo[i][at] -= h
            num[at] = (loss(*hi) - loss(*lo)) / (2 * h)
        np.testing.assert_allclose(g, num, rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("form", FORMS)
def test_tree_paths_are_scans(form):
    rng = np.random.default_rng(20 + form)
    parent = [-1, 0, 0, 2, -1, -2, 4, 5]
    q, k, v, alpha, beta = _inputs(form, len(parent), 2, 4, 3, rng)
    root = rng.normal(size=(2, 4, 3))
    o, w, states = sequence.tree(form, root, parent, q, k, v, alpha, beta)
    for t in range(len(parent)):
        if t in (5, 7):       # unused, and below an unused node
            assert states[t] is None and not o[t].any() and not w[t].any()
            continue
        p = sequence.path(parent, t)
        os, S = sequence.scan(form, q[p], k[p], v[p], alpha[p], beta[p], root)
        np.testing.assert_allclose(o[t], os[-1], rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(states[t], S, rtol=1e-12, atol=1e-12)
