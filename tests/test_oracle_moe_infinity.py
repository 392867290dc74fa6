"""The 64-bit router form (oracle/moe.py) on logits of +inf, by hand."""

import numpy as np

from oracle import moe

INF = np.inf
L = np.array([[0.0, INF, 1.0, -INF]])


def test_softmax_by_logit():
    with np.errstate(invalid="ignore"):
        for renorm in (True, False):
            idx, w, p = moe.router(L, 4, renormalize=renorm)
            assert idx.tolist() == [[1, 2, 0, -1]]
            assert np.isnan(w[0, :3]).all() and w[0, 3] == 0
            assert np.isnan(p[0, :3]).all() and p[0, 3] == 0


def test_softmax_by_value():
    with np.errstate(invalid="ignore"):
        for kw in (dict(bias=[0.0] * 4), dict(num_groups=2, topk_groups=2, group_top=2)):
            idx, w, p = moe.router(L, 2, **kw)
            assert idx.tolist() == [[-1, -1]] and w.tolist() == [[0, 0]] and np.isnan(p[0, :3]).all()


def test_sigmoid():
    idx, w, p = moe.router(L, 2, "sigmoid", renormalize=False)
    assert idx.tolist() == [[1, 2]] and w[0, 0] == 1.0 and p[0, 3] == 0


def test_backward():
    with np.errstate(invalid="ignore"):
        g = moe.router_backward(L, np.array([[1, 2]]), np.ones((1, 2)), np.ones((1, 4)), renormalize=False)
    assert np.isnan(g[0, :3]).all() and g[0, 3] == 0
    with np.errstate(over="ignore"):
        g = moe.router_backward(L, np.array([[1, 2]]), np.array([[1.0, -1.0]]), None, "sigmoid")
    assert np.isfinite(g).all() and g[0, 1] == 0 and g[0, 3] == 0
